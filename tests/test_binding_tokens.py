"""The token operators' binding refuses tensors that their kernels could not reach (no GPU needed)."""
import pytest

from frame_wise_linear_b200 import build, vda

OK = 1 << 20      # never dereferenced
F32 = vda.VDA_DTYPE_F32


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return vda.load()


class _On:
    """A tensor of another device, as far as the binding looks at it."""

    def __init__(self, device):
        self.device = device

    def get_device(self):
        return self.device

    def data_ptr(self):
        raise AssertionError("the address of a tensor that must be refused")


def _calls():
    """Every token operator as a function of its pointers, and their number."""
    n = vda.make_norm_problem(4, 64, F32)
    r = vda.make_rope_problem(1, 1, 1, 4, 1, 1, 64, (16, 24, 24), F32)
    c = vda.make_checkpoint_problem(4, 64, F32)
    p = vda.make_problem(B=1, H=2, T=3, n=64, n_txt=8, d_k=128, d_v=128, dtype=vda.VDA_DTYPE_BF16, lam=1.0)
    kw = dict(stream=0, check=False)
    wb = dict(kw, workspace_bytes=1 << 40)
    pairs = lambda a: list(zip(a[0:12:2], a[1:12:2]))  # noqa: E731
    return [
        (lambda *a: vda.vda_layer_norm(n, *a, **kw), 8),
        (lambda *a: vda.vda_layer_norm_from_checkpoint(n, *a, **kw), 5),
        (lambda *a: vda.vda_layer_norm_backward(n, *a, **wb), 9),
        (lambda *a: vda.vda_layer_norm_backward_from_checkpoint(n, *a, **wb), 9),
        (lambda *a: vda.vda_rope(r, *a, **kw), 5),
        (lambda *a: vda.vda_rope_backward(r, *a, **kw), 5),
        (lambda *a: vda.vda_checkpoint_pack(c, *a, **kw), 3),
        (lambda *a: vda.vda_checkpoint_unpack(c, *a, **kw), 3),
        (lambda *a: vda.vda_backward_from_checkpoint(p, pairs(a), *a[12:], **wb), 20),
    ]


@pytest.mark.parametrize("which", range(9))
def test_host_tensors_refused(which):
    import torch
    call, count = _calls()[which]
    for i in range(count):
        a = [OK] * count
        a[i] = torch.zeros(64)
        with pytest.raises(ValueError, match="CUDA"):
            call(*a)


@pytest.mark.parametrize("which", range(9))
def test_tensors_of_another_device_refused(which, monkeypatch):
    monkeypatch.setattr(vda, "_current_device", lambda: 0)
    call, count = _calls()[which]
    for i in range(count):
        a = [OK] * count
        a[i] = _On(1)
        with pytest.raises(ValueError, match="device 1"):
            call(*a)


@pytest.mark.parametrize("fn", ["vda_layer_norm_backward", "vda_layer_norm_backward_from_checkpoint"])
def test_no_workspace_is_an_argument_like_others(fn):
    """None for the workspace, its size not given: refused by the library where weight gradients are wanted, and
    taken where there are none (here with no tokens, so that nothing runs)."""
    call = getattr(vda, fn)
    some, none = vda.make_norm_problem(4, 64, F32), vda.make_norm_problem(0, 64, F32)
    for dw, db in ((OK, OK), (OK, None), (None, OK)):
        assert call(some, OK, OK, OK, OK, OK, OK, dw, db, None, stream=0, check=False) == vda.VDA_ERR_WORKSPACE
    assert call(none, None, None, None, None, None, None, None, None, None, stream=0, check=False) == vda.VDA_OK
