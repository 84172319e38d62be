"""The token operators' C ABI on the host: struct layouts and refusals (no GPU needed).

Every call here fails its host-side checks before anything is enqueued, or has
nothing to do; the calls that pass run only where no CUDA device exists and
must then fail loudly.
"""
import ctypes

import pytest

from frame_wise_linear_b200 import build, vda

OK = 1 << 20      # never dereferenced
F32, BF16 = vda.VDA_DTYPE_F32, vda.VDA_DTYPE_BF16


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return vda.load()


def test_struct_layouts():
    # the header's fields in order, no padding
    assert ctypes.sizeof(vda.vda_norm_problem) == 48
    assert vda.vda_norm_problem.heads.offset == 24 and vda.vda_norm_problem.eps.offset == 40
    assert ctypes.sizeof(vda.vda_rope_problem) == 144
    assert vda.vda_rope_problem.theta.offset == 32 and vda.vda_rope_problem.B.offset == 88
    assert ctypes.sizeof(vda.vda_checkpoint_problem) == 24
    assert ctypes.sizeof(vda.vda_checkpoint) == 16


def _norm(**kw):
    base = dict(tokens=4, D=64, dtype=BF16)
    base.update(kw)
    return vda.make_norm_problem(**base)


def _norm_calls(p, fwd=(OK,) * 4, bwd=(OK,) * 8, ws=OK, ws_bytes=1 << 40):
    """The status of every layer norm entry point on one problem."""
    X, W, b, Y = fwd
    kw = dict(stream=0, check=False)
    return (vda.vda_layer_norm(p, X, W, b, Y, OK, OK, **kw),
            vda.vda_layer_norm_from_checkpoint(p, OK, OK, W, b, Y, **kw),
            vda.vda_layer_norm_backward(p, *bwd, ws, workspace_bytes=ws_bytes, **kw),
            vda.vda_layer_norm_backward_from_checkpoint(p, *bwd, ws, workspace_bytes=ws_bytes, **kw))


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), vda.VDA_ERR_INVALID_ARG),
    (dict(tokens=1 << 31), vda.VDA_ERR_INVALID_ARG),
    (dict(D=0), vda.VDA_ERR_INVALID_ARG),
    (dict(D=8193), vda.VDA_ERR_UNSUPPORTED),
    (dict(heads=0), vda.VDA_ERR_INVALID_ARG),
    (dict(heads=65537), vda.VDA_ERR_UNSUPPORTED),
    (dict(dtype=vda.VDA_DTYPE_E4M3), vda.VDA_ERR_INVALID_ARG),
    (dict(dtype=9), vda.VDA_ERR_INVALID_ARG),
    (dict(w_dtype=vda.VDA_DTYPE_E4M3), vda.VDA_ERR_INVALID_ARG),
    (dict(eps=0.0), vda.VDA_ERR_INVALID_ARG),
    (dict(eps=-1.0), vda.VDA_ERR_INVALID_ARG),
    (dict(eps=float("nan")), vda.VDA_ERR_INVALID_ARG),
    (dict(eps=float("inf")), vda.VDA_ERR_INVALID_ARG),
    (dict(ld_x=63), vda.VDA_ERR_INVALID_ARG),
    (dict(ld_y=-64), vda.VDA_ERR_INVALID_ARG),
    (dict(ld_y=1 << 31), vda.VDA_ERR_INVALID_ARG),
    (dict(heads=2, ld_x=127), vda.VDA_ERR_INVALID_ARG),
])
def test_norm_problem_refused(kw, status):
    p = _norm(**kw)
    assert set(_norm_calls(p)) == {status}, vda.vda_last_error()
    out = ctypes.c_size_t(0)
    assert vda.load().vda_layer_norm_backward_workspace_size(ctypes.byref(p), ctypes.byref(out)) == status
    assert vda.vda_last_error()


def test_norm_reserved_and_null_problem(lib):
    p = _norm()
    p.reserved = 1
    assert set(_norm_calls(p)) == {vda.VDA_ERR_INVALID_ARG}
    assert lib.vda_layer_norm(None, *([OK] * 9)) == vda.VDA_ERR_INVALID_ARG
    assert lib.vda_layer_norm_backward_workspace_size(ctypes.byref(_norm()), None) == vda.VDA_ERR_INVALID_ARG


def test_norm_pointers_refused():
    p, kw = _norm(), dict(stream=0, check=False)
    bad = vda.VDA_ERR_INVALID_ARG
    for x in (0, OK + 1):                       # NULL, or not at an element
        assert vda.vda_layer_norm(p, x, OK, OK, OK, **kw) == bad
        assert vda.vda_layer_norm(p, OK, OK, OK, x, **kw) == bad
        for i in (0, 1, 2, 3, 5):               # dY, X, mean, rstd, dX
            a = [OK] * 8
            a[i] = x
            assert vda.vda_layer_norm_backward(p, *a, OK, workspace_bytes=1 << 40, **kw) == bad, i
        for i in (0, 3, 5):                     # dY, rstd, dX
            a = [OK] * 8
            a[i] = x
            assert vda.vda_layer_norm_backward_from_checkpoint(p, *a, OK, workspace_bytes=1 << 40, **kw) == bad, i
    assert vda.vda_layer_norm(p, OK, OK + 2, OK, OK, **kw) == bad          # W float32 at a half element
    assert vda.vda_layer_norm(p, OK, OK, OK, OK, OK + 2, **kw) == bad      # mean
    assert vda.vda_layer_norm(p, OK, OK, OK, OK, OK, OK, OK, None, **kw) == bad   # codes alone
    assert vda.vda_layer_norm(p, OK, OK, OK, OK, OK, OK, None, OK, **kw) == bad
    assert vda.vda_layer_norm_from_checkpoint(p, None, OK, OK, OK, OK, **kw) == bad
    a = [OK] * 8
    a[1] = None                                                               # codes
    assert vda.vda_layer_norm_backward_from_checkpoint(p, *a, OK, workspace_bytes=1 << 40, **kw) == bad


def test_norm_backward_workspace_checked():
    p, kw = _norm(), dict(stream=0, check=False)
    need = vda.vda_layer_norm_backward_workspace_size(p)
    assert need >= 2 * 64 * 4
    for ws, nb in ((None, need), (OK + 16, need), (OK, need - 1)):
        for fn in (vda.vda_layer_norm_backward, vda.vda_layer_norm_backward_from_checkpoint):
            assert fn(p, *([OK] * 8), ws, workspace_bytes=nb, **kw) == vda.VDA_ERR_WORKSPACE
    assert vda.vda_layer_norm_backward_workspace_size(_norm(tokens=0)) == 0


def _rope(**kw):
    base = dict(B=1, T=2, height=3, width=4, H_q=2, H_k=1, d=64, axes=(16, 24, 24), dtype=BF16)
    base.update(kw)
    return vda.make_rope_problem(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), vda.VDA_ERR_INVALID_ARG),
    (dict(T=-1), vda.VDA_ERR_INVALID_ARG),
    (dict(height=-2), vda.VDA_ERR_INVALID_ARG),
    (dict(T=1 << 16, height=1 << 15), vda.VDA_ERR_UNSUPPORTED),
    (dict(B=2**31 - 1, T=2**31 - 1, height=2**31 - 1, width=2**31 - 1), vda.VDA_ERR_UNSUPPORTED),
    (dict(H_q=-1), vda.VDA_ERR_INVALID_ARG),
    (dict(H_q=65535, H_k=1), vda.VDA_ERR_INVALID_ARG),
    (dict(d=0), vda.VDA_ERR_INVALID_ARG),
    (dict(d=258), vda.VDA_ERR_UNSUPPORTED),
    (dict(axes=(16, 24, 26)), vda.VDA_ERR_INVALID_ARG),         # more channels than the head has
    (dict(axes=(15, 24, 24)), vda.VDA_ERR_INVALID_ARG),         # odd
    (dict(axes=(-2, 24, 24)), vda.VDA_ERR_INVALID_ARG),
    (dict(axes=(2**31 - 2, 2**31 - 2, 2**31 - 2)), vda.VDA_ERR_INVALID_ARG),
    (dict(dtype=vda.VDA_DTYPE_E4M3), vda.VDA_ERR_INVALID_ARG),
    (dict(layout=2), vda.VDA_ERR_INVALID_ARG),
    (dict(pairing=2), vda.VDA_ERR_INVALID_ARG),
    (dict(theta=0.0), vda.VDA_ERR_INVALID_ARG),
    (dict(theta=float("inf")), vda.VDA_ERR_INVALID_ARG),
    (dict(pos0=(0.0, float("nan"), 0.0)), vda.VDA_ERR_INVALID_ARG),
    (dict(step=(float("inf"), 1.0, 1.0)), vda.VDA_ERR_INVALID_ARG),
    (dict(ld_q=128), vda.VDA_ERR_INVALID_ARG),                  # strides are the token-major layout's
    (dict(layout=1, ld_q=127), vda.VDA_ERR_INVALID_ARG),
    (dict(layout=1, ld_kr=63), vda.VDA_ERR_INVALID_ARG),
    (dict(layout=1, ld_qr=1 << 31), vda.VDA_ERR_INVALID_ARG),
    (dict(layout=1, ld_k=-64), vda.VDA_ERR_INVALID_ARG),
])
def test_rope_problem_refused(kw, status):
    p = _rope(**kw)
    for fn in (vda.vda_rope, vda.vda_rope_backward):
        assert fn(p, OK, OK, None, OK, OK, stream=0, check=False) == status, vda.vda_last_error()


def test_rope_pointers_refused():
    p, bad = _rope(), vda.VDA_ERR_INVALID_ARG
    for fn in (vda.vda_rope, vda.vda_rope_backward):
        for i in (0, 1, 3, 4):
            for x in (0, OK + 1):
                a = [OK, OK, None, OK, OK]
                a[i] = x
                assert fn(p, *a, stream=0, check=False) == bad, (i, x)
        assert fn(p, OK, OK, OK + 2, OK, OK, stream=0, check=False) == bad   # positions at a half element
    p.reserved = 3
    assert vda.vda_rope(p, OK, OK, None, OK, OK, stream=0, check=False) == bad


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), vda.VDA_ERR_INVALID_ARG),
    (dict(rows=(1 << 40) + 1), vda.VDA_ERR_INVALID_ARG),
    (dict(rows=1 << 40, D=64), vda.VDA_ERR_UNSUPPORTED),         # 2^46 elements
    (dict(D=0), vda.VDA_ERR_INVALID_ARG),
    (dict(D=(1 << 24) + 1), vda.VDA_ERR_UNSUPPORTED),
    (dict(dtype=vda.VDA_DTYPE_E4M3), vda.VDA_ERR_INVALID_ARG),
    (dict(ld=63), vda.VDA_ERR_INVALID_ARG),
    (dict(ld=1 << 31), vda.VDA_ERR_INVALID_ARG),
])
def test_checkpoint_problem_refused(kw, status):
    base = dict(rows=4, D=64, dtype=BF16)
    base.update(kw)
    p = vda.make_checkpoint_problem(**base)
    for fn in (vda.vda_checkpoint_pack, vda.vda_checkpoint_unpack):
        assert fn(p, OK, OK, OK, stream=0, check=False) == status, vda.vda_last_error()


def test_checkpoint_pointers_refused():
    p = vda.make_checkpoint_problem(4, 64, F32)
    for i in range(3):
        a = [OK] * 3
        a[i] = 0
        assert vda.vda_checkpoint_pack(p, *a, stream=0, check=False) == vda.VDA_ERR_INVALID_ARG
        assert vda.vda_checkpoint_unpack(p, *a, stream=0, check=False) == vda.VDA_ERR_INVALID_ARG
    assert vda.vda_checkpoint_pack(p, OK + 2, OK, OK, stream=0, check=False) == vda.VDA_ERR_INVALID_ARG


def test_backward_from_checkpoint_refused(lib):
    p = vda.make_problem(B=1, H=2, T=3, n=64, n_txt=8, d_k=128, d_v=128, dtype=BF16, lam=1.0)
    need = vda.vda_backward_from_checkpoint_workspace_size(p)
    assert need >= vda.vda_backward_workspace_size(p) + (4 * 2 * 3 * 64 + 2 * 2 * 8) * 128 * 2
    good = [(OK, OK)] * 6
    call = lambda c=good, g=(OK,) * 7, ws=OK, nb=need, q=p: vda.vda_backward_from_checkpoint(  # noqa: E731
        q, c, *g, ws, stream=0, workspace_bytes=nb, check=False)
    for i in range(6):
        for pair in ((None, OK), (OK, None)):
            c = list(good)
            c[i] = pair
            assert call(c) == vda.VDA_ERR_INVALID_ARG, vda.vda_last_error()
    for i in range(7):                          # dO, the four gradients, the text's two
        for x in (0, OK + 8):
            g = [OK] * 7
            g[i] = x
            assert call(g=g) == vda.VDA_ERR_INVALID_ARG, vda.vda_last_error()
    assert call(ws=None) == vda.VDA_ERR_WORKSPACE
    assert call(ws=OK + 16) == vda.VDA_ERR_WORKSPACE
    assert call(nb=need - 1) == vda.VDA_ERR_WORKSPACE
    f32 = vda.make_problem(B=1, H=2, T=3, n=64, n_txt=8, d_k=128, d_v=128, dtype=F32, lam=1.0)
    assert call(q=f32) == vda.VDA_ERR_UNSUPPORTED
    assert lib.vda_backward_from_checkpoint(ctypes.byref(p), None, *([OK] * 8), need, 0) == vda.VDA_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        vda.vda_backward_from_checkpoint(p, good[:5], *([OK] * 7), OK, stream=0, workspace_bytes=need)


def test_empty_calls_need_no_tensors():
    """No tokens: nothing is read, enqueued or refused (weight gradients aside, which become 0 on the device)."""
    p, kw = _norm(tokens=0), dict(stream=0, check=False)
    assert vda.vda_layer_norm(p, None, None, None, None, **kw) == vda.VDA_OK
    assert vda.vda_layer_norm_from_checkpoint(p, None, None, None, None, None, **kw) == vda.VDA_OK
    for fn in (vda.vda_layer_norm_backward, vda.vda_layer_norm_backward_from_checkpoint):
        assert fn(p, None, None, None, None, None, None, None, None, None, workspace_bytes=0, **kw) == vda.VDA_OK
    for kw2 in (dict(B=0), dict(T=0), dict(height=0), dict(width=0), dict(T=0, height=2**31 - 1, width=2**31 - 1),
                dict(H_q=0, H_k=0)):
        assert vda.vda_rope(_rope(**kw2), None, None, None, None, None, **kw) == vda.VDA_OK, vda.vda_last_error()
    e = vda.make_checkpoint_problem(0, 64, BF16)
    assert vda.vda_checkpoint_pack(e, None, None, None, **kw) == vda.VDA_OK
    assert vda.vda_checkpoint_unpack(e, None, None, None, **kw) == vda.VDA_OK


def _has_cuda():
    try:
        import torch
        return torch.cuda.is_available()
    except Exception:
        return False


@pytest.mark.skipif(_has_cuda(), reason="only meaningful where no CUDA device exists")
def test_no_device_fails_loudly():
    kw = dict(stream=0, check=False)
    assert set(_norm_calls(_norm())) == {vda.VDA_ERR_CUDA}
    assert vda.vda_rope(_rope(), OK, OK, None, OK, OK, **kw) == vda.VDA_ERR_CUDA
    p = vda.make_checkpoint_problem(4, 64, BF16)
    assert vda.vda_checkpoint_pack(p, OK, OK, OK, **kw) == vda.VDA_ERR_CUDA
    assert vda.vda_checkpoint_unpack(p, OK, OK, OK, **kw) == vda.VDA_ERR_CUDA
