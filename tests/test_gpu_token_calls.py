"""Calls of the token operators that the header allows and that the other files do not make."""
import threading

import numpy as np
import pytest

from oracle import token_oracle as o
from token_testutil import U32, code_of, dtype_of, f64, inside

pytestmark = pytest.mark.gpu

EPS = 1e-5


def _norm_inputs(n, D, dtype, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    X, dY = (torch.randn(n, D, device="cuda", generator=g).to(dtype_of(dtype)) for _ in range(2))
    W, b = torch.rand(2, D, device="cuda", generator=g)
    return X, dY, W, b


@pytest.mark.parametrize("D,dtype,pad", [(4096, "bf16", 0), (1001, "bf16", 0), (72, "bf16", 8), (77, "bf16", 3),
                                         (1001, "f32", 0), (60, "f32", 0)])
def test_gradient_over_dy_from_codes(D, dtype, pad):
    """dX may be dY where their strides agree, from codes as from X."""
    import torch
    from frame_wise_linear_b200 import vda
    n = 2501
    X, dY, W, b = _norm_inputs(n, D, dtype)
    ld = D + pad
    p = vda.make_norm_problem(n, D, code_of(dtype), eps=EPS, ld_x=ld, ld_y=ld)
    codes = torch.empty(n, D, dtype=torch.uint8, device="cuda")
    scales = torch.empty(n, -(-D // 32), dtype=torch.uint8, device="cuda")
    A, G, out = (inside(n, D, ld, X.dtype, 7.0)[0] for _ in range(3))
    A.copy_(X)
    G.copy_(dY)
    mean, rstd = torch.empty(2, n, device="cuda")
    vda.vda_layer_norm(p, A, W, b, out, mean, rstd, codes, scales)
    ws = torch.empty(vda.vda_layer_norm_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
    first, second = torch.empty(2, D, device="cuda"), torch.empty(2, D, device="cuda")
    vda.vda_layer_norm_backward_from_checkpoint(p, G, codes, scales, rstd, W, out, *first, ws)
    vda.vda_layer_norm_backward_from_checkpoint(p, G, codes, scales, rstd, W, G, *second, ws)
    assert torch.equal(G, out) and torch.equal(first, second)


@pytest.mark.parametrize("D,dtype", [(4096, "bf16"), (64, "f32"), (1001, "bf16")])
def test_codes_at_any_place(D, dtype):
    """Codes and scales behind other bytes: the same codes, and the same gradients to the rounding of another order."""
    import torch
    from frame_wise_linear_b200 import vda
    n, nblk = 700, -(-D // 32)
    X, dY, W, b = _norm_inputs(n, D, dtype)
    p = vda.make_norm_problem(n, D, code_of(dtype), eps=EPS)
    ws = torch.empty(vda.vda_layer_norm_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
    want = None
    for place in (0, 1, 4, 7):
        cfull, sfull = (torch.full((place + k + 64,), 9, dtype=torch.uint8, device="cuda") for k in (n * D, n * nblk))
        codes, scales = cfull[place: place + n * D].view(n, D), sfull[place: place + n * nblk].view(n, nblk)
        Y, dX, (mean, rstd), (dW, db) = torch.empty_like(X), torch.empty_like(X), torch.empty(2, n, device="cuda"), \
            torch.empty(2, D, device="cuda")
        vda.vda_layer_norm(p, X, W, b, Y, mean, rstd, codes, scales)
        c, s = o.checkpoint(f64((X.float() - mean[:, None]) * rstd[:, None]))
        assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s)
        if want is None:
            kept = codes.clone(), scales.clone(), rstd.clone()
        codes.copy_(kept[0])
        scales.copy_(kept[1])
        vda.vda_layer_norm_backward_from_checkpoint(p, dY, codes, scales, kept[2], W, dX, dW, db, ws)
        got = [f64(t) for t in (dW, db)]
        want = want or got
        size = [np.abs(f64(dY) * (o.checkpoint_values(*(k.cpu().numpy() for k in kept[:2])) if i == 0 else 1)).sum(0)
                for i in range(2)]
        for a, ref, total in zip(got, want, size):
            assert np.all(np.abs(a - ref) <= 2 * (n + 82) * U32 * total)     # both sides' sums
        assert bool((cfull[place + n * D:] == 9).all()) and bool((sfull[place + n * nblk:] == 9).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("d,axes", [(128, (16, 24, 24)), (72, (2, 4, 4)), (63, (18, 20, 22)), (70, (8, 10, 16))])
def test_channels_that_do_not_turn_keep_every_bit(d, axes, halves, dtype):
    """Any bit pattern, signalling NaN among them, in either direction and layout."""
    import torch
    from frame_wise_linear_b200 import vda
    dt = dtype_of(dtype)
    ints = {2: torch.int16, 4: torch.int32}[dt.itemsize]
    g = torch.Generator(device="cuda").manual_seed(d)
    info = torch.iinfo(ints)
    for layout in (0, 1):
        bits = torch.randint(info.min, info.max, (2, 3, 40, d) if layout == 0 else (2, 40, 3, d), device="cuda",
                             generator=g, dtype=torch.int64).to(ints)
        bits[..., -1] = torch.tensor(0x7F81 if dt.itemsize == 2 else 0x7F800001, dtype=ints)    # a signalling NaN
        x = bits.view(dt)
        p = vda.make_rope_problem(2, 2, 4, 5, 3, 0, d, axes, code_of(dtype), layout=layout, pairing=int(halves))
        for call in (vda.vda_rope, vda.vda_rope_backward):
            y = torch.zeros_like(x)
            call(p, x, None, None, y, None)
            assert torch.equal(y.view(ints)[..., sum(axes):], bits[..., sum(axes):])


def test_far_positions():
    """Positions of 10^8: the angle's double product is off by at most 3 half steps of 2^-53 of 1.6e7 turns, 3.3e-8
    rad or half a u; the reference's angles have 64 bits."""
    import torch
    from frame_wise_linear_b200 import vda
    if np.finfo(np.longdouble).nmant < 63:
        pytest.skip("no wider type than double here")
    d, axes, N = 128, (44, 42, 42), 50
    x = torch.randn(1, N, 2, d, device="cuda")
    y = torch.empty_like(x)
    pos0 = (1e8, 1e8 - 7, -1e8)
    p = vda.make_rope_problem(1, N, 1, 1, 2, 0, d, axes, vda.VDA_DTYPE_F32, layout=1, pos0=pos0)
    vda.vda_rope(p, x, None, None, y, None)
    L = np.longdouble
    pos = np.stack([L(pos0[0]) + np.arange(N, dtype=L), np.full(N, L(pos0[1])), np.full(N, L(pos0[2]))], 1)
    angle = np.concatenate([pos[:, [a]] * L(10000) ** (-np.arange(0, n, 2, dtype=L) / n) for a, n in enumerate(axes)], 1)
    c, s = np.cos(angle)[:, None].astype(float), np.sin(angle)[:, None].astype(float)
    a = f64(x)[0]
    u, v = a[..., 0::2], a[..., 1::2]
    bound = 9.5 * U32 * (np.abs(u) + np.abs(v))
    got = f64(y)[0]
    assert np.all(np.abs(got[..., 0::2] - (u * c - v * s)) <= bound + U32 * np.abs(got[..., 0::2]))
    assert np.all(np.abs(got[..., 1::2] - (u * s + v * c)) <= bound + U32 * np.abs(got[..., 1::2]))


class _Work:
    """The four groups of operators once, on tensors of one's own."""

    def __init__(self, seed):
        import torch
        from frame_wise_linear_b200 import vda
        n, D, H = 1200, 1001, 8
        self.X, self.dY, self.W, self.b = _norm_inputs(n, D, "bf16", seed)
        self.p = vda.make_norm_problem(n, D, vda.VDA_DTYPE_BF16, eps=EPS)
        self.codes = torch.empty(n, D, dtype=torch.uint8, device="cuda")
        self.scales = torch.empty(n, 32, dtype=torch.uint8, device="cuda")
        self.Y, self.dX, self.back = (torch.empty_like(self.X) for _ in range(3))
        self.stats, self.sums = torch.empty(2, n, device="cuda"), torch.empty(2, D, device="cuda")
        self.ws = torch.empty(vda.vda_layer_norm_backward_workspace_size(self.p), dtype=torch.uint8, device="cuda")
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.q = torch.randn(1, n, H, 128, device="cuda", generator=g).bfloat16()
        self.qr, self.dq = torch.empty_like(self.q), torch.empty_like(self.q)
        self.r = vda.make_rope_problem(1, 1, 30, 40, H, 0, 128, (44, 42, 42), vda.VDA_DTYPE_BF16, layout=1)
        self.c = vda.make_checkpoint_problem(n, D, vda.VDA_DTYPE_BF16)

    def run(self, stream=None):
        from frame_wise_linear_b200 import vda
        kw = dict(stream=stream)
        vda.vda_layer_norm(self.p, self.X, self.W, self.b, self.Y, *self.stats, self.codes, self.scales, **kw)
        vda.vda_layer_norm_backward(self.p, self.dY, self.X, *self.stats, self.W, self.dX, *self.sums, self.ws, **kw)
        vda.vda_rope(self.r, self.q, None, None, self.qr, None, **kw)
        vda.vda_rope_backward(self.r, self.qr, None, None, self.dq, None, **kw)
        vda.vda_checkpoint_unpack(self.c, self.codes, self.scales, self.back, **kw)

    def outputs(self):
        return [self.Y, self.dX, self.stats, self.sums, self.codes, self.scales, self.qr, self.dq, self.back]


def _expected(works):
    import torch
    for w in works:
        w.run()
    torch.cuda.synchronize()
    want = [[t.clone() for t in w.outputs()] for w in works]
    for w in works:
        for t in w.outputs():
            t.zero_()
    torch.cuda.synchronize()
    return want


def test_calls_from_several_threads():
    """Four host threads, each with its own stream and tensors, enqueue at once."""
    import torch
    works = [_Work(s) for s in range(4)]
    want = _expected(works)
    streams = [torch.cuda.Stream() for _ in works]
    failed = []

    def go(w, s):
        try:
            for _ in range(30):
                w.run(s)
            s.synchronize()
        except Exception as e:     # a thread's exception would be lost
            failed.append(e)

    threads = [threading.Thread(target=go, args=a) for a in zip(works, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for w, ref in zip(works, want):
        assert all(torch.equal(a, c) for a, c in zip(w.outputs(), ref))


def test_graphs_replayed_at_once():
    """Two captured graphs, each with its own workspace, replayed on two streams at the same time."""
    import torch
    works = [_Work(s) for s in (7, 8)]
    want = _expected(works)
    graphs, streams = [], [torch.cuda.Stream() for _ in works]
    for w, s in zip(works, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            w.run()
        graphs.append(g)
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for w, ref in zip(works, want):
        assert all(torch.equal(a, c) for a, c in zip(w.outputs(), ref))
