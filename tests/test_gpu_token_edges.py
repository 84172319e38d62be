"""The token operators where their tensors' edges are: rows of odd widths that share vectors with their neighbours,
tensors that start inside a vector, few rows, NaN all around, both sides of every rule that picks a kernel's form."""
import numpy as np
import pytest

from oracle import token_oracle as o
from token_testutil import U32, assert_close, code_of, dtype_of, f64, half_step, inside, untouched

pytestmark = pytest.mark.gpu

EPS = 1e-5
NAN = float("nan")


def _fill(view, rng, shift=0.0):
    import torch
    view.copy_(torch.from_numpy(rng.normal(shift, 1.0, tuple(view.shape))).cuda())


# Rows, width, type, elements before the tensors: dense rows, at every shift that a row can have in a vector.
SHIFTED = [(rows, D, dtype, off) for dtype in ("bf16", "f32") for D in (33, 63, 130, 1001, 2050, 4097)
           for rows, off in ((1, 0), (3, 1), (8, 3), (45, 0), (300, 5))]


@pytest.mark.parametrize("rows,D,dtype,off", SHIFTED)
def test_odd_rows_among_nan(rows, D, dtype, off):
    """Nothing from outside a tensor reaches a result, and nothing outside is written: every input stands among NaN.
    Bounds as in the layer norm's own tests."""
    import torch
    from frame_wise_linear_b200 import vda
    rng = np.random.default_rng(rows * D + off)
    dt = dtype_of(dtype)
    X, _ = inside(rows, D, D, dt, NAN, off)
    dY, _ = inside(rows, D, D, dt, NAN, off)
    _fill(X, rng, 0.5)
    _fill(dY, rng)
    W, b = (torch.from_numpy(rng.normal(m, 0.3, D)).float().cuda() for m in (1.0, 0.0))
    p = vda.make_norm_problem(rows, D, code_of(dtype), eps=EPS)
    x, dy = f64(X), f64(dY)
    y_ref, m, r, xh = o.layer_norm(x, f64(W), f64(b), EPS)
    Y, yfull = inside(rows, D, D, dt, 7.0, off)
    mean, rstd = torch.empty(2, rows, device="cuda")
    vda.vda_layer_norm(p, X, W, b, Y, mean, rstd)
    XR = (np.abs(x).max(1) + np.abs(m)) * r
    xb = (47 * U32 * XR)[:, None] + np.abs(xh) * (64 * U32 + 2 * (47 * U32 * XR[:, None]) ** 2)
    wa = np.abs(f64(W))
    assert_close(f64(Y), y_ref, xb * wa + 3 * U32 * (np.abs(xh) * wa + np.abs(y_ref)) +
                 half_step(dt) * np.abs(y_ref) * (1 + 2.0 ** -6), "Y")
    assert untouched(yfull, Y, 7.0)

    mean, rstd = (torch.from_numpy(v).float().cuda() for v in (m, r))
    m, r = f64(mean), f64(rstd)
    ws = torch.full((vda.vda_layer_norm_backward_workspace_size(p),), 255, dtype=torch.uint8, device="cuda")
    c, s = o.checkpoint(xh.astype(np.float32))
    codes = torch.full((off + rows * D + 64,), 0x7F, dtype=torch.uint8, device="cuda")[off: off + rows * D].view(rows, D)
    codes.copy_(torch.from_numpy(c).cuda())
    scales = torch.from_numpy(s).cuda()
    for ckpt in (False, True):
        h = o.checkpoint_values(c, s) if ckpt else (x - m[:, None]) * r[:, None]
        hb = 0.0 if ckpt else 3 * U32 * ((np.abs(x).max(1) + np.abs(m)) * r)[:, None]
        dX, full = inside(rows, D, D, dt, 7.0, off)
        dW, db = torch.full((2, D), 7.0, device="cuda")
        if ckpt:
            vda.vda_layer_norm_backward_from_checkpoint(p, dY, codes, scales, rstd, W, dX, dW, db, ws)
        else:
            vda.vda_layer_norm_backward(p, dY, X, mean, rstd, W, dX, dW, db, ws)
        dx_ref, dw_ref, db_ref = o.layer_norm_backward(dy, h, r, f64(W))
        g = np.abs(dy) * wa
        gx = (g * (np.abs(h) + hb)).mean(1, keepdims=True)
        err = r[:, None] * (U32 * (6 * g + 50 * g.mean(1, keepdims=True) + (50 * np.abs(h) + 6) * gx) + hb * gx +
                            (np.abs(h) + hb) * (g * hb).mean(1, keepdims=True))
        assert_close(f64(dX), dx_ref, err + half_step(dt) * (np.abs(dx_ref) + err), "dX")
        assert untouched(full, dX, 7.0)
        assert_close(f64(dW), dw_ref, 192 * U32 * np.abs(dy * h).sum(0) + (np.abs(dy) * hb).sum(0), "dW")
        assert_close(f64(db), db_ref, 192 * U32 * np.abs(dy).sum(0), "db")
    v = o.checkpoint_values(c, s)
    Y, yfull = inside(rows, D, D, dt, 7.0, off)
    vda.vda_layer_norm_from_checkpoint(p, codes, scales, W, b, Y)
    ref = v * f64(W) + f64(b)
    assert_close(f64(Y), ref, 2 * U32 * (np.abs(v) * wa + np.abs(ref)) + half_step(dt) * np.abs(ref) * (1 + 2.0 ** -6))
    assert untouched(yfull, Y, 7.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [1001, 130])
def test_odd_rows_in_place(D, dtype):
    """Y over X, dX over X and over dY, where neighbouring rows share a vector and belong to other CTAs."""
    import torch
    from frame_wise_linear_b200 import vda
    n, dt = 700, dtype_of(dtype)
    g = torch.Generator(device="cuda").manual_seed(D)
    X, dY = (torch.randn(n, D, device="cuda", generator=g).to(dt) for _ in range(2))
    W, b = torch.randn(2, D, device="cuda", generator=g)
    p = vda.make_norm_problem(n, D, code_of(dtype), eps=EPS)
    Y, dX, (mean, rstd) = torch.empty_like(X), torch.empty_like(X), torch.empty(2, n, device="cuda")
    vda.vda_layer_norm(p, X, W, b, Y, mean, rstd)
    ws = torch.empty(vda.vda_layer_norm_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
    dW, db = torch.empty(2, D, device="cuda")
    vda.vda_layer_norm_backward(p, dY, X, mean, rstd, W, dX, dW, db, ws)
    for _ in range(20):
        a = X.clone()
        vda.vda_layer_norm(p, a, W, b, a)
        assert torch.equal(a, Y)
        for over in ("X", "dY"):
            a, c = X.clone(), dY.clone()
            dW2, db2 = torch.empty(2, D, device="cuda")
            vda.vda_layer_norm_backward(p, c, a, mean, rstd, W, a if over == "X" else c, dW2, db2, ws)
            assert torch.equal(a if over == "X" else c, dX) and torch.equal(dW2, dW) and torch.equal(db2, db)


@pytest.mark.parametrize("D", [128, 1001, 4096])
def test_unlike_alignments(D):
    """One tensor at another place in a vector than the others: the same values from another form of the kernel, to
    their rounding (float32: 100 u of the row's size covers both forms' bounds)."""
    import torch
    from frame_wise_linear_b200 import vda
    n = 40
    rng = np.random.default_rng(D)
    W, b = (torch.from_numpy(rng.normal(m, 0.3, D)).float().cuda() for m in (1.0, 0.0))
    p = vda.make_norm_problem(n, D, vda.VDA_DTYPE_F32, eps=EPS)
    outs = []
    for places in ((0, 0, 0), (1, 0, 0), (0, 2, 0), (0, 0, 3), (1, 2, 3)):
        rng = np.random.default_rng(D + 1)
        X, dY = (inside(n, D, D, torch.float32, NAN, k)[0] for k in places[:2])
        _fill(X, rng)
        _fill(dY, rng)
        Y, dX = (inside(n, D, D, torch.float32, 7.0, places[2])[0] for _ in range(2))
        mean, rstd = torch.empty(2, n, device="cuda")
        dW, db = torch.empty(2, D, device="cuda")
        ws = torch.empty(vda.vda_layer_norm_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
        vda.vda_layer_norm(p, X, W, b, Y, mean, rstd)
        vda.vda_layer_norm_backward(p, dY, X, mean, rstd, W, dX, dW, db, ws)
        outs.append([f64(t) for t in (Y, dX, dW, db, mean, rstd)])
    for other in outs[1:]:
        for a, c in zip(outs[0], other):
            assert np.abs(a - c).max() <= 100 * U32 * max(1.0, np.abs(a).max()) * 4


def test_weights_at_any_place_and_of_either_type():
    """W and bias as slices that start inside 16 bytes give what aligned copies give."""
    import torch
    from frame_wise_linear_b200 import vda
    for D in (128, 1000, 77):
        for w in ("f32", "bf16"):
            X = torch.randn(50, D, device="cuda").to(torch.bfloat16)
            full = torch.randn(2 * D + 9, device="cuda").to(dtype_of(w))
            W, b = full[1: 1 + D], full[D + 4: 2 * D + 4]
            p = vda.make_norm_problem(50, D, vda.VDA_DTYPE_BF16, w_dtype=code_of(w), eps=EPS)
            Y, Z = torch.empty_like(X), torch.empty_like(X)
            vda.vda_layer_norm(p, X, W, b, Y)
            vda.vda_layer_norm(p, X, W.clone(), b.clone(), Z)
            assert torch.equal(Y, Z)


@pytest.mark.parametrize("heads,D", [(1, 128), (7, 72), (3, 33), (65536, 1)])
def test_heads_of_strided_tokens(heads, D):
    """The quotient row / heads by multiplication, and rows of the last token, against a dense copy."""
    import torch
    from frame_wise_linear_b200 import vda
    n, width = (3, heads * D) if heads > 1000 else (501, heads * D)
    full = torch.randn(n, width + 24, device="cuda")
    X = full[:, 8: 8 + width]
    W = torch.randn(D, device="cuda")
    strided = vda.make_norm_problem(n, D, vda.VDA_DTYPE_F32, heads=heads, eps=EPS, ld_x=width + 24)
    dense = vda.make_norm_problem(n, D, vda.VDA_DTYPE_F32, heads=heads, eps=EPS)
    Y, Z = torch.empty(n, width, device="cuda"), torch.empty(n, width, device="cuda")
    s1, s2 = torch.empty(2, n * heads, device="cuda"), torch.empty(2, n * heads, device="cuda")
    vda.vda_layer_norm(strided, X, W, None, Y, *s1)
    vda.vda_layer_norm(dense, X.contiguous(), W, None, Z, *s2)
    assert float((Y - Z).abs().max()) <= 200 * U32 * float(Z.abs().max())
    assert torch.allclose(s1, s2, rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("rows,D,dtype", [(1, 1, "bf16"), (300, 1, "f32"), (1000, 33, "bf16"), (257, 95, "f32"),
                                          (9, 8191, "bf16"), (3, 100003, "f32"), (70, 4090, "bf16")])
@pytest.mark.parametrize("off", [0, 1, 7])
def test_checkpoints_of_odd_rows_among_other_values(rows, D, dtype, off):
    """Stretches of blocks that begin and end anywhere: codes bit for bit, nothing else written."""
    import torch
    from frame_wise_linear_b200 import vda
    rng = np.random.default_rng(rows + D + off)
    X, _ = inside(rows, D, D, dtype_of(dtype), float("inf"), off)
    _fill(X, rng)
    X.mul_(torch.exp2(torch.randint(-20, 20, (rows, 1), device="cuda")).to(X.dtype))
    nblk = -(-D // 32)
    cfull = torch.full((off + rows * D + 64,), 9, dtype=torch.uint8, device="cuda")
    sfull = torch.full((off + rows * nblk + 64,), 9, dtype=torch.uint8, device="cuda")
    codes, scales = cfull[off: off + rows * D].view(rows, D), sfull[off: off + rows * nblk].view(rows, nblk)
    p = vda.make_checkpoint_problem(rows, D, code_of(dtype))
    vda.vda_checkpoint_pack(p, X, codes, scales)
    c, s = o.checkpoint(f64(X))
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s)
    Y, full = inside(rows, D, D, X.dtype, 7.0, off)
    vda.vda_checkpoint_unpack(p, codes, scales, Y)
    assert np.array_equal(f64(Y), o.checkpoint_values(c, s))
    assert untouched(full, Y, 7.0)
    assert untouched(cfull, codes, 9) and untouched(sfull, scales, 9)


@pytest.mark.parametrize("H_q,H_k", [(65535, 0), (1, 65534), (37, 5)])
def test_rope_many_heads(H_q, H_k):
    import torch
    from frame_wise_linear_b200 import vda
    d, axes = 8, (2, 2, 4)
    q, k = (torch.randn(1, 2, H, d, device="cuda") if H else None for H in (H_q, H_k))
    p = vda.make_rope_problem(1, 1, 1, 2, H_q, H_k, d, axes, vda.VDA_DTYPE_F32, layout=1)
    for x, H in ((q, H_q), (k, H_k)):
        if H:
            ref = o.rope(f64(x)[0], o.rope_grid(1, 1, 2), axes)
            y = torch.empty_like(x)
            one = vda.make_rope_problem(1, 1, 1, 2, H, 0, d, axes, vda.VDA_DTYPE_F32, layout=1)
            vda.vda_rope(one, x, None, None, y, None)
            assert np.abs(f64(y)[0] - ref).max() <= 16 * U32 * np.abs(f64(x)).max()
    a, b = (torch.empty_like(x) if x is not None else None for x in (q, k))
    vda.vda_rope(p, q, k, None, a, b)
    for x, y in ((q, a), (k, b)):
        if x is not None:
            ref = o.rope(f64(x)[0], o.rope_grid(1, 1, 2), axes)
            assert np.abs(f64(y)[0] - ref).max() <= 16 * U32 * np.abs(f64(x)).max()


def test_calls_on_a_side_stream_follow_it():
    """Work enqueued behind a slow producer on the same stream sees its result."""
    import torch
    from frame_wise_linear_b200 import vda
    s = torch.cuda.Stream()
    n, D = 2000, 1024
    p = vda.make_norm_problem(n, D, vda.VDA_DTYPE_F32, eps=EPS)
    src = torch.randn(n, D, device="cuda")
    X, Y, Z = torch.zeros(n, D, device="cuda"), torch.empty(n, D, device="cuda"), torch.empty(n, D, device="cuda")
    big = torch.randn(4096, 4096, device="cuda")
    vda.vda_layer_norm(p, src, None, None, Z)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(10):
            big = big @ big * 1e-4
        X.copy_(src)
        vda.vda_layer_norm(p, X, None, None, Y)             # the current stream
    s.synchronize()
    assert torch.equal(Y, Z)
    Y.zero_()
    torch.cuda.synchronize()
    vda.vda_layer_norm(p, src, None, None, Y, stream=s)     # a stream given
    s.synchronize()
    assert torch.equal(Y, Z)


@pytest.mark.parametrize("D", [33, 77, 1001])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_kept_rows_of_odd_widths(D, dtype):
    """The checkpoint of an odd-width norm is that of (x - mean) rstd with the statistics the call returns, whether
    the call writes over X, keeps its statistics, or neither: bit for bit."""
    import torch
    from frame_wise_linear_b200 import vda
    n, dt = 413, dtype_of(dtype)
    X = (torch.randn(n, D, device="cuda") + 0.5).to(dt)
    W, b = torch.randn(2, D, device="cuda")
    p = vda.make_norm_problem(n, D, code_of(dtype), eps=EPS)
    nblk = -(-D // 32)

    def run(x, y, stats):
        codes = torch.full((n, D), 9, dtype=torch.uint8, device="cuda")
        scales = torch.full((n, nblk), 9, dtype=torch.uint8, device="cuda")
        vda.vda_layer_norm(p, x, W, b, y, *stats, codes, scales)
        return codes, scales

    mean, rstd = torch.empty(2, n, device="cuda")
    Y = torch.empty_like(X)
    codes, scales = run(X, Y, (mean, rstd))
    xh = (X.float() - mean[:, None]) * rstd[:, None]
    c, s = o.checkpoint(f64(xh))
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s)
    # Other forms of the kernel sum in another order: their statistics, and with them a value at a border between
    # two codes, may differ in the last place, and then be one code step off.  With scale 2^e the codes from 2^-6 2^e
    # up have four significant bits, so neighbours differ by 2^-3 of the smaller at most; below they are the multiples
    # of 2^-9 2^e, so neighbours differ by that, which is more than 2^-3 of a value under 2^-6 2^e.
    e = np.repeat(s.astype(float) - 127, 32, axis=1)[:, :D]
    for over, stats in ((True, (torch.empty(n, device="cuda"), torch.empty(n, device="cuda"))), (False, (None, None))):
        x = X.clone()
        y = x if over else torch.empty_like(X)
        codes2, scales2 = run(x, y, stats)
        v, ref = o.checkpoint_values(codes2.cpu().numpy(), scales2.cpu().numpy()), o.checkpoint_values(c, s)
        differ = v != ref
        assert differ.mean() <= 1e-3
        step = np.maximum(2.0 ** -3 * np.abs(f64(xh)) * (1 + 2.0 ** -4), 2.0 ** (e - 9))
        assert np.all(np.abs(v - ref)[differ] <= step[differ])
