"""Layer norm, forward and backward, with and without 8-bit checkpoints, against the float64 oracle.

Bounds.  u = 2^-24 is half a step of float32.  A sum over a row adds at most
8 terms in a thread, 5 times across lanes and at most 32 warps: 45 roundings,
so |mean - m| <= 45 u max|x| and each difference x - mean is off by at most
47 u X with X = max|x| over the row + |mean|.  The variance gains the square
of that, and 47 u relative from its own sum; the root halves it, the division
and the root add 2 u.  With R = rstd this gives
    |rstd error| / R <= 30 u + (47 u X R)^2        (doubled below)
    |xh error|  <= 47 u X R + |xh| (32 u + ...)
and y is one multiply-add and one rounding to its type further.  The gradient
takes mean and rstd as given: |xh error| <= 3 u X R, g one rounding, the two
row means 47 u of the means of |g| and |g xh|.  Sums over rows: the number of
additions that a column's term passes through, times u, times the sum of the
magnitudes; at the sizes here at most 16 rows of a thread, 64 groups of a
CTA and 592 / 8 + 8 partial sums: 162, bounded by 192.
"""
import numpy as np
import pytest

from oracle import token_oracle as o
from token_testutil import U32, assert_close, code_of, dtype_of, f64, half_step, inside, untouched

pytestmark = pytest.mark.gpu

EPS = 1e-5
FILL = 7.0


def _make(tokens, heads, D, dtype, w="f32", affine=True, strided=False, offset=0, seed=0, shift=0.5):
    import torch
    rng = np.random.default_rng(seed + 1000 * tokens + D)
    width, dt = heads * D, dtype_of(dtype)
    ld = width + (16 if strided is True else strided)
    X, _ = inside(tokens, width, ld, dt, 0.0, offset)
    X.copy_(torch.from_numpy(rng.normal(shift, 1.0, (tokens, width))).cuda())
    dY, _ = inside(tokens, width, ld, dt, 0.0, offset)
    dY.copy_(torch.from_numpy(rng.normal(size=(tokens, width))).cuda())
    W = b = None
    if affine:
        W = torch.from_numpy(rng.normal(1.0, 0.3, D)).to(dtype_of(w)).cuda()
        b = torch.from_numpy(rng.normal(0.0, 0.3, D)).to(dtype_of(w)).cuda()
    from frame_wise_linear_b200 import vda
    p = vda.make_norm_problem(tokens, D, code_of(dtype), heads=heads, w_dtype=code_of(w), eps=EPS,
                              ld_x=ld if strided else 0, ld_y=ld if strided else 0)
    return p, X, dY, W, b, ld


def _rows(t, D):
    return f64(t).reshape(-1, D)


def _xh_bound(x, xh, rstd):
    """The bound on the forward's xh from the module's text."""
    XR = (np.abs(x).max(1) + np.abs(x.mean(1))) * rstd
    return (47 * U32 * XR)[:, None] + np.abs(xh) * (64 * U32 + 2 * (47 * U32 * XR[:, None]) ** 2)


CASES = [
    # tokens, heads, D, dtype, w, affine, strided, offset
    (1, 1, 4096, "bf16", "f32", True, False, 0),
    (3, 1, 1, "f32", "f32", True, False, 0),            # one feature: xh = 0
    (2, 1, 2, "bf16", "bf16", True, False, 0),
    (5, 1, 8, "bf16", "f32", True, False, 0),           # a quarter of a 32-element block
    (7, 1, 31, "f32", "f32", True, False, 0),
    (65, 1, 33, "bf16", "bf16", True, False, 0),
    (130, 1, 40, "bf16", "f32", True, False, 0),        # vectors, short last block
    (257, 4, 64, "f32", "f32", True, False, 0),
    (100, 3, 128, "bf16", "f32", True, True, 0),        # heads inside a wider token
    (100, 3, 128, "bf16", "f32", True, 5, 3),           # the same, nothing aligned
    (33, 1, 255, "bf16", "f32", True, False, 0),
    (33, 1, 256, "f32", "bf16", True, False, 0),
    (33, 1, 264, "bf16", "f32", True, False, 0),        # 33 vectors: two warps a row
    (50, 1, 520, "f32", "f32", True, True, 0),
    (50, 1, 776, "bf16", "f32", False, False, 0),       # three warps a row, no W and bias
    (700, 1, 1000, "bf16", "bf16", True, False, 0),
    (701, 1, 1001, "f32", "f32", True, False, 0),
    (2000, 1, 72, "bf16", "f32", True, False, 1),       # pointers off by one element
    (9, 1, 2049, "bf16", "f32", True, False, 0),
    (9, 1, 4104, "f32", "f32", True, False, 0),
    (5, 1, 8191, "bf16", "f32", True, False, 0),
    (5, 1, 8192, "bf16", "f32", True, False, 0),
    (5, 1, 8192, "f32", "f32", True, False, 0),
    (5, 1, 8188, "f32", "f32", True, False, 0),
]


@pytest.mark.parametrize("tokens,heads,D,dtype,w,affine,strided,offset", CASES)
@pytest.mark.parametrize("ckpt", [False, True])
def test_forward(tokens, heads, D, dtype, w, affine, strided, offset, ckpt):
    import torch
    from frame_wise_linear_b200 import vda
    p, X, _, W, b, ld = _make(tokens, heads, D, dtype, w, affine, strided, offset)
    rows = tokens * heads
    Y, full = inside(tokens, heads * D, ld, X.dtype, FILL, offset)
    mean, rstd = torch.full((2, rows), FILL, device="cuda")
    codes = torch.full((rows * D + 64,), 9, dtype=torch.uint8, device="cuda")
    nblk = -(-D // 32)
    scales = torch.full((rows * nblk + 64,), 9, dtype=torch.uint8, device="cuda")
    vda.vda_layer_norm(p, X, W, b, Y, mean, rstd, codes if ckpt else None, scales if ckpt else None)
    x = _rows(X, D)
    y_ref, m_ref, r_ref, xh = o.layer_norm(x, f64(W), f64(b), EPS)
    assert_close(f64(mean), m_ref, 47 * U32 * np.abs(x).max(1), "mean")
    XR = (np.abs(x).max(1) + np.abs(m_ref)) * r_ref
    assert_close(f64(rstd), r_ref, r_ref * (64 * U32 + 2 * (47 * U32 * XR) ** 2), "rstd")
    xb = _xh_bound(x, xh, r_ref)
    wa = np.abs(f64(W)) if affine else 1.0
    assert_close(_rows(Y, D), y_ref, xb * wa + 3 * U32 * (np.abs(xh) * wa + np.abs(y_ref)) +
                 half_step(Y.dtype) * np.abs(y_ref) * (1 + 2.0 ** -6), "Y")
    assert untouched(full, Y, FILL)
    if not ckpt:
        return
    assert bool((codes[rows * D:] == 9).all()) and bool((scales[rows * nblk:] == 9).all())
    c, s = codes[: rows * D].reshape(rows, D).cpu().numpy(), scales[: rows * nblk].reshape(rows, nblk).cpu().numpy()
    v = o.checkpoint_values(c, s)
    e = np.repeat(s.astype(float) - 127, 32, axis=1)[:, :D]
    assert_close(v, xh, np.maximum(2.0 ** -4 * (np.abs(xh) + xb), 2.0 ** (e - 10)) + xb, "checkpoint")
    # each scale is the least that covers its block, up to xh's own bound at the border
    for j in range(nblk):
        blk = slice(32 * j, 32 * j + 32)
        top, slack = np.abs(xh[:, blk]).max(1), xb[:, blk].max(1)
        cover = 448.0 * 2.0 ** (s[:, j].astype(float) - 127)
        assert np.all(top - slack <= cover) and np.all((top + slack > cover / 2) | (s[:, j] == 0))


@pytest.mark.parametrize("tokens,heads,D,dtype,w,affine,strided,offset", CASES)
@pytest.mark.parametrize("ckpt", [False, True])
def test_backward(tokens, heads, D, dtype, w, affine, strided, offset, ckpt):
    import torch
    from frame_wise_linear_b200 import vda
    p, X, dY, W, b, ld = _make(tokens, heads, D, dtype, w, affine, strided, offset)
    rows = tokens * heads
    x = _rows(X, D)
    _, m, r, xh = o.layer_norm(x, eps=EPS)
    mean, rstd = (torch.from_numpy(v).float().cuda() for v in (m, r))
    m, r = f64(mean), f64(rstd)
    dX, full = inside(tokens, heads * D, ld, X.dtype, FILL, offset)
    dW, db = torch.full((2, D), FILL, device="cuda")
    ws = torch.full((vda.vda_layer_norm_backward_workspace_size(p),), 255, dtype=torch.uint8, device="cuda")   # NaN
    if ckpt:
        c, s = o.checkpoint(xh.astype(np.float32))
        xh, xb = o.checkpoint_values(c, s), 0.0
        vda.vda_layer_norm_backward_from_checkpoint(p, dY, torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(),
                                                    rstd, W, dX, dW, db, ws)
    else:
        xh = (x - m[:, None]) * r[:, None]
        xb = 3 * U32 * ((np.abs(x).max(1) + np.abs(m)) * r)[:, None]
        vda.vda_layer_norm_backward(p, dY, X, mean, rstd, W, dX, dW, db, ws)
    dy, wa = _rows(dY, D), (f64(W) if affine else np.ones(D))
    dx_ref, dw_ref, db_ref = o.layer_norm_backward(dy, xh, r, wa)
    g = np.abs(dy * wa)
    gx = (g * (np.abs(xh) + xb)).mean(1, keepdims=True)
    err = r[:, None] * (U32 * (6 * g + 50 * g.mean(1, keepdims=True) + (50 * np.abs(xh) + 6) * gx) +
                        xb * gx + (np.abs(xh) + xb) * (g * xb).mean(1, keepdims=True))
    assert_close(_rows(dX, D), dx_ref, err + half_step(dX.dtype) * (np.abs(dx_ref) + err), "dX")
    assert untouched(full, dX, FILL)
    assert_close(f64(dW), dw_ref, 192 * U32 * np.abs(dy * xh).sum(0) + (np.abs(dy) * xb).sum(0), "dW")
    assert_close(f64(db), db_ref, 192 * U32 * np.abs(dy).sum(0), "db")


@pytest.mark.parametrize("tokens,heads,D,dtype,w,affine,strided,offset", CASES)
def test_forward_again_from_checkpoint(tokens, heads, D, dtype, w, affine, strided, offset):
    """y = xh w + b at the checkpoint's own values: one multiply-add, one rounding."""
    import torch
    from frame_wise_linear_b200 import vda
    p, X, _, W, b, ld = _make(tokens, heads, D, dtype, w, affine, strided, offset)
    c, s = o.checkpoint(o.layer_norm(_rows(X, D), eps=EPS)[3].astype(np.float32))
    Y, full = inside(tokens, heads * D, ld, X.dtype, FILL, offset)
    vda.vda_layer_norm_from_checkpoint(p, torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), W, b, Y)
    v = o.checkpoint_values(c, s)
    ref = v * (f64(W) if affine else 1.0) + (f64(b) if affine else 0.0)
    part = np.abs(v * (f64(W) if affine else 1.0))
    assert_close(_rows(Y, D), ref, 2 * U32 * (part + np.abs(ref)) + half_step(Y.dtype) * np.abs(ref) * (1 + 2.0 ** -6))
    assert untouched(full, Y, FILL)


@pytest.mark.parametrize("D", [24, 128, 1001])
def test_gradients_against_differences(D):
    """The float32 gradients along a direction against central differences of the float64 forward."""
    import torch
    from frame_wise_linear_b200 import vda
    p, X, dY, W, b, _ = _make(6, 1, D, "f32")
    mean, rstd = torch.empty(2, 6, device="cuda")
    Y, dX = torch.empty_like(X), torch.empty_like(X)
    dW, db = torch.empty(2, D, device="cuda")
    vda.vda_layer_norm(p, X, W, b, Y, mean, rstd)
    ws = torch.empty(vda.vda_layer_norm_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
    vda.vda_layer_norm_backward(p, dY, X, mean, rstd, W, dX, dW, db, ws)
    rng = np.random.default_rng(1)
    x, dy, wn, bn = f64(X), f64(dY), f64(W), f64(b)
    h = 1e-5
    for what, grad in (("x", dX), ("w", dW), ("b", db)):
        v = rng.normal(size=grad.shape)
        f = lambda t: (dy * o.layer_norm(x + t * v * (what == "x"), wn + t * v * (what == "w") if what != "x" else wn,  # noqa: E731
                                         bn + t * v if what == "b" else bn, EPS)[0]).sum()
        diff = (f(h) - f(-h)) / (2 * h)
        # differences: h^2 times third derivatives of order 1 per term; gradients: 200 u of the magnitudes
        bound = (h ** 2 * 10 + 200 * U32 * 50) * np.abs(v).sum()
        assert abs(diff - (f64(grad) * v).sum()) <= bound, what


def test_rows_do_not_mix():
    """A row with NaN or infinity is NaN, and no other row is; sums over rows become NaN where it counts."""
    import torch
    from frame_wise_linear_b200 import vda
    for D, dtype in ((128, "bf16"), (100, "f32"), (2048, "bf16")):
        p, X, dY, W, b, _ = _make(9, 1, D, dtype)
        X[2, 5], X[6, D - 1] = float("nan"), float("inf")
        Y, mean, rstd = torch.empty_like(X), *torch.empty(2, 9, device="cuda")
        codes = torch.empty(9, D, dtype=torch.uint8, device="cuda")
        scales = torch.empty(9, -(-D // 32), dtype=torch.uint8, device="cuda")
        vda.vda_layer_norm(p, X, W, b, Y, mean, rstd, codes, scales)
        bad = [2, 6]
        good = [i for i in range(9) if i not in bad]
        assert bool(torch.isnan(Y[bad]).all()) and bool(torch.isfinite(Y[good]).all())
        v = o.checkpoint_values(codes.cpu().numpy(), scales.cpu().numpy())
        assert np.all(np.isnan(v[bad])) and np.all(np.isfinite(v[good]))


def test_constant_rows_and_large_offsets():
    """Variance 0 gives xh = 0 (rstd = 1/sqrt(eps)); a mean of 1000 deviations keeps its digits (two sums)."""
    import torch
    from frame_wise_linear_b200 import vda
    D = 512
    p = vda.make_norm_problem(2, D, vda.VDA_DTYPE_F32, eps=EPS)
    rng = np.random.default_rng(2)
    x = np.stack([np.full(D, 3.25), 1000.0 + rng.normal(size=D)]).astype(np.float32)
    X = torch.from_numpy(x).cuda()
    Y, mean, rstd = torch.empty_like(X), *torch.empty(2, 2, device="cuda")
    vda.vda_layer_norm(p, X, None, None, Y, mean, rstd)
    assert bool((Y[0] == 0).all()) and abs(float(rstd[0]) * EPS ** 0.5 - 1) < 4 * U32
    y, _, r, xh = o.layer_norm(x, eps=EPS)
    assert_close(f64(Y)[1:], y[1:], _xh_bound(x.astype(np.float64), xh, r)[1:] + 3 * U32 * np.abs(y[1:]))


@pytest.mark.parametrize("D,dtype,strided", [(128, "bf16", False), (1000, "f32", True), (4096, "bf16", False),
                                             (77, "bf16", False)])
def test_in_place(D, dtype, strided):
    """Y over X; dX over X; dX over dY."""
    import torch
    from frame_wise_linear_b200 import vda
    n = 600
    p, X, dY, W, b, ld = _make(n, 1, D, dtype, strided=strided)
    Y, mean, rstd = torch.empty_strided(X.shape, X.stride(), dtype=X.dtype, device="cuda"), *torch.empty(2, n, device="cuda")
    vda.vda_layer_norm(p, X, W, b, Y, mean, rstd)
    X2, _ = inside(n, D, ld, X.dtype, 0.0)
    X2.copy_(X)
    vda.vda_layer_norm(p, X2, W, b, X2, None, None)
    assert torch.equal(X2, Y)
    ws = torch.empty(vda.vda_layer_norm_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
    dX, dW, db = torch.empty_strided(X.shape, X.stride(), dtype=X.dtype, device="cuda"), *torch.empty(2, D, device="cuda")
    vda.vda_layer_norm_backward(p, dY, X, mean, rstd, W, dX, dW, db, ws)
    for over in ("X", "dY"):
        a, c = inside(n, D, ld, X.dtype, 0.0)[0], inside(n, D, ld, X.dtype, 0.0)[0]
        a.copy_(X)
        c.copy_(dY)
        dW2, db2 = torch.empty(2, D, device="cuda")
        vda.vda_layer_norm_backward(p, c, a, mean, rstd, W, a if over == "X" else c, dW2, db2, ws)
        assert torch.equal(a if over == "X" else c, dX), over
        assert torch.equal(dW2, dW) and torch.equal(db2, db)


def test_optional_outputs_and_equal_bits():
    """Either weight gradient alone, neither (no workspace), and the same bits from equal calls."""
    import torch
    from frame_wise_linear_b200 import vda
    n, D = 3000, 384
    p, X, dY, W, b, _ = _make(n, 1, D, "bf16")
    mean, rstd, Y = *torch.empty(2, n, device="cuda"), torch.empty_like(X)
    vda.vda_layer_norm(p, X, W, b, Y, mean, rstd)
    ws = torch.empty(vda.vda_layer_norm_backward_workspace_size(p), dtype=torch.uint8, device="cuda")

    def run(dw, db, ws=ws):
        dX = torch.empty_like(X)
        out = [torch.full((D,), FILL, device="cuda") if k else None for k in (dw, db)]
        vda.vda_layer_norm_backward(p, dY, X, mean, rstd, W, dX, *out, ws, workspace_bytes=None if ws is not None else 0)
        return [dX] + out

    full = run(1, 1)
    for _ in range(5):
        assert all(torch.equal(a, c) for a, c in zip(full, run(1, 1)))
    assert torch.equal(run(1, 0)[1], full[1]) and torch.equal(run(0, 1)[2], full[2])
    assert torch.equal(run(0, 0, None)[0], full[0])
    Y2 = torch.empty_like(X)
    vda.vda_layer_norm(p, X, W, b, Y2)          # inference: no statistics
    assert torch.equal(Y2, Y)


def test_no_tokens_zero_the_weight_gradients():
    import torch
    from frame_wise_linear_b200 import vda
    p = vda.make_norm_problem(0, 96, vda.VDA_DTYPE_BF16)
    e = torch.empty(0, 96, dtype=torch.bfloat16, device="cuda")
    dW, db = torch.full((2, 96), FILL, device="cuda")
    vda.vda_layer_norm_backward(p, e, e, e, e, None, e, dW, db, None, workspace_bytes=0)
    assert bool((dW == 0).all()) and bool((db == 0).all())


@pytest.mark.slow
def test_offsets_past_32_bits():
    """More than 2^32 elements: the last rows are computed, and where they belong."""
    import torch
    from frame_wise_linear_b200 import vda
    D, n = 4096, (1 << 20) + 5
    X = torch.empty(n, D, dtype=torch.bfloat16, device="cuda")
    X.uniform_(-1, 1)
    p = vda.make_norm_problem(n, D, vda.VDA_DTYPE_BF16, eps=EPS)
    mean, rstd = torch.empty(2, n, device="cuda")
    Y = torch.empty_like(X)
    vda.vda_layer_norm(p, X, None, None, Y, mean, rstd)
    x = f64(X[-3:])
    y, m, r, xh = o.layer_norm(x, eps=EPS)
    assert_close(f64(Y[-3:]), y, _xh_bound(x, xh, r) + (half_step(Y.dtype) + 4 * U32) * np.abs(y) * (1 + 2.0 ** -6))
    ws = torch.empty(vda.vda_layer_norm_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
    dW, db = torch.empty(2, D, device="cuda")
    vda.vda_layer_norm_backward(p, Y, X, mean, rstd, None, Y, dW, db, ws)   # dX over dY
    dy = np.asarray(y)
    dx, _, _ = o.layer_norm_backward(f64(torch.from_numpy(dy).to(torch.bfloat16)), xh, r)
    # dY = y gives gradients near 0: bounded by the terms that cancel, in bf16 steps of y
    assert np.all(np.abs(f64(Y[-3:]) - dx) <= r[:, None] * (4 * 2.0 ** -8 * (1 + np.abs(xh))))
    assert bool(torch.isfinite(dW).all())
