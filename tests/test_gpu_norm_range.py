"""Layer norm near float32's end: rows of one large value, at widths that leave threads or parts of vectors empty.

Where a thread has no element of a row it holds zeros, and nothing that it computes from them may reach the row: at
these magnitudes (0 - mean) rstd overflows, and a product of it with 0 is NaN.
"""
import numpy as np
import pytest

from oracle import token_oracle as o
from token_testutil import U32, assert_close, code_of, dtype_of, f64, half_step, inside

pytestmark = pytest.mark.gpu

EPS = 1e-6
BIG = 2.0 ** 119          # BIG / sqrt(EPS) is 2^129, beyond float32

# Width, type, heads, elements between tokens beyond them: vectors that some threads lack, shifted vectors, single
# elements.
WIDTHS = [(8, "bf16", 1, 0), (24, "bf16", 1, 0), (1000, "bf16", 1, 0), (4, "f32", 1, 0), (1004, "f32", 1, 0),
          (33, "bf16", 1, 0), (1001, "bf16", 1, 0), (1001, "f32", 1, 0), (7, "bf16", 1, 0), (7, "f32", 3, 0),
          (77, "bf16", 2, 3), (1001, "f32", 1, 1), (8, "bf16", 5, 8)]


@pytest.mark.parametrize("D,dtype,heads,pad", WIDTHS)
@pytest.mark.parametrize("tokens", [3, 4000])
def test_gradients_of_large_constant_rows(D, dtype, heads, pad, tokens):
    """x = mean exactly, so xh = 0: dX = rstd (g - mean(g)), dW = 0.

    The sums of g xh are sums of zeros, and the bound is that of test_gpu_norm.py with |xh| = 0 and no error in it:
    g one rounding, its mean at most 45 roundings of the mean of |g| and the division's, the difference and the
    product one each.  db: 3 roundings a batch of rows would be few; every column's term passes at most `rows`
    additions, which is what is allowed.
    """
    import torch
    from frame_wise_linear_b200 import vda
    rng = np.random.default_rng(D + heads)
    dt, width = dtype_of(dtype), heads * D
    ld, rows = width + pad, tokens * heads
    X, _ = inside(tokens, width, ld, dt, 0.0)
    sign = rng.choice([-1.0, 1.0], (tokens, heads, 1))
    X.copy_(torch.from_numpy(np.broadcast_to(BIG * sign, (tokens, heads, D)).reshape(tokens, width).copy()).cuda())
    dY, _ = inside(tokens, width, ld, dt, 0.0)
    dY.copy_(torch.from_numpy(rng.normal(size=(tokens, width))).cuda())
    W = torch.from_numpy(rng.normal(1.0, 0.3, D)).float().cuda()
    mean = X.as_strided((tokens, heads), (ld, D)).float().reshape(rows).contiguous()
    rstd = torch.full((rows,), EPS ** -0.5, device="cuda")
    p = vda.make_norm_problem(tokens, D, code_of(dtype), heads=heads, eps=EPS, ld_x=ld if pad else 0,
                              ld_y=ld if pad else 0)
    dX, _ = inside(tokens, width, ld, dt, 7.0)
    dW, db = torch.full((2, D), 7.0, device="cuda")
    ws = torch.full((vda.vda_layer_norm_backward_workspace_size(p),), 255, dtype=torch.uint8, device="cuda")
    vda.vda_layer_norm_backward(p, dY, X, mean, rstd, W, dX, dW, db, ws)
    dy, w, r = f64(dY).reshape(rows, D), f64(W), f64(rstd)
    ref, _, db_ref = o.layer_norm_backward(dy, np.zeros((rows, D)), r, w)
    g = np.abs(dy * w)
    err = r[:, None] * U32 * (6 * g + 50 * g.mean(1, keepdims=True))
    assert_close(f64(dX).reshape(rows, D), ref, err + half_step(dt) * (np.abs(ref) + err), "dX")
    assert bool((dW == 0).all())
    assert_close(f64(db), db_ref, rows * U32 * np.abs(dy).sum(0), "db")


@pytest.mark.parametrize("D,dtype", [(8, "bf16"), (16, "bf16"), (32, "bf16"), (4, "f32"), (16, "f32")])
def test_forward_and_backward_of_large_constant_rows(D, dtype):
    """A power of two of elements: the mean of a constant row is exact, y is the bias, and the gradients are finite."""
    import torch
    from frame_wise_linear_b200 import vda
    n = 5
    X = torch.full((n, D), BIG, device="cuda").to(dtype_of(dtype))
    W, b = torch.full((D,), 2.0, device="cuda"), torch.arange(D, device="cuda").float()
    p = vda.make_norm_problem(n, D, code_of(dtype), eps=EPS)
    Y, (mean, rstd) = torch.empty_like(X), torch.empty(2, n, device="cuda")
    vda.vda_layer_norm(p, X, W, b, Y, mean, rstd)
    assert bool((mean == BIG).all()) and bool((Y == b.to(Y.dtype)).all())
    dX, (dW, db) = torch.empty_like(X), torch.empty(2, D, device="cuda")
    ws = torch.empty(vda.vda_layer_norm_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
    vda.vda_layer_norm_backward(p, torch.ones_like(X), X, mean, rstd, W, dX, dW, db, ws)
    assert bool((dX == 0).all()) and bool((dW == 0).all()) and bool((db == n).all())


@pytest.mark.parametrize("D,dtype", [(8192, "bf16"), (8192, "f32"), (4096, "bf16"), (1001, "f32"), (77, "bf16")])
def test_range_of_rows(D, dtype):
    """Elements of 10^17 are normalised at any width; where the squares pass float32 r is 0 and Y the bias, and where
    the sum does the row is NaN.  The sizes are powers of two: within the range Y is off by the statistics' bound of
    test_gpu_norm_forms.py with X R <= 2 sqrt(2), one multiply-add and the rounding to its type."""
    import torch
    from frame_wise_linear_b200 import vda
    dt = dtype_of(dtype)
    rng = np.random.default_rng(D)
    sign = np.where(rng.permutation(D) % 2, 1.0, -1.0)
    x = np.stack([sign * 2.0 ** 56, sign * 2.0 ** 90, np.full(D, 2.0 ** 127)])      # 2^56 = 0.72e17
    X = torch.from_numpy(x).to(dt).cuda()
    b = torch.full((D,), 0.5, device="cuda")
    p = vda.make_norm_problem(3, D, code_of(dtype), eps=EPS)
    Y, (mean, rstd) = torch.empty_like(X), torch.empty(2, 3, device="cuda")
    vda.vda_layer_norm(p, X, None, b, Y, mean, rstd)
    ref = o.layer_norm(x[:1], None, f64(b), EPS)[0]
    err = U32 * (32 * 3 + 2 * (16 + 96 + 3)) + 2 * U32
    assert_close(f64(Y[:1]), ref, err * 1.01 + half_step(dt) * (np.abs(ref) + err))
    assert float(rstd[1]) == 0 and bool((Y[1] == 0.5).all())
    assert bool(torch.isnan(Y[2]).all())


@pytest.mark.parametrize("D,dtype,place", [(4096, "bf16", 0), (1001, "bf16", 3), (1001, "f32", 1), (72, "bf16", 0)])
def test_equal_bits_at_equal_places(D, dtype, place):
    """Buffers elsewhere, but at the same place within 16 bytes, give the same bits, whatever else runs."""
    import torch
    from frame_wise_linear_b200 import vda
    n, dt = 3001, dtype_of(dtype)
    g = torch.Generator(device="cuda").manual_seed(D)
    x, dy = (torch.randn(n, D, device="cuda", generator=g).to(dt) for _ in range(2))
    W = torch.rand(D, device="cuda", generator=g)
    p = vda.make_norm_problem(n, D, code_of(dtype), eps=EPS)
    ws = torch.empty(vda.vda_layer_norm_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
    side, big, want = torch.cuda.Stream(), torch.randn(2048, 2048, device="cuda"), None
    for i in range(6):
        at = place + i * (16 // x.element_size())
        X, dY, dX = (inside(n, D, D, dt, 0.0, at)[0] for _ in range(3))
        X.copy_(x)
        dY.copy_(dy)
        mean, rstd = torch.empty(2, n, device="cuda")
        dW, db = torch.empty(2, D, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(i):
                big @ big
        vda.vda_layer_norm(p, X, W, None, dX, mean, rstd)
        y = dX.clone()
        vda.vda_layer_norm_backward(p, dY, X, mean, rstd, W, dX, dW, db, ws)
        got = [y, mean, rstd, dX, dW, db]
        want = want or [t.clone() for t in got]
        assert all(torch.equal(a, c) for a, c in zip(got, want)), i
