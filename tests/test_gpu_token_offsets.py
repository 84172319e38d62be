"""The token operators on tensors of more than 2^32 elements: rows around 2^31 and 2^32 elements, the first and the last,
and the weight gradients over all rows.  Bounds as in test_gpu_norm_forms.py and test_gpu_rope.py."""
import numpy as np
import pytest

import norm_forms
from oracle import token_oracle as o
from token_testutil import U32, assert_close, f64, half_step

pytestmark = [pytest.mark.gpu, pytest.mark.slow]

EPS = 1e-5
HALF = 2.0 ** -8      # half a step of bf16


def _windows(rows, stride):
    """Rows whose elements are worth a look, `stride` elements from one to the next."""
    at = [0, 1, rows - 2, rows - 1]
    for edge in (1 << 31, 1 << 32):
        at += [edge // stride + k for k in (-1, 0, 1)]
    return sorted({r for r in at if 0 <= r < rows})


def _uniform(shape, lo, hi, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").uniform_(lo, hi, generator=g)


def _check_dx(got, dy, h, r, w):
    ref, _, _ = o.layer_norm_backward(dy, h, r, w)
    ga, ha = np.abs(dy * w), np.abs(h)
    gx = (ga * ha).mean(1, keepdims=True)
    err = r[:, None] * U32 * (3 * ga + 32 * ga.mean(1, keepdims=True) + 37 * ha * gx) * (1 + 1e-5)
    assert_close(got, ref, err + HALF * (np.abs(ref) + err), "dX")


# 4096: vectors, two rows a batch; 1001: rows that start inside vectors.
@pytest.mark.parametrize("D,rows", [(4096, (1 << 20) + 5), (1001, (1 << 32) // 1001 + 4099)])
def test_layer_norm(D, rows):
    """dY has a mean of 1/4 and does not follow X: neither gradient is near 0, nor are its sums."""
    import torch
    from frame_wise_linear_b200 import vda
    assert rows * D > 1 << 32
    X, dY = _uniform((rows, D), -1, 1, 1), _uniform((rows, D), -0.5, 1, 2)
    W, b = (torch.rand(D, device="cuda") + k for k in (0.5, 0.0))
    w = f64(W)
    at = _windows(rows, D)
    x, dy = f64(X[at]), f64(dY[at])
    p = vda.make_norm_problem(rows, D, vda.VDA_DTYPE_BF16, eps=EPS)
    Y, (mean, rstd) = torch.empty_like(X), torch.empty(2, rows, device="cuda")
    codes = torch.empty(rows, D, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, -(-D // 32), dtype=torch.uint8, device="cuda")
    vda.vda_layer_norm(p, X, W, b, Y, mean, rstd, codes, scales)
    _, m_ref, r_ref, _ = o.layer_norm(x, eps=EPS)
    m, r = f64(mean[at]), f64(rstd[at])
    XR = U32 * (np.abs(x).max(1) + np.abs(m_ref)) * r_ref
    assert_close(m, m_ref, 32 * U32 * np.abs(x).max(1), "mean")
    assert_close(r, r_ref, r_ref * ((32 * U32 + 64 * XR + (32 * XR) ** 2) / 2 + 3 * U32) * (1 + 1e-3), "rstd")
    xh = (X[at].float() - mean[at][:, None]) * rstd[at][:, None]
    ref = f64(xh) * w + f64(b)
    assert_close(f64(Y[at]), ref, U32 * np.abs(ref) + HALF * np.abs(ref) * (1 + U32), "Y")
    c, s = o.checkpoint(f64(xh))
    assert np.array_equal(codes[at].cpu().numpy(), c) and np.array_equal(scales[at].cpu().numpy(), s)
    v = o.checkpoint_values(c, s)
    Y.fill_(7.0)
    vda.vda_layer_norm_from_checkpoint(p, codes, scales, W, b, Y)
    ref = v * w + f64(b)
    assert_close(f64(Y[at]), ref, U32 * np.abs(ref) + HALF * np.abs(ref) * (1 + U32), "Y again")
    del Y

    ws = torch.empty(vda.vda_layer_norm_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
    dX, (dW, db) = torch.empty_like(X), torch.empty(2, D, device="cuda")
    for step in ("bwd", "bwd_codes"):
        dX.fill_(7.0)
        if step == "bwd":
            vda.vda_layer_norm_backward(p, dY, X, mean, rstd, W, dX, dW, db, ws)
        else:
            vda.vda_layer_norm_backward_from_checkpoint(p, dY, codes, scales, rstd, W, dX, dW, db, ws)
        _check_dx(f64(dX[at]), dy, (x - m[:, None]) * r[:, None] if step == "bwd" else v, r, w)
        if step == "bwd":
            sums = torch.zeros(4, D, dtype=torch.float64, device="cuda")
            for i in range(0, rows, 1 << 16):
                part = slice(i, i + (1 << 16))
                h = (X[part].double() - mean[part, None].double()) * rstd[part, None].double()
                g = dY[part].double()
                t = g * h
                for k, q in enumerate((t, g, t.abs(), g.abs())):
                    sums[k] += q.sum(0)
            n = norm_forms.form("bwd", rows, 1, D, 2)
            u = (n.thread_rows + n.groups + 18) * U32 * (1 + 1e-2)
            dw_ref, db_ref, dw_abs, db_abs = (f64(q) for q in sums)
            assert np.median(np.abs(dw_ref)) > 0 and np.abs(db_ref).min() > 0.2 * rows
            assert_close(f64(dW), dw_ref, u * dw_abs, "dW")
        assert_close(f64(db), db_ref, u * db_abs, "db")    # the same sum from either


def test_layer_norm_of_distant_tokens():
    """Single elements: odd rows 2^20 + 1 elements apart."""
    import torch
    from frame_wise_linear_b200 import vda
    D, ld, rows = 77, (1 << 20) + 1, 4200
    full, grads = _uniform(rows * ld, -1, 1, 1), torch.full((rows * ld,), 7.0, dtype=torch.bfloat16, device="cuda")
    X, dX = (t.as_strided((rows, D), (ld, 1)) for t in (full, grads))
    W = torch.rand(D, device="cuda") + 0.5
    dY = _uniform((rows, D), -0.5, 1, 2)
    p = vda.make_norm_problem(rows, D, vda.VDA_DTYPE_BF16, eps=EPS, ld_x=ld)
    Y, (mean, rstd) = torch.empty(rows, D, dtype=torch.bfloat16, device="cuda"), torch.empty(2, rows, device="cuda")
    vda.vda_layer_norm(p, X, W, None, Y, mean, rstd)
    xh = (X.float() - mean[:, None]) * rstd[:, None]
    ref = f64(xh) * f64(W)
    assert_close(f64(Y), ref, U32 * np.abs(ref) + HALF * np.abs(ref) * (1 + U32), "Y")
    _, m_ref, _, _ = o.layer_norm(f64(X), eps=EPS)
    assert_close(f64(mean), m_ref, 32 * U32 * np.abs(f64(X)).max(1), "mean")
    vda.vda_layer_norm_backward(p, dY, X, mean, rstd, W, dX, None, None, None)
    m, r = f64(mean), f64(rstd)
    _check_dx(f64(dX), f64(dY), (f64(X) - m[:, None]) * r[:, None], r, f64(W))
    dX.fill_(7.0)
    assert bool((grads == 7).all())


# 1001: dense rows through shared memory; 128 and 77 with a gap: vectors and single elements.
@pytest.mark.parametrize("rows,D,ld", [((1 << 32) // 1001 + 4099, 1001, 0), (4200, 128, 1 << 20),
                                       (4200, 77, (1 << 20) + 1)])
def test_checkpoints(rows, D, ld):
    import torch
    from frame_wise_linear_b200 import vda
    step = ld or D
    assert rows * step > 1 << 32
    full = _uniform(rows * step, -1, 1, 1)
    X = full.as_strided((rows, D), (step, 1))
    codes = torch.empty(rows, D, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, -(-D // 32), dtype=torch.uint8, device="cuda")
    p = vda.make_checkpoint_problem(rows, D, vda.VDA_DTYPE_BF16, ld=ld)
    vda.vda_checkpoint_pack(p, X, codes, scales)
    at = _windows(rows, step)
    c, s = o.checkpoint(f64(X[at]))
    assert np.array_equal(codes[at].cpu().numpy(), c) and np.array_equal(scales[at].cpu().numpy(), s)
    back = torch.full_like(full, 7.0)
    Z = back.as_strided((rows, D), (step, 1))
    vda.vda_checkpoint_unpack(p, codes, scales, Z)
    assert np.array_equal(f64(Z[at]), o.checkpoint_values(c, s))
    # every element within half a code step: 2^-4 of it, or 2^-10 of the block's 2^e with 448 2^e < 2 max|x| <= 2
    for i in range(0, rows, 1 << 16):
        x, z = X[i: i + (1 << 16)].float(), Z[i: i + (1 << 16)].float()
        assert bool(((x - z).abs() <= torch.clamp(x.abs() * 2.0 ** -4, min=2.0 ** -10 * 2 / 448)).all())
    if ld:
        Z.fill_(7.0)
        assert bool((back == 7).all())


@pytest.mark.parametrize("layout", [0, 1])
def test_rope_of_halves(layout):
    """Pairs half the width apart, the last heads and tokens of either layout, in place."""
    import torch
    from frame_wise_linear_b200 import vda
    T, h, w, H, d, axes = 130, 64, 129, 32, 128, (32, 48, 48)
    N = T * h * w
    assert N * H * d > 1 << 32
    q = _uniform((H, N, d) if layout == 0 else (N, H, d), -1, 1, 1)
    tokens = [0, 1, N // 2, N - 2, N - 1]
    heads = [0, 15, 16, 31]
    pick = lambda: f64(q[heads][:, tokens]).transpose(1, 0, 2) if layout == 0 else f64(q[tokens][:, heads])  # noqa: E731
    x = pick()
    p = vda.make_rope_problem(1, T, h, w, H, 0, d, axes, vda.VDA_DTYPE_BF16, layout=layout, pairing=1)
    vda.vda_rope(p, q, None, None, q, None)
    ref = o.rope(x, o.rope_grid(T, h, w)[tokens], axes, halves=True)
    err = 16 * U32
    assert_close(pick(), ref, err + half_step(torch.bfloat16) * (np.abs(ref) + err))
