"""Every form of the layer norm's kernels against the oracle: all rows, several batches of rows, ragged ends.

A form is a pass, a type, vectors or single elements, the elements of a thread, whether every thread has all of them,
and the rows of a batch.  tests/norm_forms.py replays the choice; test_cases_take_every_form (on the CPU) holds the
cases below to the whole list, with more than one batch a CTA wherever a batch has several rows.

Rows differ in mean and size, so that a row that is given another's statistics is far off.

Bounds, with u = 2^-24 half a step of float32.
Mean: a thread's 32 or fewer elements go to two accumulators (two pairs: 8 additions each, and 2 to join them; single
elements: 16 and 1), 5 additions across lanes, the reciprocal and its product, the weight of a warp (2) and its product,
4 additions across warps: 17 + 5 + 2 + 3 + 4 = 31 at most, so |mean - m| <= 32 u max|x|.
Variance: a square 2 u of itself (the difference is rounded once), 17 + 5 + 4 additions, the weights and 1 / D 4: 32 u.
The means that join it are off by at most 32 u X, X = max|x| + |m|: that enters as 2 (m_i - m) 32 u X summed, at most
64 u X R relative, and as its square.  The root halves it; the sum with eps, the root and the division add 3 u.
Y and codes, from the mean and rstd that the call returned: xh = (x - mean) rstd is two float32 roundings, which torch
repeats bit for bit, so the codes are exactly the oracle's for that xh; y is one multiply-add and one rounding.
Gradients, from mean and rstd as given: xh 2 u.  A row's sums of g and g xh: a thread's 16 or fewer pairs are
multiply-adds, 1 to join the pair, 5 + 4 additions: 26, and 2 for the mean; g xh also one product: 29.  Then three more
roundings of each term.  dW: a column's term passes its product (1), xh (2), the rows that its thread adds, the groups
of its CTA, and ten partial sums and five shuffles of the last sum: rows + groups + 18.  db: the same without xh.
"""
import numpy as np
import pytest

import norm_forms
from oracle import token_oracle as o
from token_testutil import U32, assert_close, code_of, dtype_of, f64, half_step, inside, untouched

EPS = 1e-5
FILL = 7.0

# tokens, heads, width, type, elements between tokens, place behind a 16-byte boundary
CASES = [
    # bf16: vectors
    (77000, 1, 32, "bf16", 0, 0), (90, 1, 32, "bf16", 0, 0),            # 8 elements a thread
    (77001, 1, 24, "bf16", 0, 0), (90, 1, 8, "bf16", 0, 0),
    (2501, 1, 4096, "bf16", 0, 0), (300, 1, 4096, "bf16", 0, 0),        # 16
    (2501, 1, 4000, "bf16", 0, 0), (130, 1, 1000, "bf16", 0, 0),
    (5100, 8, 128, "bf16", 16, 0),                                     # heads of strided tokens
    (761, 1, 8192, "bf16", 0, 0), (90, 1, 8192, "bf16", 0, 0),          # 32
    (761, 1, 5000, "bf16", 0, 0), (90, 1, 8184, "bf16", 0, 0),
    # bf16: rows that start inside vectors
    (9501, 1, 1001, "bf16", 0, 0), (300, 1, 1001, "bf16", 0, 3),
    (9500, 1, 1002, "bf16", 0, 1),
    (901, 1, 4097, "bf16", 0, 0), (90, 1, 7001, "bf16", 0, 5),
    # bf16: single elements
    (700, 1, 77, "bf16", 3, 1), (650, 1, 1001, "bf16", 1, 0), (400, 1, 4099, "bf16", 1, 0),
    # float32: vectors
    (20001, 1, 64, "f32", 0, 0), (90, 1, 64, "f32", 0, 0),              # 8
    (20001, 1, 60, "f32", 0, 0), (90, 1, 4, "f32", 0, 0),
    (1201, 1, 2048, "f32", 0, 0), (900, 1, 1000, "f32", 0, 0),          # 16
    (450, 1, 8192, "f32", 0, 0), (450, 1, 5000, "f32", 0, 0),           # 32
    # float32: rows that start inside vectors
    (40001, 1, 33, "f32", 0, 0), (90, 1, 33, "f32", 0, 1),
    (5001, 1, 1001, "f32", 0, 0), (500, 1, 4099, "f32", 0, 2),
    # float32: single elements
    (700, 1, 77, "f32", 1, 1), (650, 1, 1001, "f32", 3, 0), (300, 1, 4099, "f32", 1, 0),
]


def _forms(tokens, heads, D, dtype, pad, place):
    return {s: norm_forms.form(s, tokens, heads, D, {"bf16": 2, "f32": 4}[dtype], pad, place, place)
            for s in norm_forms.PASSES}


def test_cases_take_every_form():
    """The forms of any call, found by walking over widths, rows, strides and places, are the cases' forms."""
    key = lambda f: (f.step, f.bytes, f.ve, f.per, f.fill, f.rows)  # noqa: E731
    widths = [*range(1, 140), 255, 256, 257, 1000, 1001, 2048, 4088, 4092, *range(4094, 4106), 5000, 8180, 8184, 8188,
              *range(8189, 8193)]
    any_call = set()
    for element in (2, 4):
        for D in widths:
            for pad, place in ((0, 0), (0, 1), (0, 2), (1, 0), (8, 0)):
                for rows in (1, 3, 8, 300, 1200, 5000, 20000, 100000):
                    for s in norm_forms.PASSES:
                        any_call.add(key(norm_forms.form(s, rows, 1, D, element, pad, place, place)))
    taken = [f for c in CASES for f in _forms(*c).values()]
    assert {key(f) for f in taken} == any_call
    several = {key(f) for f in taken if f.rows > 1 and f.batches > 1}
    assert several == {k for k in any_call if k[-1] > 1}


def _draw(tokens, heads, D, dtype, ld, place, seed):
    """Rows with means within 3 and sizes from 1/4 to 4, among other values."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, _ = inside(tokens, heads * D, ld, dtype_of(dtype), float("nan"), place)
    shape = (tokens * heads, D)
    size = torch.exp2(4 * torch.rand(shape[0], 1, device="cuda", generator=g) - 2)
    mean = 6 * torch.rand(shape[0], 1, device="cuda", generator=g) - 3
    x.copy_((torch.randn(shape, device="cuda", generator=g) * size + mean).view(tokens, heads * D))
    return x


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,heads,D,dtype,pad,place", CASES)
def test_form(tokens, heads, D, dtype, pad, place):
    import torch
    from frame_wise_linear_b200 import vda
    forms = _forms(tokens, heads, D, dtype, pad, place)
    dt, width, rows, nblk = dtype_of(dtype), heads * D, tokens * heads, -(-D // 32)
    ld, half = width + pad, half_step(dt)
    X, dY = (_draw(tokens, heads, D, dtype, ld, place, seed) for seed in (D, D + 1))
    flat = lambda t: t.reshape(rows, D)  # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(1)
    W, b = (torch.randn(D, device="cuda", generator=g) * 0.3 + m for m in (1.0, 0.0))
    w, bn, x, dy = f64(W), f64(b), f64(flat(X)), f64(flat(dY))
    p = vda.make_norm_problem(tokens, D, code_of(dtype), heads=heads, eps=EPS, ld_x=ld if pad else 0,
                              ld_y=ld if pad else 0)

    def bytes_at(n, m, fill):
        full = torch.full((place + n * m + 64,), fill, dtype=torch.uint8, device="cuda")
        return full, full[place: place + n * m].view(n, m)

    # The forward, without and with codes.
    _, m_ref, r_ref, _ = o.layer_norm(x, eps=EPS)
    X_ = np.abs(x).max(1) + np.abs(m_ref)
    XR = U32 * X_ * r_ref
    for keep in (False, True):
        Y, full = inside(tokens, width, ld, dt, FILL, place)
        mean, rstd = torch.full((2, rows), FILL, device="cuda")
        cfull, codes = bytes_at(rows, D, 9)
        sfull, scales = bytes_at(rows, nblk, 9)
        vda.vda_layer_norm(p, X, W, b, Y, mean, rstd, codes if keep else None, scales if keep else None)
        assert_close(f64(mean), m_ref, 32 * U32 * np.abs(x).max(1), "mean")
        assert_close(f64(rstd), r_ref, r_ref * ((32 * U32 + 64 * XR + (32 * XR) ** 2) / 2 + 3 * U32) * (1 + 1e-3), "rstd")
        xh = (flat(X).float() - mean[:, None]) * rstd[:, None]
        ref = f64(xh) * w + bn
        assert_close(f64(flat(Y)), ref, U32 * np.abs(ref) + half * np.abs(ref) * (1 + U32), "Y")
        assert untouched(full, Y, FILL)
        if keep:
            c, s = o.checkpoint(f64(xh))
            assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s)
            v = o.checkpoint_values(c, s)
            Y, full = inside(tokens, width, ld, dt, FILL, place)
            vda.vda_layer_norm_from_checkpoint(p, codes, scales, W, b, Y)
            ref = v * w + bn
            assert_close(f64(flat(Y)), ref, U32 * np.abs(ref) + half * np.abs(ref) * (1 + U32), "Y again")
            assert untouched(full, Y, FILL)
            assert untouched(cfull, codes.fill_(9), 9) and untouched(sfull, scales.fill_(9), 9)

    # The gradients, from X and from the codes.
    m, r = f64(mean), f64(rstd)
    codes.copy_(torch.from_numpy(c).cuda())
    scales.copy_(torch.from_numpy(s).cuda())
    ws = torch.full((vda.vda_layer_norm_backward_workspace_size(p),), 255, dtype=torch.uint8, device="cuda")   # NaN
    for step in ("bwd", "bwd_codes"):
        dX, full = inside(tokens, width, ld, dt, FILL, place)
        dW, db = torch.full((2, D), FILL, device="cuda")
        if step == "bwd":
            h = (x - m[:, None]) * r[:, None]
            vda.vda_layer_norm_backward(p, dY, X, mean, rstd, W, dX, dW, db, ws)
        else:
            h = v
            vda.vda_layer_norm_backward_from_checkpoint(p, dY, codes, scales, rstd, W, dX, dW, db, ws)
        dx_ref, dw_ref, db_ref = o.layer_norm_backward(dy, h, r, w)
        ga, ha = np.abs(dy * w), np.abs(h)
        gm, gx = ga.mean(1, keepdims=True), (ga * ha).mean(1, keepdims=True)
        err = r[:, None] * U32 * (3 * ga + 32 * gm + (29 + 2 + 4 + 2) * ha * gx) * (1 + 1e-5)
        assert_close(f64(flat(dX)), dx_ref, err + half * (np.abs(dx_ref) + err), "dX")
        assert untouched(full, dX, FILL)
        n = forms[step].thread_rows + forms[step].groups + 18
        assert_close(f64(dW), dw_ref, n * U32 * np.abs(dy * h).sum(0) * (1 + 1e-3), "dW")
        assert_close(f64(db), db_ref, n * U32 * np.abs(dy).sum(0) * (1 + 1e-3), "db")
