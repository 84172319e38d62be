"""Rotary positions over three axes, forward and backward, against the float64 oracle.

Bounds.  The angle is a double product, reduced in double, and rounded to
float32 as a number of half turns in [-1, 1]: off by 2^-25 half turns, pi
2^-25 rad; the sine and cosine of it are off by at most 2 steps (2^-22 of 1 at
most), so c and s are each off by less than 2^-24 pi / 2 + 2^-22 < 6 u with
u = 2^-24.  Two products and a sum add 2 u of each term: an output is off by
at most 8 u (|a| + |b|), and by one rounding to its type.
"""
import numpy as np
import pytest

from oracle import token_oracle as o
from token_testutil import U32, assert_close, code_of, dtype_of, f64, half_step, inside, untouched

pytestmark = pytest.mark.gpu

FILL = 7.0


def _tensors(B, N, H, d, dt, layout, pad, offset, rng):
    """Input (drawn) and output (filled) of one of Q, K as flat views, with the output's buffer and the stride."""
    import torch
    if H == 0:
        return None, None, None, 0
    if layout == 0:
        x, _ = inside(B * H * N, d, d, dt, 0.0, offset)
        y, full = inside(B * H * N, d, d, dt, FILL, offset)
        ld = 0
    else:
        ld = H * d + pad
        x, _ = inside(B * N, H * d, ld, dt, 0.0, offset)
        y, full = inside(B * N, H * d, ld, dt, FILL, offset)
        ld = ld if pad else 0
    x.copy_(torch.from_numpy(rng.normal(size=tuple(x.shape))).cuda())
    return x, y, full, ld


def _as_tokens(t, B, N, H, d, layout):
    """[B, N, H, d] float64."""
    a = f64(t)
    return a.reshape(B, H, N, d).transpose(0, 2, 1, 3) if layout == 0 else a.reshape(B, N, H, d)


CASES = [
    # B, (T, h, w), Hq, Hk, d, axes, dtype, layout, halves, pad, offset
    (1, (1, 1, 1), 1, 1, 128, (44, 42, 42), "bf16", 1, False, 0, 0),        # one token
    (2, (3, 4, 5), 4, 2, 128, (44, 42, 42), "bf16", 1, False, 0, 0),
    (2, (3, 4, 5), 4, 2, 128, (44, 42, 42), "bf16", 0, False, 0, 0),
    (1, (2, 7, 9), 3, 3, 128, (32, 48, 48), "bf16", 1, True, 0, 0),
    (1, (2, 7, 9), 3, 1, 128, (32, 48, 48), "bf16", 0, True, 0, 0),
    (1, (5, 3, 11), 5, 0, 64, (16, 24, 24), "f32", 0, False, 0, 0),         # Q alone
    (1, (5, 3, 11), 0, 5, 64, (16, 24, 24), "f32", 1, True, 0, 0),          # K alone
    (3, (2, 3, 3), 2, 2, 64, (8, 12, 12), "bf16", 1, False, 64, 0),         # part of the head turns, a wider token
    (3, (2, 3, 3), 2, 2, 64, (8, 12, 12), "f32", 1, True, 64, 0),
    (1, (2, 5, 7), 4, 4, 72, (18, 26, 26), "bf16", 1, True, 0, 0),          # pairs 35 apart: single elements
    (1, (2, 5, 7), 4, 4, 72, (18, 26, 26), "bf16", 1, False, 0, 0),
    (1, (2, 5, 7), 4, 4, 72, (20, 20, 28), "bf16", 0, True, 0, 0),          # pairs 34 apart
    (1, (4, 4, 4), 2, 2, 6, (2, 2, 2), "bf16", 1, False, 0, 0),
    (1, (4, 4, 4), 2, 2, 7, (2, 2, 2), "bf16", 1, False, 0, 0),             # an odd width
    (1, (4, 4, 4), 2, 2, 7, (2, 2, 2), "f32", 0, True, 0, 0),
    (1, (4, 4, 4), 2, 2, 1, (0, 0, 0), "f32", 0, False, 0, 0),              # nothing turns
    (1, (4, 4, 4), 2, 2, 16, (0, 0, 0), "bf16", 1, True, 0, 0),
    (1, (1, 1, 300), 2, 1, 256, (0, 0, 256), "bf16", 1, False, 0, 0),       # one axis, the widest head
    (2, (3, 4, 5), 2, 2, 128, (44, 42, 42), "bf16", 1, False, 3, 1),        # nothing aligned
    (2, (3, 4, 5), 2, 2, 128, (44, 42, 42), "bf16", 1, True, 3, 1),
    (2, (3, 4, 5), 2, 2, 128, (44, 42, 42), "f32", 1, False, 2, 2),         # 8-byte vectors
    (1, (9, 24, 42), 8, 8, 128, (44, 42, 42), "bf16", 1, False, 0, 0),      # more than one wave of blocks
]


@pytest.mark.parametrize("B,grid,Hq,Hk,d,axes,dtype,layout,halves,pad,offset", CASES)
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("where", ["grid", "far", "given"])
def test_rope(B, grid, Hq, Hk, d, axes, dtype, layout, halves, pad, offset, backward, where):
    import torch
    from frame_wise_linear_b200 import vda
    rng = np.random.default_rng(B + 7 * Hq + d)
    dt = dtype_of(dtype)
    N = grid[0] * grid[1] * grid[2]
    q, qo, qfull, ldq = _tensors(B, N, Hq, d, dt, layout, pad, offset, rng)
    k, ko, kfull, ldk = _tensors(B, N, Hk, d, dt, layout, pad, offset, rng)
    pos0, step = ((1e6, 0.25, -3.0), (1.0, 0.5, 2.0)) if where == "far" else ((0.0,) * 3, (1.0,) * 3)
    given = None
    pos = np.broadcast_to(o.rope_grid(*grid, pos0, step), (B, N, 3))
    if where == "given":
        given = torch.from_numpy(rng.integers(-5, 100000, (B, N, 3)).astype(np.float32) +
                                 rng.integers(0, 2, (B, N, 3)).astype(np.float32) / 2).cuda()
        pos = f64(given)
    p = vda.make_rope_problem(B, *grid, Hq, Hk, d, axes, code_of(dtype), layout=layout,
                              pairing=vda.VDA_ROPE_HALVES if halves else vda.VDA_ROPE_INTERLEAVED, theta=1000.0,
                              pos0=pos0, step=step, ld_q=ldq, ld_k=ldk, ld_qr=ldq, ld_kr=ldk)
    (vda.vda_rope_backward if backward else vda.vda_rope)(p, q, k, given, qo, ko)
    rot = sum(axes)
    for x, y, full, H in ((q, qo, qfull, Hq), (k, ko, kfull, Hk)):
        if H == 0:
            continue
        a, got = _as_tokens(x, B, N, H, d, layout), _as_tokens(y, B, N, H, d, layout)
        for i in range(B):
            ref = o.rope(a[i], pos[i], axes, 1000.0, halves, inverse=backward)
            size = np.abs(a[i, ..., :rot])
            if halves:
                size = np.concatenate([size[..., : rot // 2] + size[..., rot // 2:]] * 2, -1)
            else:
                size = np.repeat(size[..., 0::2] + size[..., 1::2], 2, axis=-1)
            err = 8 * U32 * size
            assert_close(got[i, ..., :rot], ref[..., :rot], err + half_step(dt) * (np.abs(ref[..., :rot]) + err))
            assert np.array_equal(got[i, ..., rot:], a[i, ..., rot:])      # copied bit for bit
        assert untouched(full, y, FILL)


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("halves", [False, True])
def test_backward_undoes_forward_and_is_its_transpose(layout, halves):
    import torch
    from frame_wise_linear_b200 import vda
    B, grid, H, d, axes = 2, (3, 5, 7), 3, 64, (16, 20, 24)
    N = 105
    shape = (B, H, N, d) if layout == 0 else (B, N, H, d)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, v = (torch.randn(shape, device="cuda", generator=g) for _ in range(2))
    p = vda.make_rope_problem(B, *grid, H, H, d, axes, vda.VDA_DTYPE_F32, layout=layout, pairing=int(halves))
    y, z, back, vt = (torch.empty_like(x) for _ in range(4))
    vda.vda_rope(p, x, v, None, y, z)
    vda.vda_rope_backward(p, y, v, None, back, vt)
    assert float((back - x).abs().max()) <= 32 * U32 * float(x.abs().max())     # twice 8 u (|a| + |b|)
    # <rope(x), v> = <x, rope_backward(v)>: each side off by 8 u of 2 |x||v| a term
    lhs, rhs = (y.double() * v.double()).sum(), (x.double() * vt.double()).sum()
    assert abs(float(lhs - rhs)) <= 32 * U32 * float(4 * x.abs().max() * v.abs().double().sum())
    # differences of the forward along v (it is linear): exact up to the same bound
    xp, xm = torch.empty_like(x), torch.empty_like(x)
    vda.vda_rope(p, x + v, x - v, None, xp, xm)
    assert float(((xp - xm) / 2 - z).abs().max()) <= 64 * U32 * float((x.abs() + v.abs()).max())


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("layout,pad", [(0, 0), (1, 0), (1, 40)])
def test_in_place(layout, pad, halves):
    import torch
    from frame_wise_linear_b200 import vda
    rng = np.random.default_rng(0)
    B, grid, H, d = 2, (2, 5, 6), 3, 128
    q, qo, _, ld = _tensors(B, 60, H, d, torch.bfloat16, layout, pad, 0, rng)
    k, ko, _, _ = _tensors(B, 60, H, d, torch.bfloat16, layout, pad, 0, rng)
    p = vda.make_rope_problem(B, *grid, H, H, d, (44, 42, 42) if not halves else (32, 48, 48), vda.VDA_DTYPE_BF16,
                              layout=layout, pairing=int(halves), ld_q=ld, ld_k=ld, ld_qr=ld, ld_kr=ld)
    vda.vda_rope(p, q, k, None, qo, ko)
    vda.vda_rope(p, q, k, None, q, k)
    assert torch.equal(q, qo) and torch.equal(k, ko)


def test_different_strides_in_and_out():
    """Out of a fused projection into dense tensors, and the gradients back into one."""
    import torch
    from frame_wise_linear_b200 import vda
    B, grid, H, d = 2, (2, 3, 4), 2, 64
    N = 24
    qkv = torch.randn(B, N, 3, H, d, device="cuda")
    q, k = qkv[:, :, 0], qkv[:, :, 1]
    ld = 3 * H * d
    p = vda.make_rope_problem(B, *grid, H, H, d, (16, 24, 24), vda.VDA_DTYPE_F32, layout=1, ld_q=ld, ld_k=ld)
    qr, kr, q2, k2 = (torch.empty(B, N, H, d, device="cuda") for _ in range(4))
    vda.vda_rope(p, q, k, None, qr, kr)
    dense = vda.make_rope_problem(B, *grid, H, H, d, (16, 24, 24), vda.VDA_DTYPE_F32, layout=1)
    vda.vda_rope(dense, q.contiguous(), k.contiguous(), None, q2, k2)
    assert torch.equal(qr, q2) and torch.equal(kr, k2)
    grads = torch.full_like(qkv, FILL)
    vda.vda_rope_backward(p, qr, kr, None, grads[:, :, 0], grads[:, :, 1])
    vda.vda_rope_backward(dense, qr, kr, None, q2, k2)
    assert torch.equal(grads[:, :, 0], q2) and torch.equal(grads[:, :, 1], k2)
    assert bool((grads[:, :, 2] == FILL).all())


def test_values_that_are_not_finite_stay_in_their_pair():
    import torch
    from frame_wise_linear_b200 import vda
    for halves in (False, True):
        x = torch.randn(1, 12, 1, 64, device="cuda")
        x[0, 3, 0, 2], x[0, 5, 0, 40], x[0, 7, 0, 60] = float("nan"), float("inf"), float("nan")
        y, z = torch.empty_like(x), torch.empty_like(x)
        p = vda.make_rope_problem(1, 3, 2, 2, 1, 1, 64, (16, 16, 16), vda.VDA_DTYPE_F32, layout=1, pairing=int(halves))
        vda.vda_rope(p, x, x, None, y, z)
        bad = set(map(tuple, (~torch.isfinite(y[0, :, 0])).nonzero().tolist()))
        pair = (lambda c: {c, (c + 24) % 48}) if halves else (lambda c: {c, c ^ 1})
        want = {(3, c) for c in pair(2)} | {(5, c) for c in pair(40)} | {(7, 60)}
        assert bad == want, (halves, bad)
        # a position that is not finite: that token's turned channels alone
        pos = torch.zeros(1, 12, 3, device="cuda")
        pos[0, 4, 1] = float("nan")
        x = torch.randn(1, 12, 1, 64, device="cuda")
        vda.vda_rope(p, x, x, pos, y, z)
        assert torch.equal(torch.isnan(y).any(-1).flatten().nonzero().flatten().cpu(), torch.tensor([4]))
        assert not bool(torch.isnan(y[0, 4, 0, 48:]).any())


@pytest.mark.slow
def test_offsets_past_32_bits():
    """More than 2^32 elements in Q, token-major: the last token of the last item."""
    import torch
    from frame_wise_linear_b200 import vda
    B, T, h, w, H, d = 1, 130, 64, 129, 32, 128
    N = T * h * w
    assert B * N * H * d > 1 << 32
    q = torch.empty(B, N, H, d, dtype=torch.bfloat16, device="cuda")
    q.uniform_(-1, 1)
    last = f64(q[0, -2:])
    p = vda.make_rope_problem(B, T, h, w, H, 0, d, (44, 42, 42), vda.VDA_DTYPE_BF16, layout=1)
    vda.vda_rope(p, q, None, None, q, None)
    ref = o.rope(last, o.rope_grid(T, h, w)[-2:], (44, 42, 42))
    assert_close(f64(q[0, -2:]), ref, 16 * U32 + 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -6))
