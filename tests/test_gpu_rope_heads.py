"""Rotary positions where a thread takes its heads in several passes: the refill of the heads on their way, of their
partners, the change from Q to K within a pass, and a last pass that is not full.

A CTA takes a tile of tokens; `lanes` threads share a unit of a token, and each has kAhead of every lanes-th head on its
way at once.  _walk replays the choice (launch and kAhead of vda_rope.cu) and the cases are held to it on the CPU.
Bounds as in test_gpu_rope.py.
"""
import numpy as np
import pytest

from oracle import token_oracle as o
from token_testutil import U32, assert_close, code_of, dtype_of, f64, half_step, inside, untouched

FILL = 7.0

# (T, h, w), Hq, Hk, d, axes, dtype, layout, halves, pad, place, elements of a load
CASES = [
    # half the width apart
    ((3, 28, 30), 13, 8, 128, (44, 42, 42), "bf16", 1, True, 0, 0, 8),
    ((3, 28, 30), 13, 8, 128, (32, 48, 48), "bf16", 1, True, 0, 0, 8),
    ((3, 28, 30), 13, 8, 128, (32, 48, 48), "bf16", 0, True, 0, 0, 8),
    ((3, 28, 30), 11, 6, 128, (32, 48, 32), "bf16", 1, True, 16, 0, 8),     # 16 channels copied
    ((3, 28, 30), 15, 4, 72, (24, 24, 24), "bf16", 1, True, 0, 0, 4),       # 36 apart
    ((3, 28, 30), 15, 4, 72, (20, 20, 28), "bf16", 0, True, 0, 0, 2),       # 34 apart
    ((2, 21, 30), 16, 3, 72, (18, 26, 26), "bf16", 1, True, 0, 0, 1),       # 35 apart
    ((2, 21, 30), 16, 3, 72, (18, 26, 26), "bf16", 0, True, 0, 0, 1),
    ((3, 28, 30), 9, 8, 128, (32, 48, 48), "f32", 1, True, 0, 0, 4),
    ((3, 28, 30), 17, 2, 72, (20, 20, 28), "f32", 1, True, 0, 0, 2),
    ((2, 21, 30), 9, 6, 70, (18, 26, 26), "f32", 0, True, 0, 0, 1),
    # neighbours
    ((3, 28, 30), 25, 10, 128, (44, 42, 42), "bf16", 1, False, 0, 0, 8),
    ((3, 28, 30), 25, 10, 128, (44, 42, 42), "bf16", 0, False, 0, 0, 8),
    ((2, 21, 30), 31, 4, 128, (44, 42, 42), "bf16", 1, False, 2, 2, 2),
    ((2, 21, 30), 31, 4, 128, (44, 42, 42), "bf16", 1, False, 3, 1, 0),     # pairs as single elements
    ((2, 21, 30), 19, 12, 63, (18, 20, 22), "bf16", 0, False, 0, 0, 0),     # and the last channel of an odd width
    ((3, 28, 30), 25, 10, 128, (44, 42, 42), "f32", 1, False, 0, 0, 4),
    ((2, 21, 30), 31, 4, 128, (44, 42, 42), "f32", 1, False, 2, 2, 2),
    ((2, 21, 30), 19, 12, 63, (18, 20, 22), "f32", 1, False, 1, 0, 0),
]


def _walk(grid, Hq, Hk, d, axes, dtype, layout, halves, pad, place, load):
    """Heads of one pass of a unit's threads, and whether a pass holds both Q's last head and K's first."""
    element, rot, tokens = {"bf16": 2, "f32": 4}[dtype], sum(axes), grid[0] * grid[1] * grid[2]
    fits = lambda n: d % n == 0 and (not halves or rot // 2 % n == 0) and place % n == 0 and \
        (layout == 0 or (Hq * d + pad) % n == 0 and (Hk * d + pad) % n == 0)  # noqa: E731
    widest = 16 // element
    if halves:
        ve = next(n for n in (8, 4, 2, 1) if n <= widest and fits(n))
        units, size = rot // 2 // ve + (d - rot) // ve, 2 * ve
    else:
        ve = next(n for n in (widest, 2, 0) if n == 0 or fits(n))
        units, size = (d // ve, ve) if ve else ((d + 1) // 2, 2)
    assert ve == load, (ve, load)
    ahead = 2 if halves and ve == 1 else min(64 // (size * element), 4)
    tile = max(256 // (units * 4), 1)
    while tile > 1 and -(-tokens // tile) < 296:
        tile = (tile + 1) // 2
    once = ahead * (256 // (tile * units))
    return once, Hq % once != 0


@pytest.mark.parametrize("case", CASES)
def test_cases_walk(case):
    once, both = _walk(*case)
    total = case[1] + case[2]
    assert total > once and total % once and both, (once, total)


def _tensors(N, H, d, dt, layout, pad, place, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape, ld = ((H * N, d), d) if layout == 0 else ((N, H * d), H * d + pad)
    x, _ = inside(*shape, ld, dt, float("nan"), place)
    x.copy_(torch.randn(shape, device="cuda", generator=g))
    y, full = inside(*shape, ld, dt, FILL, place)
    return x, y, full, ld if layout and pad else 0


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("backward", [False, True])
def test_heads_in_several_passes(case, backward):
    import torch
    from frame_wise_linear_b200 import vda
    grid, Hq, Hk, d, axes, dtype, layout, halves, pad, place, _ = case
    dt, N, rot = dtype_of(dtype), grid[0] * grid[1] * grid[2], sum(axes)
    q, qo, qfull, ldq = _tensors(N, Hq, d, dt, layout, pad, place, 1)
    k, ko, kfull, ldk = _tensors(N, Hk, d, dt, layout, pad, place, 2)
    p = vda.make_rope_problem(1, *grid, Hq, Hk, d, axes, code_of(dtype), layout=layout, pairing=int(halves),
                              theta=1000.0, ld_q=ldq, ld_k=ldk, ld_qr=ldq, ld_kr=ldk)
    call = vda.vda_rope_backward if backward else vda.vda_rope
    call(p, q, k, None, qo, ko)
    pos = o.rope_grid(*grid)
    for x, y, full, H in ((q, qo, qfull, Hq), (k, ko, kfull, Hk)):
        tokens = lambda t: f64(t).reshape(H, N, d).transpose(1, 0, 2) if layout == 0 else f64(t).reshape(N, H, d)  # noqa: E731
        a, got = tokens(x), tokens(y)
        ref = o.rope(a, pos, axes, 1000.0, halves, inverse=backward)
        size = np.abs(a[..., :rot])
        if halves:
            size = np.concatenate([size[..., : rot // 2] + size[..., rot // 2:]] * 2, -1)
        else:
            size = np.repeat(size[..., 0::2] + size[..., 1::2], 2, axis=-1)
        err = 8 * U32 * size
        assert_close(got[..., :rot], ref[..., :rot], err + half_step(dt) * (np.abs(ref[..., :rot]) + err))
        assert np.array_equal(got[..., rot:], a[..., rot:])
    want = qo.clone(), ko.clone()
    assert untouched(qfull, qo, FILL) and untouched(kfull, ko, FILL)
    call(p, q, k, None, q, k)                       # in place
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
