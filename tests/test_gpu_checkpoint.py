"""8-bit checkpoints: codes and scale bytes bit for bit the oracle's, and the values they stand for."""
import numpy as np
import pytest

from oracle import token_oracle as o
from token_testutil import code_of, dtype_of, f64, inside, untouched

pytestmark = pytest.mark.gpu

FILL = 7.0

CASES = [
    # rows, D, dtype, pad, offset
    (1, 1, "bf16", 0, 0), (1, 31, "f32", 0, 0), (3, 32, "bf16", 0, 0), (3, 33, "f32", 0, 0),
    (5, 8, "bf16", 0, 0), (5, 4, "f32", 0, 0), (7, 40, "bf16", 0, 0), (7, 36, "f32", 0, 0),
    (100, 128, "bf16", 0, 0), (100, 128, "f32", 0, 0), (64, 1001, "f32", 0, 0), (64, 1001, "bf16", 0, 0),
    (33, 128, "bf16", 64, 0), (33, 128, "f32", 3, 1), (33, 100, "bf16", 1, 0), (9, 4096, "bf16", 0, 0),
    (2, 70000, "bf16", 0, 0), (40000, 128, "bf16", 0, 0),
]


def _draw(rows, D, dtype, seed):
    """Rows of very different sizes, with zeros, blocks of zeros and values at the type's ends among them."""
    import torch
    rng = np.random.default_rng(seed + rows + D)
    x = rng.normal(size=(rows, D)) * np.exp(rng.normal(0, 8, (rows, 1)))
    x[rng.random((rows, D)) < 0.05] = 0.0
    x[rng.random(rows) < 0.1] = 0.0
    return torch.from_numpy(x).to(dtype_of(dtype))


def _pack(X, rows, D, dtype, ld):
    import torch
    from frame_wise_linear_b200 import vda
    nblk = -(-D // 32)
    codes = torch.full((rows * D + 64,), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows * nblk + 64,), 9, dtype=torch.uint8, device="cuda")
    p = vda.make_checkpoint_problem(rows, D, code_of(dtype), ld=ld)
    vda.vda_checkpoint_pack(p, X, codes, scales)
    assert bool((codes[rows * D:] == 9).all()) and bool((scales[rows * nblk:] == 9).all())
    return p, codes[: rows * D].reshape(rows, D), scales[: rows * nblk].reshape(rows, nblk)


def _same_codes(got, want):
    """Equal, but for the sign of a NaN."""
    got, want = got.cpu().numpy(), want
    nan = (want & 0x7F) == 0x7F
    return np.array_equal(got[~nan], want[~nan]) and np.all((got[nan] & 0x7F) == 0x7F)


@pytest.mark.parametrize("rows,D,dtype,pad,offset", CASES)
def test_pack_and_unpack(rows, D, dtype, pad, offset):
    from frame_wise_linear_b200 import vda
    ld = D + pad
    X, _ = inside(rows, D, ld, dtype_of(dtype), 0.0, offset)
    X.copy_(_draw(rows, D, dtype, 1).cuda())
    p, codes, scales = _pack(X, rows, D, dtype, ld if pad else 0)
    c, s = o.checkpoint(f64(X))
    assert np.array_equal(scales.cpu().numpy(), s)
    assert _same_codes(codes, c)
    Y, full = inside(rows, D, ld, X.dtype, FILL, offset)
    vda.vda_checkpoint_unpack(p, codes, scales, Y)
    assert np.array_equal(f64(Y), o.checkpoint_values(c, s))     # 4 bits at a power of two: exact in either type
    assert untouched(full, Y, FILL)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 61])
def test_special_values(dtype, D):
    """NaN and infinities, blocks of nothing else, the largest and smallest magnitudes, both zeros."""
    import torch
    from frame_wise_linear_b200 import vda
    dt = dtype_of(dtype)
    big, tiny = float(torch.finfo(dt).max), float(torch.finfo(dt).smallest_normal)
    X = torch.randn(12, D, device="cuda").to(dt)
    X[0, 3], X[1, 4], X[2, 5] = float("nan"), float("inf"), -float("inf")
    X[3, :32] = float("inf")
    X[4, :32] = float("nan")
    X[5, 0], X[5, 1] = big, -big
    X[6] = X[6] * tiny
    X[7, :32] = 0.0
    X[8, :32] = -0.0
    X[9, :32] = torch.tensor([448.0, 449.0, 464.0, 480.0] * 8, device="cuda").to(dt)
    X[10, :32] = torch.tensor([1.0625, 1.1875, 17.0, 19.0, -17.0, -19.0, 2.0 ** -10, 3 * 2.0 ** -10] * 4,
                              device="cuda").to(dt)                 # halfway between two codes
    X[10, 0] = 448.0
    X[11, :32] = torch.tensor([448.0 * 2.0 ** -127, 2.0 ** -136] * 16, device="cuda").to(dt)
    p, codes, scales = _pack(X, 12, D, dtype, 0)
    c, s = o.checkpoint(f64(X))
    assert np.array_equal(scales.cpu().numpy(), s)
    assert _same_codes(codes, c)
    Y = torch.empty_like(X)
    vda.vda_checkpoint_unpack(p, codes, scales, Y)
    v, ref = f64(Y), o.checkpoint_values(c, s)
    assert np.array_equal(np.isnan(v), np.isnan(ref)) and np.array_equal(v[~np.isnan(v)], ref[~np.isnan(ref)])
    assert np.all(np.isfinite(v[5])) and np.array_equal(np.isnan(v[0]), np.arange(D) == 3)
    assert bool(torch.signbit(Y[8, :32]).all())


def test_every_code_unpacks():
    """All 256 codes at several scales, to both types."""
    import torch
    from frame_wise_linear_b200 import vda
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(8, 1).contiguous()
    scales = torch.tensor([0, 1, 7, 100, 127, 130, 200, 246], dtype=torch.uint8, device="cuda")[:, None].repeat(1, 8)
    ref = o.checkpoint_values(codes.cpu().numpy(), scales.cpu().numpy())
    for dtype in ("f32", "bf16"):
        Y = torch.empty(8, 256, dtype=dtype_of(dtype), device="cuda")
        vda.vda_checkpoint_unpack(vda.make_checkpoint_problem(8, 256, code_of(dtype)), codes, scales.contiguous(), Y)
        v = f64(Y)
        assert np.array_equal(np.isnan(v), np.isnan(ref))
        # bf16 below its smallest normal rounds to multiples of 2^-133
        slack = 2.0 ** -134 if dtype == "bf16" else 0.0
        assert np.all(np.abs(v - ref)[~np.isnan(ref)] <= slack)


@pytest.mark.slow
def test_offsets_past_32_bits():
    import torch
    from frame_wise_linear_b200 import vda
    rows, D = (1 << 25) + 3, 128
    X = torch.empty(rows, D, dtype=torch.bfloat16, device="cuda")
    X.uniform_(-1, 1)
    p = vda.make_checkpoint_problem(rows, D, vda.VDA_DTYPE_BF16)
    codes = torch.empty(rows, D, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, 4, dtype=torch.uint8, device="cuda")
    vda.vda_checkpoint_pack(p, X, codes, scales)
    c, s = o.checkpoint(f64(X[-4:]))
    assert np.array_equal(codes[-4:].cpu().numpy(), c) and np.array_equal(scales[-4:].cpu().numpy(), s)
    vda.vda_checkpoint_unpack(p, codes, scales, X)
    assert np.array_equal(f64(X[-4:]), o.checkpoint_values(c, s))
