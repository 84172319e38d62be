"""Helpers shared by the token operators' GPU tests."""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24                       # half a step of float32, relative


def half_step(dtype) -> float:
    """Largest relative error of one rounding to the type."""
    import torch
    return torch.finfo(dtype).eps / 2


def dtype_of(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def code_of(name):
    from frame_wise_linear_b200 import vda
    return {"bf16": vda.VDA_DTYPE_BF16, "f32": vda.VDA_DTYPE_F32}[name]


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def inside(rows, width, ld, dtype, fill, offset=0):
    """A [rows, width] view with `ld` elements a row, `offset` elements into a filled buffer, and the buffer."""
    import torch
    full = torch.full((offset + max(rows, 1) * ld + 64,), fill, dtype=dtype, device="cuda")
    return full[offset:].as_strided((rows, width), (ld, 1)), full


def untouched(full, view, fill) -> bool:
    """Nothing outside the view has changed (the view is overwritten with the fill to check it)."""
    view.fill_(fill)
    return bool((full == fill).all())


def assert_close(got, ref, bound, what=""):
    """|got - ref| <= bound element by element (arrays or scalars); NaN must meet NaN."""
    got, ref = np.asarray(got), np.asarray(ref)
    bound = np.broadcast_to(np.asarray(bound, dtype=np.float64), ref.shape)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan), (what, "NaN in other places")
    over = np.where(nan, 0.0, np.abs(got - ref) - bound)
    i = np.unravel_index(np.argmax(over), over.shape) if over.size else None
    assert over.size == 0 or over[i] <= 0, (what, i, got[i], ref[i], bound[i])
