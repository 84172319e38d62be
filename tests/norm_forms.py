"""The layer norm's choice of a kernel, replayed on the host: which form a call takes, and how many rows a thread adds.

Follows shape_for, grid_for, batched, kinds_for, wide, shifted, run_shape and run_type of vda_layer_norm.cuh; the
tests that use it say which forms their cases take, and fail when a case no longer takes the form it is there for.
"""
from __future__ import annotations

from collections import namedtuple

THREADS = 256
SMS = 148
PASSES = ("fwd", "fwd_codes", "bwd", "bwd_codes", "apply")

# bytes: of the type; ve: elements of a vector; per: of a thread; fill: all, some or shift; rows: of a batch;
# thread_rows: rows that a thread adds to its column sums at most; groups: rows that a CTA works on side by side.
Form = namedtuple("Form", "step bytes ve per fill rows batches thread_rows groups")


def _up(a, b):
    return -(-a // b)


def _shape(D, ve, kinds=0):
    least = 32 // ve
    nvec = (D + 2 * ve - 2) // ve if kinds else D // ve
    per = 8 if nvec * ve <= 8 * least else 16 if nvec * ve <= 16 * THREADS else 32
    need = _up(nvec, per // ve)
    tpr = least
    while tpr < 32 and tpr < need:
        tpr *= 2
    if need > 32:
        tpr = _up(need, 32) * 32
    groups = 0 if tpr > THREADS else THREADS // tpr
    fill = "shift" if kinds else "all" if ve > 1 and nvec == tpr * (per // ve) else "some"
    return per, groups, kinds or 1, fill


def _grid(rows, per, groups, kinds, n):
    batches = _up(_up(rows, kinds), groups * n)
    return min(batches, SMS * (1 if per == 32 else 2) // kinds) * kinds


def form(step, tokens, heads, D, element, pad=0, place=0, codes_place=0):
    """The form of one pass: `pad` elements between tokens, tensors `place` elements (codes `codes_place`) behind
    a 16-byte boundary."""
    ve, rows, width = 16 // element, tokens * heads, heads * D
    codes = step in ("fwd_codes", "bwd_codes", "apply")
    if pad == 0:
        heads, width = 1, D
    wide = D % ve == 0 and (width + pad) % ve == 0 and place % ve == 0 and (not codes or codes_place % ve == 0)
    kinds = 0
    if not wide:
        shifted = step != "fwd_codes" and D >= 4 * ve and pad == 0 and (not codes or codes_place % ve == place % ve) \
            and _shape(D, ve, 1)[1] > 0
        if shifted:
            kinds = 1
            while kinds * D % ve:
                kinds *= 2
            kinds = min(kinds, rows)
        else:
            ve = 1
    per, groups, kinds, fill = _shape(D, ve, kinds)
    backward = step in ("bwd", "bwd_codes")
    if ve == 1:
        most = 1
    elif step == "bwd_codes" and element == 2 and per == 16 and fill != "shift":
        most = 4
    else:
        most = (64 if element == 4 and not backward else 128) // (per * element) // (2 if backward else 1)
        most = min(max(most, 1), 4)
    if rows < _grid(rows, per, groups, kinds, 1) * groups * most:
        most = 1
    ctas = _grid(rows, per, groups, kinds, most) // kinds
    batches = _up(_up(_up(rows, kinds), groups * most), ctas)
    return Form(step, element, ve, per, fill, most, batches, batches * most, groups)
