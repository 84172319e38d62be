"""Every stage of an attention block's training step against the oracles, at the values that the stage was given.

The step is the one of test_gpu_token_run.py.  There its end is compared with a chain of oracles that skips the 8-bit
rounding, which needs a wide bound; here each stage starts from the tensors that the stage before it left, the
checkpoints' own values among them, so that each is held to its own rounding.  VDA's stages take the repository's bar for
one operator on bf16 (2e-2 in the 2-norm); the token operators take the bounds of test_gpu_norm_forms.py and
test_gpu_rope.py; a product of two bf16 matrices with K terms is summed in float32 (K u of the sum of magnitudes, in
any order) and rounded once.
"""
import numpy as np
import pytest

from oracle import token_oracle as o
from oracle import vda_oracle as vo
from test_gpu_token_run import _Block
from token_testutil import U32, assert_close, f64
from vda_testutil import rel_fro

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8
AXES = (44, 42, 42)


def _product(got, a, b, what):
    ref, size = a @ b, np.abs(a) @ np.abs(b)
    err = a.shape[1] * U32 * size
    assert_close(got, ref, err + HALF * (np.abs(ref) + err), what)


def _norm(Y, mean, rstd, X, w, b, what):
    """Y at the statistics that the call returned, and those."""
    _, m_ref, r_ref, _ = o.layer_norm(X, eps=1e-6)
    XR = U32 * (np.abs(X).max(1) + np.abs(m_ref)) * r_ref
    assert_close(mean, m_ref, 32 * U32 * np.abs(X).max(1), what)
    assert_close(rstd, r_ref, r_ref * ((32 * U32 + 64 * XR + (32 * XR) ** 2) / 2 + 3 * U32) * (1 + 1e-3), what)
    xh = (X - mean[:, None]) * rstd[:, None]
    ref = xh * w + b
    err = U32 * (2 * np.abs(xh * w) + np.abs(ref)) * (1 + 1e-5)
    assert_close(Y, ref, err + HALF * (np.abs(ref) + err), what)
    return xh


def _norm_backward(dX, dW, db, dY, xh, rstd, w, what):
    """`xh` float64 of the operands; every row adds at most rows + 82 times to a column (64 groups and 18 more)."""
    ref, dw_ref, db_ref = o.layer_norm_backward(dY, xh, rstd, w)
    g, h = np.abs(dY * w), np.abs(xh)
    gx = (g * h).mean(1, keepdims=True)
    err = rstd[:, None] * U32 * (3 * g + 32 * g.mean(1, keepdims=True) + 37 * h * gx) * (1 + 1e-5)
    assert_close(dX, ref, err + HALF * (np.abs(ref) + err), what)
    n = (len(dY) + 82) * U32
    assert_close(dW, dw_ref, n * np.abs(dY * xh).sum(0), what)
    if db is not None:
        assert_close(db, db_ref, n * np.abs(dY).sum(0), what)


def _rope(got, x, pos, inverse, what):
    ref = o.rope(x, pos, AXES, inverse=inverse)
    err = 8 * U32 * np.repeat(np.abs(x[..., 0::2]) + np.abs(x[..., 1::2]), 2, axis=-1)
    assert_close(got, ref, err + HALF * (np.abs(ref) + err), what)


@pytest.mark.parametrize("seed", [0, 5])
def test_each_stage_at_its_own_inputs(seed):
    from frame_wise_linear_b200 import vda
    b = _Block(seed=seed)
    b.step()
    vda.vda_sync_status(b.ws)
    N, H, d, C = b.N, b.H, b.d, b.C
    pos = o.rope_grid(b.T, b.gh, b.gw)
    P, qkvg = f64(b.P), f64(b.qkvg)
    part = lambda t, i: t[:, i * C: (i + 1) * C]  # noqa: E731
    heads = lambda t: f64(t)[0]  # noqa: E731      [N, H, d]

    # Forward.
    _norm(f64(b.Y), f64(b.mean), f64(b.rstd), f64(b.X), f64(b.Wn), f64(b.bn), "norm")
    _product(qkvg, f64(b.Y), P, "projection")
    per_head = []
    for i, (y, s, w, yr) in enumerate(((b.q, b.qs, b.Wq, b.qr), (b.k, b.ks, b.Wk, b.kr))):
        x = part(qkvg, i).reshape(-1, d)
        per_head.append(_norm(heads(y).reshape(-1, d), f64(s[0]), f64(s[1]), x, f64(w), 0.0, "head norm"))
        _rope(heads(yr), heads(y), pos, False, "rope")
    kept = []
    for x, (codes, scales) in zip((b.qr, b.kr, b.v, b.g), b.kept):
        c, s = o.checkpoint(heads(x).reshape(-1, d))
        assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s)
        kept.append(o.checkpoint_values(c, s).reshape(N, H, d))
    frames = lambda t, h: t[:, h].reshape(b.T, b.n, d)  # noqa: E731
    O, grads, dO = np.empty((N, H, d)), [np.empty((N, H, d)) for _ in range(4)], heads(b.dO)
    for h in range(H):
        O[:, h] = vo.vda_head(*(frames(heads(t), h) for t in (b.qr, b.kr, b.v, b.g)), None, None,
                              float(b.n)).reshape(N, d)
        got = vo.vda_head_backward(*(frames(t, h) for t in kept), None, None, float(b.n), frames(dO, h))
        for t, name in zip(grads, ("dQ", "dK", "dV", "dG")):
            t[:, h] = got[name].reshape(N, d)
    assert rel_fro(heads(b.O), O) <= 2e-2

    # Backward, from the checkpoints' values.
    for got, ref, what in zip((b.dqr, b.dkr, b.dv, b.dg), grads, ("dQ", "dK", "dV", "dG")):
        assert rel_fro(heads(got), ref) <= 2e-2, (what, rel_fro(heads(got), ref))
    dqkvg = f64(b.dqkvg)
    for i, (s, w, dyr, dy, xh, dw) in enumerate(((b.qs, b.Wq, b.dqr, b.dq, per_head[0], b.dWq),
                                                 (b.ks, b.Wk, b.dkr, b.dk, per_head[1], b.dWk))):
        _rope(heads(dy), heads(dyr), pos, True, "rope backward")
        _norm_backward(part(dqkvg, i).reshape(-1, d), f64(dw), None, heads(dy).reshape(-1, d), xh, f64(s[1]), f64(w),
                       "head norm backward")
    for i, t in ((2, b.dv), (3, b.dg)):
        assert np.array_equal(part(dqkvg, i), heads(t).reshape(N, C))
    xh = o.checkpoint_values(b.nc.cpu().numpy(), b.ns.cpu().numpy())
    own = (f64(b.X) - f64(b.mean)[:, None]) * f64(b.rstd)[:, None]
    e = np.repeat(b.ns.cpu().numpy().astype(float) - 127, 32, axis=1)[:, :C]
    assert_close(xh, own, np.maximum(2.0 ** -4 * np.abs(own), 2.0 ** (e - 10)) + 4 * U32 * np.abs(own), "norm's codes")
    again = xh * f64(b.Wn) + f64(b.bn)
    assert_close(f64(b.Yagain), again, U32 * np.abs(again) + HALF * np.abs(again) * (1 + U32), "norm again")
    _product(f64(b.dP), f64(b.Yagain).T, dqkvg, "dP")
    _product(f64(b.dY), dqkvg, P.T, "dY")
    _norm_backward(f64(b.dX), f64(b.dWn), f64(b.dbn), f64(b.dY), xh, f64(b.rstd), f64(b.Wn), "norm backward")
