"""Cases of the token operators around the attention branches: layer norm, rotary positions, 8-bit checkpoints.

A case names one operator and its sizes.  ``run`` computes it either in its
plain form (elementary torch operations in 32 bits, angles in 64) or, where
``own`` is set, with the calls a user makes of
:mod:`frame_wise_linear_b200.vda`; ``exact`` computes it again in 64 bits.

Operators (``op``):
  norm           y = (x - mean) rstd w + b, with mean and rstd (training keeps them)
  norm_ckpt      the same, and the normalised row kept in 8 bits (blocks of 32, a power-of-two scale each)
  norm_bwd       dx, dw, db from dy, x, mean, rstd
  norm_bwd_ckpt  dx, dw, db from dy and the 8-bit normalised row, and y again from it (the next product's operand)
  rope           rotary positions over (time, height, width) on Q and K
  rope_bwd       its gradients
  pack           a tensor into 8 bits and back
"""
import math

import torch

own = False

EPS = 1e-6
THETA = 10000.0
BLOCK = 32
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_MOST_BYTES = 4 * 45 * 1008 * 4096 * 2   # Q, K in and out at 45 x 1008 tokens, 32 heads x 128


# ---------------------------------------------------------------- cases
def _norm(name, op, tokens, heads, D, dtype, w="f32", strided=False, affine=True):
    return dict(name=name, op=op, tokens=tokens, heads=heads, D=D, dtype=dtype, w=w, strided=strided, affine=affine)


def _rope(name, op, B, T, gh, gw, hq, hk, d, dt, dy, dx, dtype, layout, pairing, given=False, strided=False, t0=0.0):
    return dict(name=name, op=op, B=B, T=T, gh=gh, gw=gw, hq=hq, hk=hk, d=d, dt=dt, dy=dy, dx=dx, dtype=dtype,
                layout=layout, pairing=pairing, given=given, strided=strided, t0=t0)


def listed():
    return [
        # One token at the model width (32 heads x 128): the smallest call, launch latency alone.
        _norm("norm 1x4096 bf16", "norm", 1, 1, 4096, "bf16"),
        # The norm in front of the attention of a 768p, 14.4 s clip (45 frames x 1008 tokens).
        _norm("norm 45360x4096 bf16", "norm", 45360, 1, 4096, "bf16", w="bf16"),
        # Its backward.
        _norm("norm_bwd 45360x4096 bf16", "norm_bwd", 45360, 1, 4096, "bf16", w="bf16"),
        # Per-head norm of Q inside a fused Q, K, V projection (token stride of three tensors): narrow rows.
        _norm("norm_bwd 45360x32x128 bf16 strided", "norm_bwd", 45360, 32, 128, "bf16", strided=True),
        # An odd width in float32: nothing is 16-byte aligned but the tensors' starts.
        _norm("norm_bwd 4097x1001 f32", "norm_bwd", 4097, 1, 1001, "f32"),
        # Training with 8-bit activations, 16 frames: the forward that keeps the normalised rows ...
        _norm("norm_ckpt 16128x4096 bf16", "norm_ckpt", 16128, 1, 4096, "bf16"),
        # ... and the backward that works from them (45 frames).
        _norm("norm_bwd_ckpt 45360x4096 bf16", "norm_bwd_ckpt", 45360, 1, 4096, "bf16"),
        # Q and K of the 768p clip (24 x 42 grid), heads inside tokens: the largest.
        _rope("rope 768p 32 heads bf16", "rope", 1, 45, 24, 42, 32, 32, 128, 44, 42, 42, "bf16", "btnhd", "interleaved"),
        # A packed sequence with a position per token (images of several sizes), fewer K heads, odd length.
        _rope("rope packed 8191 16/4 heads bf16", "rope", 1, 1, 1, 8191, 16, 4, 128, 32, 48, 48, "bf16", "btnhd", "halves",
              given=True),
        # A small clip in float32, heads outside tokens: gradients, far along in a long video.
        _rope("rope_bwd 2x4x5x7x9x64 f32", "rope_bwd", 2, 5, 7, 9, 4, 4, 64, 16, 24, 24, "f32", "bhtnd", "interleaved",
              t0=1.0e5),
        # Keys of the 768p clip kept in 8 bits for the backward.
        dict(name="pack 1451520x128 bf16", op="pack", rows=45 * 1008 * 32, D=128, dtype="bf16"),
        # A small ragged float32 tensor: rows that end inside a block.
        dict(name="pack 257x1001 f32", op="pack", rows=257, D=1001, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_ckpt", "norm_bwd", "norm_bwd", "norm_bwd_ckpt", "rope", "rope", "rope_bwd", "pack"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    es = 2 if dtype == "bf16" else 4
    if op.startswith("norm"):
        D = _log_int(rng, 16, 8192)
        if rng.random() < 0.7:
            D = max(16, D // 16 * 16)
        heads = rng.choice([1, 2, 8, 32]) if D <= 256 else 1
        most = max(1, min(45360, _MOST_BYTES // (4 * es * heads * D)))
        tokens = _log_int(rng, 1, most)
        return dict(op=op, tokens=tokens, heads=heads, D=D, dtype=dtype, w=rng.choice(["f32", dtype]),
                    strided=rng.random() < 0.3, affine=rng.random() < 0.9)
    if op.startswith("rope"):
        d = rng.choice([32, 48, 64, 72, 80, 96, 120, 128])
        dt = 2 * rng.randint(0, d // 4)
        dy = 2 * rng.randint(0, (d - dt) // 4)
        dx = 2 * rng.randint(1, max(1, (d - dt - dy) // 2))
        gh, gw = rng.randint(1, 32), rng.randint(1, 48)
        hq = rng.choice([1, 4, 8, 16, 32])
        hk = rng.choice([h for h in (1, 2, 4, 8, 16, 32) if hq % h == 0])
        B = rng.choice([1, 1, 2])
        most = max(1, _MOST_BYTES // (2 * es * B * gh * gw * (hq + hk) * d))
        layout = rng.choice(["btnhd", "bhtnd"])
        return dict(op=op, B=B, T=_log_int(rng, 1, min(90, most)), gh=gh, gw=gw, hq=hq, hk=hk, d=d, dt=dt, dy=dy, dx=dx,
                    dtype=dtype, layout=layout, pairing=rng.choice(["interleaved", "halves"]),
                    given=rng.random() < 0.4, strided=layout == "btnhd" and rng.random() < 0.4,
                    t0=rng.choice([0.0, 17.0, 1.0e5]))
    D = _log_int(rng, 16, 8192)
    rows = _log_int(rng, 1, max(1, min(1451520, _MOST_BYTES // (4 * es * D))))
    return dict(op=op, rows=rows, D=D, dtype=dtype)


# ---------------------------------------------------------------- 8-bit blocks, plain form
def _blocks(x):
    """Rows padded with zeros to whole blocks, as [rows, blocks, 32]."""
    D = x.shape[-1]
    x = torch.nn.functional.pad(x, (0, -D % BLOCK))
    return x.reshape(x.shape[0], -1, BLOCK)


def _to_8_bits(x32):
    """Codes (float8_e4m3fn) [rows, D] and the scales' exponents (int32) [rows, blocks] of float32 rows."""
    b = _blocks(x32)
    top = torch.where(torch.isfinite(b), b.abs(), 0.0).amax(-1)
    m, k = torch.frexp(top)                       # top = m 2^k, m in [0.5, 1)
    e = (k - 9 + (m > 0.875).to(torch.int32)).clamp(min=-127)
    e = torch.where(top == 0, -127, e)
    y = torch.ldexp(b, -e[..., None])
    # At the largest exponent 256 would stand for 2^128: the next value below is taken.
    y = torch.where((e == 120)[..., None] & torch.isfinite(y), y.clamp(-240.0, 240.0), y)
    codes = y.to(torch.float8_e4m3fn)
    return codes.reshape(x32.shape[0], -1)[:, : x32.shape[1]].contiguous(), e


def _from_8_bits(codes, e):
    """The float32 values that codes and exponents stand for."""
    v = torch.ldexp(_blocks(codes.float()), e[..., None])
    return v.reshape(codes.shape[0], -1)[:, : codes.shape[1]]


# ---------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _tokens(g, shape, dtype, stride=None):
    """A [tokens, width] activation; with a stride, a slice of a wider buffer."""
    if stride is None:
        return torch.randn(shape, device="cuda", generator=g).to(dtype)
    full = torch.randn((shape[0], stride), device="cuda", generator=g).to(dtype)
    return full[:, shape[1]: 2 * shape[1]]


def _prepare_norm(c, seed):
    g, dt, wdt = _generator(seed), _DT[c["dtype"]], _DT[c["w"]]
    tokens, heads, D = c["tokens"], c["heads"], c["D"]
    width = heads * D
    st = {"W": None, "b": None}
    # Activations with an offset per row and a few strong features, as a residual stream has.
    x = torch.randn((tokens, width), device="cuda", generator=g)
    x *= 1.0 + 9.0 * (torch.rand((width,), device="cuda", generator=g) < 0.01)
    x += 0.3 + 0.5 * torch.randn((tokens, 1), device="cuda", generator=g)
    if c["strided"]:
        full = torch.zeros((tokens, 3 * width), device="cuda", dtype=dt)
        full[:, width: 2 * width] = x.to(dt)
        st["X"] = full[:, width: 2 * width]
    else:
        st["X"] = x.to(dt)
    del x
    if c["affine"]:
        st["W"] = (1.0 + 0.1 * torch.randn((D,), device="cuda", generator=g)).to(wdt)
        st["b"] = (0.1 * torch.randn((D,), device="cuda", generator=g)).to(wdt)
    rows = tokens * heads
    f32 = dict(device="cuda", dtype=torch.float32)
    if c["op"] in ("norm", "norm_ckpt"):
        st["Y"] = torch.empty((tokens, width), device="cuda", dtype=dt)
        st["mean"], st["rstd"] = torch.empty(rows, **f32), torch.empty(rows, **f32)
    else:
        st["dY"] = torch.randn((tokens, width), device="cuda", generator=g).to(dt)
        x = st["X"].reshape(rows, D).double()
        mean = x.mean(-1, keepdim=True)
        rstd = ((x - mean).square().mean(-1, keepdim=True) + EPS).rsqrt()
        st["mean"], st["rstd"] = mean.float().reshape(-1), rstd.float().reshape(-1)
        if c["op"] == "norm_bwd_ckpt":
            st["codes"], e = _to_8_bits(((x - mean) * rstd).float())
            st["scales"] = (e + 127).to(torch.uint8)
            st["Y"] = torch.empty((tokens, width), device="cuda", dtype=dt)
            st["X"] = None
        if c["op"] == "norm_bwd" and c["strided"]:
            st["dX"] = torch.empty((tokens, 3 * width), device="cuda", dtype=dt)[:, width: 2 * width]
        else:
            st["dX"] = torch.empty((tokens, width), device="cuda", dtype=dt)
        st["dW"], st["db"] = (torch.empty(D, **f32), torch.empty(D, **f32)) if c["affine"] else (None, None)
    if c["op"] == "norm_ckpt":
        st["codes"] = torch.empty((rows, D), device="cuda", dtype=torch.float8_e4m3fn)
        st["scales"] = torch.empty((rows, -(-D // BLOCK)), device="cuda", dtype=torch.uint8)
        st["kept"] = torch.empty((rows, D), device="cuda", dtype=torch.bfloat16)
    return st


def _heads_tensor(g, c, H, dt):
    """[B, T*n, H, d] (a slice of a wider projection where strided) or [B, H, T*n, d]."""
    B, N, d = c["B"], c["T"] * c["gh"] * c["gw"], c["d"]
    if c["layout"] == "bhtnd":
        return torch.randn((B, H, N, d), device="cuda", generator=g).to(dt)
    if c["strided"]:
        full = torch.randn((B, N, H * d + 256), device="cuda", generator=g).to(dt)
        return full[:, :, 128: 128 + H * d].unflatten(2, (H, d))
    return torch.randn((B, N, H, d), device="cuda", generator=g).to(dt)


def _prepare_rope(c, seed):
    g, dt = _generator(seed), _DT[c["dtype"]]
    st = {"Q": _heads_tensor(g, c, c["hq"], dt), "K": _heads_tensor(g, c, c["hk"], dt), "positions": None}
    if c["given"]:
        # Images of 16 to 64 patches a side, one after the other, each with a time of its own.
        N = c["T"] * c["gh"] * c["gw"]
        at = torch.arange(N, device="cuda").expand(c["B"], N)
        side = 16 + torch.randint(0, 49, (c["B"], 1), device="cuda", generator=g)
        area = side * side
        st["positions"] = torch.stack((at // area + c["t0"], at % area // side, at % side), -1).float().contiguous()
    B, N, d = c["B"], c["T"] * c["gh"] * c["gw"], c["d"]
    shape = (lambda H: (B, H, N, d)) if c["layout"] == "bhtnd" else (lambda H: (B, N, H, d))
    st["Qo"] = torch.empty(shape(c["hq"]), device="cuda", dtype=dt)
    st["Ko"] = torch.empty(shape(c["hk"]), device="cuda", dtype=dt)
    return st


def prepare(case, seed):
    c = case
    if c["op"].startswith("norm"):
        st = _prepare_norm(c, seed)
    elif c["op"].startswith("rope"):
        st = _prepare_rope(c, seed)
    else:
        g, dt = _generator(seed), _DT[c["dtype"]]
        x = torch.randn((c["rows"], c["D"]), device="cuda", generator=g)
        x *= torch.exp(2.0 * torch.randn((c["rows"], 1), device="cuda", generator=g))   # rows of unlike size
        st = {"X": x.to(dt), "back": torch.empty((c["rows"], c["D"]), device="cuda", dtype=dt),
              "codes": torch.empty((c["rows"], c["D"]), device="cuda", dtype=torch.float8_e4m3fn),
              "scales": torch.empty((c["rows"], -(-c["D"] // BLOCK)), device="cuda", dtype=torch.uint8)}
    st["case"] = dict(c)
    return st


# ---------------------------------------------------------------- plain forms
def _plain_norm(c, st):
    dt, D = _DT[c["dtype"]], c["D"]
    w = st["W"].float() if c["affine"] else 1.0
    b = st["b"].float() if c["affine"] else 0.0
    if c["op"] in ("norm", "norm_ckpt"):
        x = st["X"].float().reshape(-1, D)
        mean = x.sum(-1, keepdim=True) / D
        x = x - mean
        rstd = 1.0 / torch.sqrt(x.square().sum(-1, keepdim=True) / D + EPS)
        xh = x * rstd
        y = (xh * w + b).to(dt).reshape(c["tokens"], -1)
        out = {"Y": y, "mean": mean.reshape(-1), "rstd": rstd.reshape(-1)}
        if c["op"] == "norm_ckpt":
            out["kept"] = _from_8_bits(*_to_8_bits(xh)).to(torch.bfloat16)
        return out
    out = {}
    rstd = st["rstd"][:, None]
    if c["op"] == "norm_bwd":
        xh = (st["X"].float().reshape(-1, D) - st["mean"][:, None]) * rstd
    else:
        xh = _from_8_bits(st["codes"], st["scales"].to(torch.int32) - 127)
        out["Y"] = (xh * w + b).to(dt).reshape(c["tokens"], -1)
    dy = st["dY"].float().reshape(-1, D)
    if c["affine"]:
        out["dW"], out["db"] = (dy * xh).sum(0), dy.sum(0)
    gr = dy * w
    dx = rstd * (gr - gr.sum(-1, keepdim=True) / D - xh * ((gr * xh).sum(-1, keepdim=True) / D))
    out["dX"] = dx.to(dt).reshape(c["tokens"], -1)
    return out


def _grid(c):
    """Positions (time, height, width) of the grid's tokens, 64 bits."""
    t, y, x = (torch.arange(n, device="cuda", dtype=torch.float64) for n in (c["T"], c["gh"], c["gw"]))
    return torch.stack(torch.meshgrid(t + c["t0"], y, x, indexing="ij"), -1).reshape(1, -1, 3)


def _frequencies(c, like):
    """[d_rot / 2] angular frequencies, and the axis of each pair."""
    fs = [THETA ** (-2.0 * torch.arange(n // 2, device=like.device, dtype=torch.float64) / max(n, 1))
          for n in (c["dt"], c["dy"], c["dx"])]
    axis = torch.cat([torch.full_like(f, i).long() for i, f in enumerate(fs)])
    return torch.cat(fs), axis


def _plain_rope(c, st):
    pos = st["positions"].double() if c["given"] else _grid(c)
    f, axis = _frequencies(c, pos)
    ang = pos[..., axis] * f                                       # [B or 1, N, pairs]
    ang = ang[:, :, None] if c["layout"] == "btnhd" else ang[:, None]
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    if c["op"] == "rope_bwd":
        sin = -sin
    rot = c["dt"] + c["dy"] + c["dx"]

    def turn(x):
        v = x[..., :rot].float()
        if c["pairing"] == "interleaved":
            a, b = v[..., 0::2], v[..., 1::2]
            out = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
        else:
            a, b = v[..., : rot // 2], v[..., rot // 2:]
            out = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        return torch.cat((out.to(x.dtype), x[..., rot:]), -1)

    return {"Q": turn(st["Q"]), "K": turn(st["K"])}


# ---------------------------------------------------------------- the library's calls
def _own_norm(c, st):
    from frame_wise_linear_b200 import vda
    dt = {"bf16": vda.VDA_DTYPE_BF16, "f32": vda.VDA_DTYPE_F32}
    out_strided = c["strided"] and c["op"] == "norm_bwd"
    p = vda.make_norm_problem(c["tokens"], c["D"], dt[c["dtype"]], heads=c["heads"], w_dtype=dt[c["w"]], eps=EPS,
                              ld_x=st["X"].stride(0) if c["op"] in ("norm", "norm_ckpt") or out_strided else 0)
    if c["op"] == "norm":
        vda.vda_layer_norm(p, st["X"], st["W"], st["b"], st["Y"], st["mean"], st["rstd"])
        return {k: st[k] for k in ("Y", "mean", "rstd")}
    if c["op"] == "norm_ckpt":
        vda.vda_layer_norm(p, st["X"], st["W"], st["b"], st["Y"], st["mean"], st["rstd"], st["codes"], st["scales"])
        back = vda.make_checkpoint_problem(c["tokens"] * c["heads"], c["D"], vda.VDA_DTYPE_BF16)
        vda.vda_checkpoint_unpack(back, st["codes"], st["scales"], st["kept"])
        return {k: st[k] for k in ("Y", "mean", "rstd", "kept")}
    if "ws" not in st:
        st["ws"] = torch.empty(vda.vda_layer_norm_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
    out = {"dX": st["dX"]}
    if c["affine"]:
        out["dW"], out["db"] = st["dW"], st["db"]
    if c["op"] == "norm_bwd":
        vda.vda_layer_norm_backward(p, st["dY"], st["X"], st["mean"], st["rstd"], st["W"], st["dX"], st["dW"], st["db"],
                                    st["ws"])
        return out
    vda.vda_layer_norm_from_checkpoint(p, st["codes"], st["scales"], st["W"], st["b"], st["Y"])
    vda.vda_layer_norm_backward_from_checkpoint(p, st["dY"], st["codes"], st["scales"], st["rstd"], st["W"], st["dX"],
                                                st["dW"], st["db"], st["ws"])
    out["Y"] = st["Y"]
    return out


def _own_rope(c, st):
    from frame_wise_linear_b200 import vda
    strided = c["strided"]
    p = vda.make_rope_problem(
        c["B"], c["T"], c["gh"], c["gw"], c["hq"], c["hk"], c["d"], (c["dt"], c["dy"], c["dx"]),
        {"bf16": vda.VDA_DTYPE_BF16, "f32": vda.VDA_DTYPE_F32}[c["dtype"]],
        layout={"btnhd": vda.VDA_LAYOUT_BTNHD, "bhtnd": vda.VDA_LAYOUT_BHTND}[c["layout"]],
        pairing={"interleaved": vda.VDA_ROPE_INTERLEAVED, "halves": vda.VDA_ROPE_HALVES}[c["pairing"]],
        theta=THETA, pos0=(c["t0"], 0.0, 0.0),
        **({("ld_qr" if c["op"] == "rope_bwd" else "ld_q"): st["Q"].stride(1),
            ("ld_kr" if c["op"] == "rope_bwd" else "ld_k"): st["K"].stride(1)} if strided else {}))
    call = vda.vda_rope_backward if c["op"] == "rope_bwd" else vda.vda_rope
    call(p, st["Q"], st["K"], st["positions"], st["Qo"], st["Ko"])
    return {"Q": st["Qo"], "K": st["Ko"]}


def _own_pack(c, st):
    from frame_wise_linear_b200 import vda
    p = vda.make_checkpoint_problem(c["rows"], c["D"], {"bf16": vda.VDA_DTYPE_BF16, "f32": vda.VDA_DTYPE_F32}[c["dtype"]])
    vda.vda_checkpoint_pack(p, st["X"], st["codes"], st["scales"])
    vda.vda_checkpoint_unpack(p, st["codes"], st["scales"], st["back"])
    return {"back": st["back"]}


def run(state):
    c = state["case"]
    if c["op"].startswith("norm"):
        return _own_norm(c, state) if own else _plain_norm(c, state)
    if c["op"].startswith("rope"):
        return _own_rope(c, state) if own else _plain_rope(c, state)
    if own:
        return _own_pack(c, state)
    return {"back": _from_8_bits(*_to_8_bits(state["X"].float())).to(_DT[c["dtype"]])}


# ---------------------------------------------------------------- what cannot be done without
def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"].startswith("norm"):
        rows, D = c["tokens"] * c["heads"], c["D"]
        n, ws = rows * D, (2 if c["w"] == "bf16" else 4) * D if c["affine"] else 0
        kept = n + rows * -(-D // BLOCK)
        if c["op"] == "norm":
            return {"bytes": 2 * es * n + 8 * rows + 2 * ws, "flops": 8 * n}
        if c["op"] == "norm_ckpt":   # the codes are written, and read once for the values that are returned
            return {"bytes": 2 * es * n + 8 * rows + 2 * ws + 2 * kept + 2 * n, "flops": 14 * n}
        grads = 8 * D if c["affine"] else 0
        if c["op"] == "norm_bwd":
            return {"bytes": 3 * es * n + 8 * rows + ws + grads, "flops": 14 * n}
        return {"bytes": 3 * es * n + kept + 4 * rows + 2 * ws + grads, "flops": 16 * n}
    if c["op"].startswith("rope"):
        N = c["B"] * c["T"] * c["gh"] * c["gw"]
        n = N * (c["hq"] + c["hk"]) * c["d"]
        return {"bytes": 2 * es * n + (12 * N if c["given"] else 0), "flops": 3 * n}
    n = c["rows"] * c["D"]
    return {"bytes": 2 * es * n + 2 * (n + c["rows"] * -(-c["D"] // BLOCK)), "flops": 5 * n}


# ---------------------------------------------------------------- 64 bits
def _exact_8_bits(x):
    """The values that the 8-bit blocks of float64 rows stand for, from the format's definition: the least
    power of two 2^e (e >= -127) whose 448-fold covers the block's largest finite value, and the nearest
    multiple of the format's step there, ties to even."""
    out = torch.empty_like(x)
    D = x.shape[1]
    full = D - D % BLOCK
    for part, shape in ((slice(0, full), (-1, BLOCK)), (slice(full, D), (-1, max(1, D - full)))):
        v = x[:, part]
        if v.numel() == 0:
            continue
        v = v.reshape(shape)
        top = torch.nan_to_num(v, nan=0.0, posinf=0.0, neginf=0.0).abs().max(1, keepdim=True).values
        e = torch.ceil(torch.log2(top / 448.0)).clamp(min=-127.0)
        s = torch.exp2(e)
        y = v / s
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3.0)
        y = torch.round(y / step) * step
        y = torch.where(e == 120.0, y.clamp(-240.0, 240.0), y)
        out[:, part] = (y * s).reshape(x.shape[0], -1)
    return out


def _exact_norm(c, st):
    D = c["D"]
    one = torch.ones((D,), device="cuda", dtype=torch.float64)
    w, b = (st["W"].double(), st["b"].double()) if c["affine"] else (one, 0 * one)
    if c["op"] in ("norm", "norm_ckpt"):
        x = st["X"].reshape(-1, D).double()
        mean = torch.mv(x, one) / D
        rstd = (((x - mean[:, None]) ** 2).mean(1) + EPS) ** -0.5
        xh = (x - mean[:, None]) * rstd[:, None]
        out = {"mean": mean, "rstd": rstd, "Y": torch.addcmul(b, xh, w).reshape(c["tokens"], -1)}
        if c["op"] == "norm_ckpt":
            out["kept"] = _exact_8_bits(xh)
        return out
    out = {}
    if c["op"] == "norm_bwd":
        xh = (st["X"].reshape(-1, D).double() - st["mean"].double()[:, None]) * st["rstd"].double()[:, None]
    else:
        scale = torch.exp2(st["scales"].double() - 127.0).repeat_interleave(BLOCK, dim=1)[:, :D]
        xh = st["codes"].double() * scale
        out["Y"] = torch.addcmul(b, xh, w).reshape(c["tokens"], -1)
    dy = st["dY"].reshape(-1, D).double()
    if c["affine"]:
        out["dW"], out["db"] = torch.einsum("rd,rd->d", dy, xh), torch.einsum("rd->d", dy)
    # dx = rstd (I - (1 1' + xh xh') / D) (w dy): the projection, then the scale.
    along, mean = torch.einsum("rd,rd,d->r", dy, xh, w) / D, torch.mv(dy, w) / D
    dx = (dy * w - mean[:, None] - along[:, None] * xh) * st["rstd"].double()[:, None]
    out["dX"] = dx.reshape(c["tokens"], -1)
    return out


def _exact_rope(c, st):
    """Each pair as a complex number times e^(i angle)."""
    if c["given"]:
        pos = st["positions"].double()
    else:
        at = torch.arange(c["T"] * c["gh"] * c["gw"], device="cuda")
        pos = torch.stack(((at // (c["gh"] * c["gw"])).double() + c["t0"], (at // c["gw"] % c["gh"]).double(),
                           (at % c["gw"]).double()), -1)[None]
    parts = []
    for i, n in enumerate((c["dt"], c["dy"], c["dx"])):
        j = torch.arange(n // 2, device="cuda", dtype=torch.float64)
        parts.append(pos[..., i: i + 1] * torch.exp(-math.log(THETA) * 2.0 * j / max(n, 1)))
    ang = torch.cat(parts, -1)
    turn = torch.polar(torch.ones_like(ang), -ang if c["op"] == "rope_bwd" else ang)
    turn = turn.unsqueeze(2 if c["layout"] == "btnhd" else 1)
    rot = c["dt"] + c["dy"] + c["dx"]
    out = {}
    for k in ("Q", "K"):
        x = st[k].double()
        v = x[..., :rot]
        v = v.unflatten(-1, (-1, 2)) if c["pairing"] == "interleaved" else v.unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(v.contiguous()) * turn)
        z = z if c["pairing"] == "interleaved" else z.transpose(-1, -2)
        out[k] = torch.cat((z.flatten(-2), x[..., rot:]), -1)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(case, st)
    if case["op"].startswith("rope"):
        return _exact_rope(case, st)
    return {"back": _exact_8_bits(st["X"].double())}
