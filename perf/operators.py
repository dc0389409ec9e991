"""Cases of five operators of the MoE block, in plain torch and as the library's calls.

  few    the whole MoE layer for 1 to 16 tokens (moe_layer_forward_few)
  pack   expert weights to microscaled 4-bit floating point and back
         (moe_mx_pack_weights, moe_mx_unpack_weights)
  ffn    the ragged grouped SwiGLU experts on microscaled 4-bit rows and weights (moe_grouped_ffn)
  norm   leaving a block and entering the next: post-norm, gate, residual scale, residual add, next
         block's pre-norm (moe_block_norm)
  block  a whole block around the residual stream: pre-norm, layer, exit (moe_block_forward)

Microscaled 4-bit values: 32 consecutive values of a row share one power of two
2^(floor(log2(amax)) - 2); each is rounded to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 times it
(ties to the even code, larger values to 6).
"""

import math

import torch

own = False

DEV = "cuda"
MX_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _few(name, T, D, E, k, I, shared, w, begin=0, local=None, given=False):
    return {"name": name, "op": "few", "T": T, "D": D, "E": E, "k": k, "I": I, "shared": shared, "w": w,
            "begin": begin, "local": E if local is None else local, "given": given}


def _block(name, T, D, E, k, I, shared, w, gate, post):
    return {**_few(name, T, D, E, k, I, shared, w), "op": "block", "gate": gate, "post": post}


def listed():
    return [
        # one request's next token through the 512-expert layer: the weight stream of 11 experts
        _few("few_one_bf16", 1, 4096, 512, 10, 1024, 1024, "bf16"),
        # a handful of requests on 4-bit experts, bf16 shared expert
        _few("few_four_mx", 4, 4096, 128, 8, 1024, 1024, "mxfp4"),
        # 13 requests' tokens at one device's share of an expert-parallel layer, e4m3 experts, routing given
        _few("few_share_fp8", 13, 4096, 512, 10, 1024, 0, "e4m3", begin=64, local=64, given=True),
        # one attention projection's worth of weights to 4 bits and back
        {"name": "pack_one", "op": "pack", "n": 1, "rows": 1024, "cols": 4096, "src": "bf16"},
        # one device's 64 experts' gate matrices, once at load time
        {"name": "pack_experts", "op": "pack", "n": 64, "rows": 1024, "cols": 4096, "src": "bf16"},
        # a decode batch on one device's experts: about 10 rows each
        {"name": "ffn_decode", "op": "ffn", "T": 64, "D": 4096, "n": 64, "k": 10, "I": 1024, "skew": 0.0},
        # a prefill chunk: about 160 rows each
        {"name": "ffn_prefill", "op": "ffn", "T": 1024, "D": 4096, "n": 64, "k": 10, "I": 1024, "skew": 0.0},
        # widths that end inside a 128-value slice, popular and empty experts
        {"name": "ffn_ragged", "op": "ffn", "T": 333, "D": 704, "n": 24, "k": 3, "I": 320, "skew": 2.0},
        # one token between two blocks: launch latency
        {"name": "norm_one", "op": "norm", "T": 1, "D": 4096, "dtype": "bf16", "gate": "channel", "post": True,
         "next": True},
        # a prefill chunk between two blocks, a gate of its own for every value
        {"name": "norm_prefill", "op": "norm", "T": 8192, "D": 4096, "dtype": "bf16", "gate": "full", "post": True,
         "next": True},
        # the tiny fp32 block: three tokens, latency only
        _block("block_tiny_fp32", 3, 256, 16, 2, 128, 128, "f32", "token", True),
        # a block over a medium batch in bf16
        _block("block_batch_bf16", 200, 1024, 32, 4, 512, 512, "bf16", "channel", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    return 64 * max(1, round(_log(rng, lo, hi) / 64))


def draw(rng):
    op = rng.choice(["few", "few", "pack", "ffn", "ffn", "norm", "block"])
    if op == "pack":
        return {"op": "pack", "n": _log(rng, 1, 32), "rows": 16 * _log(rng, 1, 64), "cols": _width(rng, 64, 4096),
                "src": rng.choice(["bf16", "f32"])}
    if op == "ffn":
        n = _log(rng, 1, 64)
        return {"op": "ffn", "T": _log(rng, 1, 1000), "D": _width(rng, 64, 4096), "n": n,
                "k": rng.randint(1, min(10, n)), "I": _width(rng, 64, 1024), "skew": rng.choice([0.0, 1.0, 3.0])}
    if op == "norm":
        return {"op": "norm", "T": _log(rng, 1, 8192), "D": _log(rng, 1, 4096), "dtype": rng.choice(["bf16", "f32"]),
                "gate": rng.choice(["none", "token", "channel", "full"]), "post": rng.random() < 0.6,
                "next": rng.random() < 0.8}
    E = _log(rng, 4, 256)
    k = rng.randint(1, min(10, E))
    D, I = _width(rng, 64, 4096), _width(rng, 64, 1024)
    w = rng.choice(["bf16", "e4m3", "mxfp4", "f32"])
    shared = rng.choice([0, I, _width(rng, 64, 1024)])
    if op == "block":
        # the 4-bit layer keeps its hidden states in bf16 up to 16 tokens; 8-bit and longer 4-bit batches round them
        T, w = _log(rng, 1, 16 if w == "mxfp4" else 256), "bf16" if w == "e4m3" else w
        c = _block("", T, D, min(E, 64), min(k, 8), I, shared, w, rng.choice(["none", "token", "channel", "full"]),
                   rng.random() < 0.5)
        del c["name"]
        return c
    c = _few("", rng.randint(1, 16), D, E, k, I, shared, w)
    del c["name"]
    if rng.random() < 0.3:
        c["local"] = rng.randint(1, E)
        c["begin"] = rng.randint(0, E - c["local"])
        c["given"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed, what):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1009 + what)
    return g


def _randn(seed, what, shape, std=1.0):
    return torch.randn(shape, generator=_gen(seed, what), device=DEV, dtype=torch.float32).mul_(std)


def _torch_dtype(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _mx_encode(v):
    """[..., K] float32, K a multiple of 64 -> (codes [..., K] uint8 0..15, scale exponents [..., K / 32] int32)."""
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    amax = b.abs().amax(-1)
    e = (torch.frexp(amax)[1] - 3).clamp(-126, 127)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    a = torch.ldexp(b.abs(), -e[..., None])
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    r = (torch.round(a / step) * step).clamp_max(6.0)
    code = torch.where(r < 2, r * 2, torch.where(r < 4, r + 2, r / 2 + 4)).to(torch.uint8)
    code |= (torch.signbit(b)).to(torch.uint8) << 3
    return code.reshape(v.shape), e


def _mx_decode(codes, exps):
    """Float32 values of codes [..., K] with block exponents [..., K / 32]."""
    lut = torch.tensor(MX_LEVELS + tuple(-x for x in MX_LEVELS), device=codes.device)
    v = lut[codes.long()].reshape(*exps.shape, 32)
    return torch.ldexp(v, exps[..., None]).reshape(codes.shape)


def _mx_image(codes, exps):
    """The library's storage of [n][rows][K] 4-bit weights: for each 16 rows and each 512 values of the
    reduction dimension up to four 1 KB runs (one per 128 values: 16 bytes of row l % 16 for lane l, its 32
    values at (l / 16) * 32), then 256 bytes of scales (lane l: the four runs' scale bytes)."""
    n, R, K = codes.shape
    S = -(-K // 128)
    G = -(-S // 4)
    c = torch.zeros(n, R, S * 128, dtype=torch.uint8, device=codes.device)
    c[..., :K] = codes
    c = c[..., 0::2] | (c[..., 1::2] << 4)
    c = c.reshape(n, R // 16, 16, S, 4, 16).permute(0, 1, 3, 4, 2, 5).reshape(n, R // 16, S, 1024)
    s = torch.full((n, R, G * 16), 127, dtype=torch.uint8, device=codes.device)
    s[..., :K // 32] = (exps + 127).to(torch.uint8)
    s = s.reshape(n, R // 16, 16, G, 4, 4).permute(0, 1, 3, 5, 2, 4).reshape(n, R // 16, G, 256)
    q = S // 4
    parts = [torch.cat([c[:, :, :4 * q].reshape(n, R // 16, q, 4096), s[:, :, :q]], -1).reshape(n, R // 16, -1)]
    if S % 4:
        parts += [c[:, :, 4 * q:].reshape(n, R // 16, -1), s[:, :, q]]
    return torch.cat(parts, -1).reshape(n, -1)


def _runs(w):
    """[n][rows][cols] weights in the library's fragment-major order."""
    n, R, K = w.shape
    b = w.view(torch.uint8).reshape(n, R // 16, 16, -1, 4, 16)
    return b.permute(0, 1, 3, 4, 2, 5).reshape(n, R, -1).view(w.dtype)


def _weights(seed, what, n, rows, cols, kind):
    """n matrices [rows][cols] ~ N(0, 1 / cols) as a user's program holds them: the row-major form (`rows`,
    with scales) and the library's laid-out form (`laid`)."""
    step = max(1, (1 << 27) // (rows * cols))
    rows_, laid, scales = [], [], []
    for i in range(0, n, step):
        m = min(step, n - i)
        z = _randn(seed, what * 4096 + i, (m, rows, cols), cols ** -0.5)
        if kind == "mxfp4":
            c, e = _mx_encode(z)
            rows_.append(c[..., 0::2] | (c[..., 1::2] << 4))
            scales.append(e.to(torch.int8))
            laid.append(_mx_image(c, e))
            continue
        if kind == "e4m3":
            amax = z.abs().amax(-1, keepdim=True).clamp_min(1e-30)
            scales.append((amax[..., 0] / 448).float())
            z = (z * (448 / amax)).clamp(-448, 448).to(torch.float8_e4m3fn)
        else:
            z = z.to(_torch_dtype(kind))
        rows_.append(z)
        laid.append(_runs(z))
    cat = lambda v: (v[0] if len(v) == 1 else torch.cat(v)) if v else None  # noqa: E731
    return {"rows": cat(rows_), "laid": cat(laid), "scale": cat(scales), "kind": kind}


def _values(w, at=None):
    """Float32 values of the matrices (or of those at `at`), from the row-major form."""
    r = w["rows"] if at is None else w["rows"][at]
    s = None if w["scale"] is None else w["scale"] if at is None else w["scale"][at]
    if w["kind"] == "mxfp4":
        c = torch.stack([r & 15, r >> 4], -1).reshape(*r.shape[:-1], -1)
        return _mx_decode(c, s.int())
    return r.float() if s is None else r.float() * s[..., None]


def _layer_state(c, seed):
    act = _torch_dtype("f32" if c["w"] == "f32" else "bf16")
    T, D, E, k, I, n, Is = (c[x] for x in ("T", "D", "E", "k", "I", "local", "shared"))
    s = {"case": c, "x": _randn(seed, 1, (T, D)).to(act),
         "router": None if c["given"] else _randn(seed, 2, (E, D), D ** -0.5).to(act),
         "gate_w": _weights(seed, 3, n, I, D, c["w"]), "up_w": _weights(seed, 4, n, I, D, c["w"]),
         "down_w": _weights(seed, 5, n, D, I, c["w"]), "packed": None}
    plain = "f32" if c["w"] == "f32" else "bf16"
    if Is:
        s["sh"] = [_weights(seed, 6, 1, Is, D, plain), _weights(seed, 7, 1, Is, D, plain),
                   _weights(seed, 8, 1, D, Is, plain)]
    if c["given"]:
        ids = torch.rand((T, E), generator=_gen(seed, 9), device=DEV).argsort(1)[:, :k].int()
        wt = -torch.rand((T, k), generator=_gen(seed, 10), device=DEV).clamp_min(1e-6).log()
        wt = (wt / wt.sum(1, keepdim=True)).sort(1, descending=True)[0]
        s["packed"] = torch.stack([ids, wt.view(torch.int32)], 1).contiguous()
    s["y"] = torch.empty(T, D, dtype=act, device=DEV)
    s["ws"] = torch.empty(_workspace_bound(c), dtype=torch.uint8, device=DEV)
    return s


def _workspace_bound(c):
    """More scratch than the layer needs for a case of these ranges."""
    pairs = c["T"] * c["k"]
    return (64 << 20) + pairs * (c["D"] + c["I"]) * 12 + c["T"] * (c["shared"] + c["E"] * 8 + c["D"] * 4) * 8


def _norm_state(c, seed, T, D, act):
    g = c["gate"]
    shape = {"none": None, "token": (T,), "channel": (D,), "full": (T, D)}[g]
    one = lambda what: (1 + _randn(seed, what, (D,), 0.1)).to(act)  # noqa: E731
    return {"r": _randn(seed, 20, (T, D), 2.0).to(act), "w_in": one(21), "w_post": one(22) if c["post"] else None,
            "w_next": one(23), "res_scale": 0.875, "eps": 1e-6,
            "gate": None if shape is None else _randn(seed, 24, shape, 0.5).to(torch.float32 if g == "token" else act)}


def prepare(case, seed):
    if case["op"] == "few":
        return _layer_state(case, seed)
    if case["op"] == "pack":
        src = _randn(seed, 1, (case["n"], case["rows"], case["cols"]), case["cols"] ** -0.5)
        return {"case": case, "src": src.to(_torch_dtype(case["src"]))}
    if case["op"] == "ffn":
        T, D, n, k, I = (case[x] for x in ("T", "D", "n", "k", "I"))
        # popularity of the experts: a skew leaves some of them without a row
        keys = torch.rand((T, n), generator=_gen(seed, 2), device=DEV)
        keys = keys + case["skew"] * torch.rand((n,), generator=_gen(seed, 3), device=DEV)
        ids = keys.topk(k, 1)[1].reshape(-1)
        perm = torch.argsort(ids, stable=True)
        counts = torch.bincount(ids, minlength=n)
        offsets = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
        offsets[1:] = counts.cumsum(0)
        return {"case": case, "x": _randn(seed, 4, (T, D)).bfloat16(), "perm": (perm // k).int(), "offsets": offsets,
                "cap": int(counts.max()), "gate_w": _weights(seed, 5, n, I, D, "mxfp4"),
                "up_w": _weights(seed, 6, n, I, D, "mxfp4"), "down_w": _weights(seed, 7, n, D, I, "mxfp4"),
                "out": torch.empty(T * k, D, dtype=torch.bfloat16, device=DEV),
                "ws": torch.empty(_workspace_bound({**case, "E": n, "shared": 0}), dtype=torch.uint8, device=DEV)}
    if case["op"] == "norm":
        T, D, act = case["T"], case["D"], _torch_dtype(case["dtype"])
        s = _norm_state(case, seed, T, D, act)
        return {**s, "case": case, "y": _randn(seed, 25, (T, D)).to(act),
                "r_out": torch.empty(T, D, dtype=act, device=DEV), "x_next": torch.empty(T, D, dtype=act, device=DEV)}
    s = _layer_state(case, seed)
    return {**s, **_norm_state(case, seed, case["T"], case["D"], s["x"].dtype), "r_out": torch.empty_like(s["x"]),
            "x_next": torch.empty_like(s["x"])}


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _silu(z):
    return z / (1 + torch.exp(-z))


def _route(s, x):
    """ids [T][k] (larger key first, ties to the lower id) and weights over the kept keys."""
    k = s["case"]["k"]
    if s["packed"] is not None:
        return s["packed"][:, 0].long(), s["packed"][:, 1].contiguous().view(torch.float32)
    key = x.double() @ s["router"].double().t()
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    w = torch.exp(top[:, :k] - top[:, :1])
    return ids[:, :k], (w / w.sum(1, keepdim=True)).float()


def _plain_layer(s, x):
    c = s["case"]
    x = x.float()
    ids, w = _route(s, x)
    local = ids - c["begin"]
    here = (local >= 0) & (local < c["local"])
    local = local.clamp(0, c["local"] - 1)
    w = torch.where(here, w, 0.0)
    T, k = ids.shape
    if T * k < c["local"]:
        # each token's own experts
        at = local.reshape(-1)
        xp = x.repeat_interleave(k, 0)[..., None]
        h = _silu(torch.bmm(_values(s["gate_w"], at), xp)) * torch.bmm(_values(s["up_w"], at), xp)
        o = torch.bmm(_values(s["down_w"], at), h).reshape(T, k, -1)
        y = torch.where(here[..., None], w[..., None] * o, 0.0).sum(1)
    else:
        # every expert on every token, weighted by the routing
        full = torch.zeros(T, c["local"], device=x.device).scatter_add_(1, local, w)
        xe = x[None].expand(c["local"], -1, -1)
        h = _silu(torch.bmm(xe, _values(s["gate_w"]).transpose(1, 2))) * torch.bmm(xe, _values(s["up_w"]).transpose(1, 2))
        y = torch.bmm(h * full.t()[..., None], _values(s["down_w"]).transpose(1, 2)).sum(0)
    if c["shared"]:
        g, u, d = (_values(m)[0] for m in s["sh"])
        y = y + (_silu(x @ g.t()) * (x @ u.t())) @ d.t()
    return y


def _rms(v, w, eps):
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + eps) * w.float()


def _plain_exit(s, y, r):
    z = y if s["w_post"] is None else _rms(y, s["w_post"], s["eps"])
    g = s["gate"]
    if g is not None:
        z = z * (g.float()[:, None] if g.dim() == 1 and s["case"]["gate"] == "token" else g.float())
    return s["res_scale"] * r + z


def _plain(s):
    c = s["case"]
    if c["op"] == "few":
        return {"y": _plain_layer(s, s["x"]).to(s["x"].dtype)}
    if c["op"] == "pack":
        return {"values": _mx_decode(*_mx_encode(s["src"].float())).to(torch.bfloat16)}
    if c["op"] == "ffn":
        off = s["offsets"].long()
        rows = torch.arange(s["perm"].numel(), device=DEV)
        grp = torch.searchsorted(off[1:], rows, right=True)
        pos = rows - off[grp]
        at = (off[:-1, None] + torch.arange(s["cap"], device=DEV)).clamp_max(rows.numel() - 1)
        a = _mx_decode(*_mx_encode(s["x"].float()))[s["perm"].long()[at]]
        h = _silu(torch.bmm(a, _values(s["gate_w"]).transpose(1, 2))) * torch.bmm(a, _values(s["up_w"]).transpose(1, 2))
        o = torch.bmm(_mx_decode(*_mx_encode(h)), _values(s["down_w"]).transpose(1, 2))
        return {"rows": o[grp, pos].to(torch.bfloat16)}
    r = s["r"].float()
    if c["op"] == "norm":
        out = _plain_exit(s, s["y"].float(), r)
        to = s["r"].dtype
        return {"r": out.to(to)} | ({"x": _rms(out, s["w_next"], s["eps"]).to(to)} if c["next"] else {})
    x = _rms(r, s["w_in"], s["eps"]).to(s["r"].dtype)
    out = _plain_exit(s, _plain_layer(s, x), r)
    return {"r": out.to(x.dtype), "x": _rms(out, s["w_next"], s["eps"]).to(x.dtype)}


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------

def _own_dims(moe, c, w, local, begin, shared):
    act = "f32" if w == "f32" else "bf16"
    return moe.make_dims(c["T"], c["D"], c["E"] if "E" in c else c["n"], c["k"], c["I"], shared, begin, local, True, act,
                         w, act, "packed")


def _own(s):
    import sparse_moe_ffn_route_amd as moe

    c = s["case"]
    if c["op"] == "pack":
        image = moe.moe_mx_pack_weights(s["src"])
        return {"values": moe.moe_mx_unpack_weights(image, c["rows"], c["cols"])}
    if c["op"] == "norm":
        x_next = s["x_next"] if c["next"] else None
        moe.moe_block_norm(s["y"], s["r"], s["r_out"], w_post=s["w_post"], gate=s["gate"], gate_kind=c["gate"],
                           res_scale=s["res_scale"], eps=s["eps"], w_next=s["w_next"] if c["next"] else None,
                           x_next=x_next)
        return {"r": s["r_out"]} | ({"x": x_next} if c["next"] else {})
    if c["op"] == "ffn":
        d = _own_dims(moe, c, "mxfp4", c["n"], 0, 0)
        moe.moe_grouped_ffn(d, s["x"], None, s["perm"], s["offsets"], s["gate_w"]["laid"], s["up_w"]["laid"],
                            s["down_w"]["laid"], None, None, None, s["out"], s["ws"])
        return {"rows": s["out"]}
    d = _own_dims(moe, c, c["w"], c["local"], c["begin"], c["shared"])
    sh = [m["laid"] for m in s["sh"]] if c["shared"] else [None] * 3
    sc = [s[m]["scale"] if c["w"] == "e4m3" else None for m in ("gate_w", "up_w", "down_w")]
    w = moe.make_weights(s["router"], s["gate_w"]["laid"], s["up_w"]["laid"], s["down_w"]["laid"], *sc, *sh)
    if c["op"] == "few":
        moe.moe_layer_forward_few(d, w, s["x"], s["packed"], None, s["y"], ws=s["ws"])
        return {"y": s["y"]}
    moe.moe_block_forward(d, w, s["r"], s["r_out"], w_in=s["w_in"], w_post=s["w_post"], gate=s["gate"],
                          gate_kind=c["gate"], res_scale=s["res_scale"], eps=s["eps"], w_next=s["w_next"],
                          x_next=s["x_next"], ws=s["ws"])
    return {"r": s["r_out"], "x": s["x_next"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

_BYTES = {"f32": 4.0, "bf16": 2.0, "e4m3": 1.0, "mxfp4": 4.25 / 8}


def work(case):
    c = case
    if c["op"] == "pack":
        v = c["n"] * c["rows"] * c["cols"]
        return {"bytes": v * (_BYTES[c["src"]] + 2 * _BYTES["mxfp4"] + 2), "flops": 0}
    if c["op"] == "norm":
        v, es = c["T"] * c["D"], _BYTES[c["dtype"]]
        gate = {"none": 0, "token": 4 * c["T"], "channel": es * c["D"], "full": es * v}[c["gate"]]
        return {"bytes": es * v * (4 if c["next"] else 3) + gate + 2 * es * c["D"], "flops": 8 * v}
    if c["op"] == "ffn":
        used = c["n"] * (1 - (1 - c["k"] / c["n"]) ** c["T"])
        m = 3 * c["D"] * c["I"]
        return {"bytes": used * m * _BYTES["mxfp4"] + 2 * c["T"] * c["D"] * (1 + c["k"]), "flops": 2 * c["T"] * c["k"] * m}
    es = _BYTES["f32" if c["w"] == "f32" else "bf16"]
    used = c["local"] * (1 - (1 - c["k"] / c["E"]) ** c["T"])
    m, sh = 3 * c["D"] * c["I"], 3 * c["D"] * c["shared"]
    router = 0 if c["given"] else c["E"] * c["D"]
    pairs = c["T"] * c["k"] * c["local"] / c["E"]
    io = 2 if c["op"] == "few" else 3 + (c["gate"] == "full")
    return {"bytes": used * m * _BYTES[c["w"]] + (sh + router + io * c["T"] * c["D"]) * es,
            "flops": 2 * (pairs * m + c["T"] * (sh + router))}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_mx(v):
    """The values that v's rows stand for once they are held in 4 bits, by the distance to each level."""
    b = v.double().reshape(-1, 32)
    big = b.abs().amax(1)
    e = torch.where(big > 0, torch.floor(torch.log2(big.clamp_min(2.0 ** -140))), torch.full_like(big, 2.0))
    # log2 of a value just below a power of two may round up to it
    e = torch.where((big > 0) & (torch.exp2(e) > big), e - 1, e)
    unit = torch.exp2((e - 2).clamp(-126, 127))[:, None]
    a = b.abs() / unit
    code = torch.zeros_like(a)
    for low, border in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += (a > border) if low % 2 == 0 else (a >= border)
    lv = torch.tensor(MX_LEVELS, dtype=torch.float64, device=v.device)
    return (torch.sign(b) * lv[code.long()] * unit).reshape(v.shape)


def _exact_expert(x, g, u, d, quantised=False):
    z = x @ g.T
    h = z * torch.sigmoid(z) * (x @ u.T)
    return (_exact_mx(h) if quantised else h) @ d.T


def _exact_matrix(w, e):
    r = w["rows"][e]
    if w["kind"] == "mxfp4":
        v = torch.stack([r & 15, r >> 4], -1).reshape(r.shape[0], -1).long()
        lv = torch.tensor(MX_LEVELS, dtype=torch.float64, device=r.device)[v & 7] * (1 - 2 * (v >> 3)).double()
        return lv * torch.exp2(w["scale"][e].double()).repeat_interleave(32, 1)
    return r.double() * w["scale"][e].double()[:, None] if w["kind"] == "e4m3" else r.double()


def _exact_layer(s, x):
    c = s["case"]
    if s["packed"] is not None:
        ids, wt = s["packed"][:, 0], s["packed"][:, 1].contiguous().view(torch.float32).double()
    else:
        logits = x @ s["router"].double().T
        order = torch.argsort(-logits, dim=1, stable=True)[:, :c["k"]]
        ids, wt = order, torch.softmax(torch.gather(logits, 1, order), 1)
    y = torch.zeros_like(x)
    for e in range(c["local"]):
        t, j = torch.nonzero(ids == e + c["begin"], as_tuple=True)
        if t.numel():
            o = _exact_expert(x[t], *(_exact_matrix(s[m], e) for m in ("gate_w", "up_w", "down_w")))
            y.index_add_(0, t, wt[t, j][:, None] * o)
    if c["shared"]:
        y += _exact_expert(x, *(_exact_matrix(m, 0) for m in s["sh"]))
    return y


def _exact_norm(v, w, eps):
    return v / torch.sqrt((v * v).sum(1, keepdim=True) / v.shape[1] + eps) * w.double()


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "few":
        return {"y": _exact_layer(s, s["x"].double())}
    if c["op"] == "pack":
        return {"values": _exact_mx(s["src"])}
    if c["op"] == "ffn":
        x = _exact_mx(s["x"])[s["perm"].long()]
        at = s["offsets"].tolist()
        parts = [_exact_expert(x[a:b], *(_exact_matrix(s[m], e) for m in ("gate_w", "up_w", "down_w")), quantised=True)
                 for e, (a, b) in enumerate(zip(at, at[1:])) if b > a]
        return {"rows": torch.cat(parts)}
    r = s["r"].double()
    if c["op"] == "norm":
        y = s["y"].double()
    else:
        y = _exact_layer(s, _exact_norm(r, s["w_in"], s["eps"]).to(s["r"].dtype).double())
    if s["w_post"] is not None:
        y = _exact_norm(y, s["w_post"], s["eps"])
    if c["gate"] != "none":
        y = y * (s["gate"].double()[:, None] if c["gate"] == "token" else s["gate"].double())
    out = s["res_scale"] * r + y
    if c["op"] == "norm" and not c["next"]:
        return {"r": out}
    return {"r": out, "x": _exact_norm(out, s["w_next"], s["eps"])}
