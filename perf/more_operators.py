"""Cases of what training the MoE layer needs, in plain torch and as the library's calls.

  gemm     products grouped by expert with ragged sizes, and both gradients (moe_grouped_gemm,
           moe_grouped_gemm_backward_rows, moe_grouped_gemm_backward_weights)
  drop     dropout whose mask is made from a counter and never stored: on the branch that joins a residual
           stream (moe_dropout), and inside the experts' activation and its gradient (moe_swiglu,
           moe_swiglu_backward)
  combine  gradients of the weighted unpermute-combine and of the permutation
           (moe_unpermute_combine_backward, moe_permute_backward)
  route    load-balance and z losses of the router and the gradient of its logits (moe_route_loss,
           moe_route_backward)

The mask: Philox-4x32-10 (Salmon, Moraes, Dror, Shaw: Parallel random numbers: as easy as 1, 2, 3, 2011) with the seed
as its key and (block, offset) as its counter gives 128 bits for each block of 8 consecutive elements; element
i of a block is dropped where its 16 bits (field i, from the low end) are below round(65536 p).
"""

import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _gemm(name, dir, n, T, k, N, K, dtype="bf16", out=None, gather=False, add=False, skew=0.0):
    return {"name": name, "op": "gemm", "dir": dir, "n": n, "T": T, "k": k, "N": N, "K": K, "dtype": dtype,
            "out": out or dtype, "gather": gather, "add": add, "skew": skew}


def listed():
    return [
        # a decode batch's rows through one matrix of one device's 64 experts: the weights' bytes
        _gemm("fwd_decode", "fwd", 64, 64, 10, 1024, 4096, gather=True),
        # a training batch's tokens through the experts' up projection
        _gemm("fwd_batch", "fwd", 64, 4096, 8, 1024, 4096, gather=True),
        # the gradient of those rows, added to the gate projection's
        _gemm("rows_batch", "rows", 64, 4096, 8, 1024, 4096, add=True),
        # the gradient of the down projection's weights, added to the step's fp32 sums
        _gemm("weights_batch", "weights", 64, 4096, 8, 4096, 1024, out="f32", add=True),
        # popular and empty experts, widths that end inside every tile, fp32
        _gemm("rows_ragged_f32", "rows", 24, 333, 3, 328, 712, dtype="f32", skew=2.0),
        # the router's weight gradient: one group, few outputs, every token in the sum
        _gemm("weights_router", "weights", 1, 8192, 1, 512, 4096),
        # one token's branch joining the residual stream: launch latency
        {"name": "drop_one", "op": "drop", "dir": "residual", "rows": 1, "cols": 4096, "dtype": "bf16", "p": 0.1},
        # the experts' activation in the backward pass of a training batch
        {"name": "drop_swiglu_grad", "op": "drop", "dir": "swiglu_grad", "rows": 32768, "cols": 1024, "dtype": "bf16",
         "p": 0.1},
        # a prefill-sized batch: every expert row's gradient from its token's
        {"name": "combine_batch", "op": "combine", "dir": "combine", "T": 8192, "D": 4096, "E": 512, "k": 10,
         "local": 512, "dtype": "bf16"},
        # one device's share of a decode-sized batch: row gradients back to their tokens, most slots elsewhere
        {"name": "permute_share", "op": "combine", "dir": "permute", "T": 512, "D": 4096, "E": 512, "k": 10, "local": 64,
         "dtype": "bf16"},
        # the tiny layer's router: latency
        {"name": "route_tiny", "op": "route", "T": 64, "E": 16, "k": 2, "renorm": True, "out": "f32", "mask": False,
         "bias": False},
        # a prefill-sized batch over 512 experts, padding tokens among them, experts that a bias closes
        {"name": "route_batch", "op": "route", "T": 8192, "E": 512, "k": 10, "renorm": True, "out": "bf16",
         "mask": True, "bias": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "gemm", "drop", "combine", "route"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "gemm":
        n = _log(rng, 1, 64)
        k = rng.randint(1, min(8, n))
        N, K = 8 * _log(rng, 1, 512), 8 * _log(rng, 1, 512)
        T = _log(rng, 1, 32768 // k)
        # no more work than the largest listed case; the matrix cores do fp32 at a sixteenth of bf16's rate
        most = (1 << 37) // (16 if dtype == "f32" else 1)
        T = max(1, min(T, most // (k * N * K)))
        c = _gemm("", rng.choice(["fwd", "rows", "weights"]), n, T, k, N, K, dtype,
                  rng.choice(["bf16", "f32"]) if dtype == "bf16" else "f32", rng.random() < 0.5, rng.random() < 0.5,
                  rng.choice([0.0, 1.0, 3.0]))
        while c["n"] * N * K > 1 << 28:
            c["n"] = (c["n"] + 1) // 2
        c["k"] = min(c["k"], c["n"])
        c["gather"] = c["gather"] and c["dir"] != "rows"
    elif op == "drop":
        c = {"op": "drop", "dir": rng.choice(["residual", "swiglu", "swiglu_grad"]), "rows": _log(rng, 1, 16384),
             "cols": _log(rng, 1, 2048), "dtype": dtype, "p": rng.choice([0.0, 0.05, 0.1, 0.5, rng.random()])}
    elif op == "combine":
        E = _log(rng, 2, 512)
        c = {"op": "combine", "dir": rng.choice(["combine", "permute"]), "T": _log(rng, 1, 4096),
             "D": 64 * _log(rng, 1, 64), "E": E, "k": rng.randint(1, min(10, E)),
             "local": E if rng.random() < 0.5 else rng.randint(1, E), "dtype": dtype}
    else:
        E = _log(rng, 2, 1024)
        c = {"op": "route", "T": _log(rng, 1, 8192), "E": E, "k": rng.randint(1, min(10, (E + 1) // 2)),
             "renorm": rng.random() < 0.5, "out": dtype, "mask": rng.random() < 0.5, "bias": rng.random() < 0.5}
    c.pop("name", None)
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed, what):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1009 + what)
    return g


def _randn(seed, what, shape, std=1.0, dtype="f32"):
    return torch.randn(shape, generator=_gen(seed, what), device=DEV, dtype=torch.float32).mul_(std).to(_dt(dtype))


def _dt(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _empty(shape, dtype):
    return torch.empty(shape, dtype=_dt(dtype), device=DEV)


def _choices(seed, T, E, k, skew=0.0):
    """k distinct experts of each of T tokens; a skew leaves some experts without a token."""
    keys = torch.rand((T, E), generator=_gen(seed, 1), device=DEV)
    keys = keys + skew * torch.rand((E,), generator=_gen(seed, 2), device=DEV)
    return keys.topk(k, 1)[1]


def _blob(seed, ids):
    """The packed routing of the choices, with weights that sum to one, larger first."""
    w = -torch.rand(ids.shape, generator=_gen(seed, 3), device=DEV).clamp_min(1e-6).log()
    w = (w / w.sum(1, keepdim=True)).sort(1, descending=True)[0]
    return torch.stack([ids.int(), w.view(torch.int32)], 1).contiguous()


def _prepare_gemm(c, seed):
    T, n, k, N, K, dt = (c[x] for x in ("T", "n", "k", "N", "K", "dtype"))
    ids = _choices(seed, T, n, k, c["skew"]).reshape(-1)
    order = torch.argsort(ids, stable=True)
    offsets = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.bincount(ids, minlength=n).cumsum(0)
    R, src = T * k, T if c["gather"] else T * k
    s = {"case": c, "offsets": offsets, "at": offsets.tolist(),
         "index": (order // k).int() if c["gather"] else None,
         "ws": torch.empty(128 << 20, dtype=torch.uint8, device=DEV)}
    shape = {"fwd": (R, N), "rows": (R, K), "weights": (n, N, K)}[c["dir"]]
    if c["dir"] != "rows":
        s["a"] = _randn(seed, 4, (src, K), 1.0, dt)
    if c["dir"] != "fwd":
        s["d_out"] = _randn(seed, 5, (R, N), 0.1, dt)
    if c["dir"] != "weights":
        s["w"] = _randn(seed, 6, (n, N, K), K ** -0.5, dt)
    s["add"] = _randn(seed, 7, shape, 1.0, c["out"]) if c["add"] else None
    s["out"] = _empty(shape, c["out"])
    return s


def prepare(case, seed):
    c = case
    if c["op"] == "gemm":
        return _prepare_gemm(c, seed)
    if c["op"] == "drop":
        shape, dt = (c["rows"], c["cols"]), c["dtype"]
        rng = torch.randint(0, 1 << 62, (2,), generator=_gen(seed, 1), device=DEV, dtype=torch.int64)
        if c["dir"] == "residual":
            return {"case": c, "rng": rng, "x": _randn(seed, 2, shape, 1.0, dt), "r": _randn(seed, 3, shape, 2.0, dt),
                    "out": _empty(shape, dt)}
        s = {"case": c, "rng": rng, "gate": _randn(seed, 2, shape, 1.5, dt), "up": _randn(seed, 3, shape, 1.0, dt),
             "h": _empty(shape, dt)}
        if c["dir"] == "swiglu_grad":
            s |= {"d_h": _randn(seed, 4, shape, 0.1, dt), "d_gate": _empty(shape, dt), "d_up": _empty(shape, dt)}
        return s
    if c["op"] == "combine":
        T, D, E, k, dt = (c[x] for x in ("T", "D", "E", "k", "dtype"))
        ids = _choices(seed, T, E, k)
        first = (E - c["local"]) // 2
        here = (ids >= first) & (ids < first + c["local"])
        order = torch.argsort(torch.where(here, ids, E).reshape(-1), stable=True)
        inv = torch.empty(T * k, dtype=torch.int32, device=DEV)
        inv[order] = torch.arange(T * k, dtype=torch.int32, device=DEV)
        inv = torch.where(here, inv.reshape(T, k), -1)
        # the rows of this device's experts; as many of the buffers' rows are in use
        s = {"case": c, "packed": _blob(seed, ids), "inv": inv, "used": int(here.sum()),
             "rows": _randn(seed, 4, (T * k, D), 1.0, dt)}
        if c["dir"] == "combine":
            return s | {"dy": _randn(seed, 5, (T, D), 0.1, dt), "d_rows": _empty((T * k, D), dt),
                        "d_w": _empty((T, k), "f32")}
        return s | {"add": _randn(seed, 5, (T, D), 1.0, dt), "dx": _empty((T, D), dt)}
    T, E, k = c["T"], c["E"], c["k"]
    logits = _randn(seed, 1, (T, E), 1.5)
    bias = None
    if c["bias"]:
        bias = _randn(seed, 2, (E,), 0.5)
        bias[torch.randperm(E, generator=_gen(seed, 3), device=DEV)[:(E - k) // 4]] = -math.inf
    key = logits if bias is None else logits + bias
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    w = torch.softmax(top, 1)[:, :k]
    w = w / w.sum(1, keepdim=True) if c["renorm"] else w
    mask = (torch.rand(T, generator=_gen(seed, 4), device=DEV) < 0.9).to(torch.uint8) if c["mask"] else None
    return {"case": c, "logits": logits, "bias": bias, "mask": mask,
            "packed": torch.stack([ids[:, :k].int(), w.contiguous().view(torch.int32)], 1).contiguous(),
            "d_w": _randn(seed, 5, (T, k), 0.1), "d_loss": torch.tensor([1e-2, 1e-3], device=DEV),
            "loss": _empty((2,), "f32"), "load": torch.empty(E + 1, dtype=torch.int32, device=DEV),
            "d_logits": _empty((T, E), c["out"]), "ws": torch.empty(16 << 20, dtype=torch.uint8, device=DEV)}


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _plain_gemm(s):
    c, at, out = s["case"], s["at"], s["out"]
    if c["dir"] == "weights":
        for e, (b, t) in enumerate(zip(at, at[1:])):
            a = s["a"][b:t] if s["index"] is None else s["a"][s["index"][b:t].long()]
            v = s["d_out"][b:t].float().t() @ a.float()
            out[e] = v if s["add"] is None else v + s["add"][e].float()
        return {"d_w": out}
    for e, (b, t) in enumerate(zip(at, at[1:])):
        if b == t:
            continue
        if c["dir"] == "fwd":
            a = s["a"][b:t] if s["index"] is None else s["a"][s["index"][b:t].long()]
            v = a.float() @ s["w"][e].float().t()
        else:
            v = s["d_out"][b:t].float() @ s["w"][e].float()
        out[b:t] = v if s["add"] is None else v + s["add"][b:t].float()
    return {"rows": out}


PHILOX_M = (0xD2511F53, 0xCD9E8D57)
PHILOX_W = (0x9E3779B9, 0xBB67AE85)
LOW32 = 0xFFFFFFFF


def _philox(blocks, rng):
    """[n, 4] words (int64, 0 .. 2^32 - 1) of the counters (blocks, rng[1]) under the key rng[0]."""
    c = [blocks & LOW32, blocks >> 32, (rng[1] & LOW32).expand_as(blocks), ((rng[1] >> 32) & LOW32).expand_as(blocks)]
    k = [rng[0] & LOW32, (rng[0] >> 32) & LOW32]
    for _ in range(10):
        p0, p1 = c[0] * PHILOX_M[0], c[2] * PHILOX_M[1]
        c = [((p1 >> 32) & LOW32) ^ c[1] ^ k[0], p1 & LOW32, ((p0 >> 32) & LOW32) ^ c[3] ^ k[1], p0 & LOW32]
        k = [(k[0] + PHILOX_W[0]) & LOW32, (k[1] + PHILOX_W[1]) & LOW32]
    return torch.stack(c, -1)


def _keep(s):
    """Which elements stay, and the factor of those."""
    c = s["case"]
    n, low = c["rows"] * c["cols"], round(c["p"] * 65536)
    words = _philox(torch.arange((n + 7) // 8, device=DEV), s["rng"])
    fields = torch.stack([words & 0xFFFF, words >> 16], -1).reshape(-1)[:n]
    return (fields >= low).reshape(c["rows"], c["cols"]), 65536 / (65536 - low) if low < 65536 else 0.0


def _plain_drop(s):
    c, dt = s["case"], _dt(s["case"]["dtype"])
    keep, factor = _keep(s)
    drop = lambda v: torch.where(keep, v * factor, 0.0)  # noqa: E731
    if c["dir"] == "residual":
        return {"out": (s["r"].float() + drop(s["x"].float())).to(dt)}
    g, u = s["gate"].float(), s["up"].float()
    sig = 1 / (1 + torch.exp(-g))
    h = drop(g * sig * u).to(dt)
    if c["dir"] == "swiglu":
        return {"h": h}
    d = drop(s["d_h"].float())
    return {"h": h, "d_gate": (d * u * sig * (1 + g * (1 - sig))).to(dt), "d_up": (d * g * sig).to(dt)}


def _plain_combine(s):
    c, dt, inv = s["case"], _dt(s["case"]["dtype"]), s["inv"].long()
    here, at = inv >= 0, inv.clamp_min(0)
    if c["dir"] == "permute":
        dx = s["add"].float()
        for j in range(c["k"]):
            dx = dx + torch.where(here[:, j, None], s["rows"][at[:, j]].float(), 0.0)
        return {"dx": dx.to(dt)}
    w = s["packed"][:, 1].contiguous().view(torch.float32)
    dy = s["dy"].float()
    for j in range(c["k"]):
        s["d_w"][:, j] = torch.where(here[:, j], (dy * s["rows"][at[:, j]].float()).sum(1), 0.0)
        m = here[:, j]
        s["d_rows"][at[m, j]] = (dy[m] * w[m, j, None]).to(dt)
    return {"d_w": s["d_w"], "d_rows": s["d_rows"][:s["used"]]}


def _plain_route(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    key = s["logits"] if s["bias"] is None else s["logits"] + s["bias"]
    top = key.amax(1, keepdim=True)
    ex = torch.exp(key - top)
    total = ex.sum(1, keepdim=True)
    p, lse = ex / total, top + torch.log(total)
    on = torch.ones(T, 1, device=DEV) if s["mask"] is None else (s["mask"] != 0).float()[:, None]
    ids = s["packed"][:, 0].long()
    w = s["packed"][:, 1].contiguous().view(torch.float32)
    n = on.sum()
    load = torch.zeros(E, device=DEV).index_add_(0, ids.reshape(-1), on.expand(T, k).reshape(-1))
    inv_n = 1 / n.clamp_min(1)
    balance = E / k * (load * inv_n * (p * on).sum(0) * inv_n).sum()
    z = (lse.square() * on).sum() * inv_n
    mean = (w * s["d_w"]).sum(1, keepdim=True)
    if c["renorm"]:
        d = torch.zeros(T, E, device=DEV).scatter_add_(1, ids, w * (s["d_w"] - mean))
    else:
        d = p * (torch.zeros(T, E, device=DEV).scatter_add_(1, ids, s["d_w"]) - mean)
    cb, cz = s["d_loss"][0], s["d_loss"][1]
    d = d + on * p * (cb * E / k * inv_n * inv_n * (load - (p * load).sum(1, keepdim=True)) + cz * 2 * inv_n * lse)
    return {"loss": torch.stack([balance, z]), "load": torch.cat([load, n[None]]).int(), "d_logits": d.to(_dt(c["out"]))}


_PLAIN = {"gemm": _plain_gemm, "drop": _plain_drop, "combine": _plain_combine, "route": _plain_route}


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------

def _own(s):
    import sparse_moe_ffn_route_amd as moe

    c = s["case"]
    if c["op"] == "gemm":
        g = moe.make_groups(c["n"], c["T"] * c["k"], c["N"], c["K"], c["dtype"], c["out"])
        if c["dir"] == "fwd":
            moe.moe_grouped_gemm(g, s["a"], s["offsets"], s["w"], s["out"], index=s["index"], add=s["add"], ws=s["ws"])
        elif c["dir"] == "rows":
            moe.moe_grouped_gemm_backward_rows(g, s["d_out"], s["offsets"], s["w"], s["out"], add=s["add"], ws=s["ws"])
        else:
            moe.moe_grouped_gemm_backward_weights(g, s["d_out"], s["a"], s["offsets"], s["out"], index=s["index"],
                                                  add=s["add"], ws=s["ws"])
        return {"d_w" if c["dir"] == "weights" else "rows": s["out"]}
    if c["op"] == "drop":
        if c["dir"] == "residual":
            moe.moe_dropout(s["x"], s["out"], c["p"], s["rng"], residual=s["r"])
            return {"out": s["out"]}
        if c["dir"] == "swiglu":
            moe.moe_swiglu(s["gate"], s["up"], s["h"], p=c["p"], rng=s["rng"])
            return {"h": s["h"]}
        moe.moe_swiglu_backward(s["d_h"], s["gate"], s["up"], s["d_gate"], s["d_up"], h=s["h"], p=c["p"], rng=s["rng"])
        return {"h": s["h"], "d_gate": s["d_gate"], "d_up": s["d_up"]}
    if c["op"] == "combine":
        d = moe.make_dims(c["T"], c["D"], c["E"], c["k"], 64, 0, (c["E"] - c["local"]) // 2, c["local"], True, c["dtype"],
                          c["dtype"], c["dtype"])
        if c["dir"] == "permute":
            moe.moe_permute_backward(d, s["rows"], s["inv"], s["dx"], add=s["add"])
            return {"dx": s["dx"]}
        moe.moe_unpermute_combine_backward(d, s["dy"], s["packed"], s["inv"], s["rows"], s["d_rows"], s["d_w"])
        return {"d_w": s["d_w"], "d_rows": s["d_rows"][:s["used"]]}
    d = moe.make_dims(c["T"], 64, c["E"], c["k"], 64, renormalize=c["renorm"])
    moe.moe_route_loss(d, s["logits"], s["bias"], s["packed"], s["loss"], s["load"], mask=s["mask"], ws=s["ws"])
    moe.moe_route_backward(d, s["logits"], s["bias"], s["packed"], s["d_w"], s["load"], s["d_loss"], s["d_logits"],
                           mask=s["mask"])
    return {"loss": s["loss"], "load": s["load"], "d_logits": s["d_logits"]}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

_BYTES = {"f32": 4, "bf16": 2}


def work(case):
    c = case
    if c["op"] == "gemm":
        es, os, R = _BYTES[c["dtype"]], _BYTES[c["out"]], c["T"] * c["k"]
        used = c["n"] * (1 - (1 - c["k"] / c["n"]) ** c["T"])
        a = (c["T"] if c["gather"] else R) * c["K"]
        m = c["N"] * c["K"]
        read = {"fwd": a + used * m, "rows": R * c["N"] + used * m, "weights": a + R * c["N"]}[c["dir"]] * es
        out = {"fwd": R * c["N"], "rows": R * c["K"], "weights": c["n"] * m}[c["dir"]] * os
        return {"bytes": read + out * (2 if c["add"] else 1), "flops": 2 * R * m}
    if c["op"] == "drop":
        v = c["rows"] * c["cols"]
        return {"bytes": v * _BYTES[c["dtype"]] * {"residual": 3, "swiglu": 3, "swiglu_grad": 6}[c["dir"]], "flops": 8 * v}
    if c["op"] == "combine":
        es, v = _BYTES[c["dtype"]], c["T"] * c["D"]
        rows = v * c["k"] * c["local"] / c["E"]
        if c["dir"] == "permute":
            return {"bytes": es * (rows + 2 * v), "flops": rows}
        return {"bytes": es * (2 * rows + v) + 12 * c["T"] * c["k"], "flops": 3 * rows}
    v = c["T"] * c["E"]
    return {"bytes": v * (8 + _BYTES[c["out"]]) + 24 * c["T"] * c["k"], "flops": 20 * v}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_gemm(s):
    c, at = s["case"], s["at"]
    index = torch.arange(at[-1], device=DEV) if s["index"] is None else s["index"].long()
    parts = []
    for e in range(c["n"]):
        r = slice(at[e], at[e + 1])
        if c["dir"] == "weights":
            v = (s["a"][index[r]].double().T @ s["d_out"][r].double()).T
            parts.append(v if s["add"] is None else s["add"][e].double() + v)
        else:
            w = s["w"][e].double()
            v = (w @ s["a"][index[r]].double().T).T if c["dir"] == "fwd" else (w.T @ s["d_out"][r].double().T).T
            parts.append(v if s["add"] is None else s["add"][r].double() + v)
    return {"d_w": torch.stack(parts)} if c["dir"] == "weights" else {"rows": torch.cat(parts)}


def _exact_mask(s):
    """Each element's factor by the generator's definition, in numpy's unsigned 64-bit numbers."""
    import numpy as np

    c = s["case"]
    n = c["rows"] * c["cols"]
    seed, offset = (int(v) for v in s["rng"].tolist())
    mask32, m0, m1 = np.uint64(LOW32), np.uint64(PHILOX_M[0]), np.uint64(PHILOX_M[1])
    b = np.arange(-(-n // 8), dtype=np.uint64)
    x0, x1 = b & mask32, b >> np.uint64(32)
    x2, x3 = np.full_like(b, offset & LOW32), np.full_like(b, (offset >> 32) & LOW32)
    k0, k1 = seed & LOW32, (seed >> 32) & LOW32
    for r in range(10):
        a, d = x0 * m0, x2 * m1
        x0, x1, x2, x3 = ((d >> np.uint64(32)) ^ x1 ^ np.uint64((k0 + r * PHILOX_W[0]) & LOW32), d & mask32,
                          (a >> np.uint64(32)) ^ x3 ^ np.uint64((k1 + r * PHILOX_W[1]) & LOW32), a & mask32)
    bits = np.empty((b.size, 8), dtype=np.int32)
    for i, x in enumerate((x0, x1, x2, x3)):
        bits[:, 2 * i], bits[:, 2 * i + 1] = x & np.uint64(0xFFFF), x >> np.uint64(16)
    low = int(np.rint(c["p"] * 65536))
    m = np.zeros(n) if low == 65536 else np.where(bits.reshape(-1)[:n] < low, 0.0, 65536.0 / (65536 - low))
    return torch.from_numpy(m.reshape(c["rows"], c["cols"])).to(DEV)


def _exact_drop(s):
    c, m = s["case"], _exact_mask(s)
    if c["dir"] == "residual":
        return {"out": m * s["x"].double() + s["r"].double()}
    g, u = s["gate"].double(), s["up"].double()
    silu = g * torch.sigmoid(g)
    if c["dir"] == "swiglu":
        return {"h": m * silu * u}
    slope = torch.sigmoid(g) + silu * torch.sigmoid(-g)
    d = m * s["d_h"].double()
    return {"h": m * silu * u, "d_gate": d * slope * u, "d_up": d * silu}


def _exact_combine(s):
    c, inv = s["case"], s["inv"].long()
    t, j = torch.nonzero(inv >= 0, as_tuple=True)
    at = inv[t, j]
    if c["dir"] == "permute":
        dx = s["add"].double()
        for i in range(c["k"]):
            dx.index_add_(0, t[j == i], s["rows"][at[j == i]].double())
        return {"dx": dx}
    w = s["packed"][:, 1].contiguous().view(torch.float32).double()
    dy = s["dy"].double()
    d_w = torch.zeros(c["T"], c["k"], dtype=torch.float64, device=DEV)
    d_rows = torch.zeros(s["used"], c["D"], dtype=torch.float64, device=DEV)
    for i in range(c["k"]):
        ti, ai = t[j == i], at[j == i]
        d_w[ti, i] = torch.linalg.vecdot(dy[ti], s["rows"][ai].double())
        d_rows[ai] = w[ti, i, None] * dy[ti]
    return {"d_w": d_w, "d_rows": d_rows}


def _exact_route(s):
    c = s["case"]
    E, k = c["E"], c["k"]
    key = s["logits"].double()
    if s["bias"] is not None:
        key = (s["logits"] + s["bias"]).double()
    lse = torch.logsumexp(key, 1)
    p = torch.exp(key - lse[:, None])
    on = torch.ones(c["T"], dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"] != 0
    ids = s["packed"][:, 0].long()
    w = s["packed"][:, 1].contiguous().view(torch.float32).double()
    n = int(on.sum())
    load = torch.bincount(ids[on].reshape(-1), minlength=E)
    many = max(n, 1)
    share = load.double() / (k * many)
    loss = torch.stack([E * (share * p[on].sum(0)).sum() / many, (lse[on] ** 2).sum() / many])
    # of sum_j d_w[j] w[j]: of the softmax over the kept keys, or over all
    dw = s["d_w"].double()
    if c["renorm"]:
        jac = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]
        d = torch.zeros_like(p).scatter_add_(1, ids, (jac * dw[:, None, :]).sum(2))
    else:
        d = torch.zeros_like(p).scatter_add_(1, ids, dw * w) - p * (dw * w).sum(1, keepdim=True)
    cb, cz = s["d_loss"].double()
    own_ = cb * E / many * (p * share - p * (p @ share)[:, None]) + cz * 2 / many * lse[:, None] * p
    d[on] += own_[on]
    return {"loss": loss, "load": torch.cat([load, load.new_tensor([n])]).int(), "d_logits": d}


def exact(case, seed):
    s = prepare(case, seed)
    return {"gemm": _exact_gemm, "drop": _exact_drop, "combine": _exact_combine, "route": _exact_route}[case["op"]](s)
