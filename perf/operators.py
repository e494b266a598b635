"""The measured cases of the standalone operators: 4-bit linear products for few tokens, products grouped by
expert, the permutation and the combination around them, and the norms around a block.

`own` False computes each operator in its plain form (elementary torch operations in fp32, rounded once);
`own` True calls the package's operators. A case's "op" names the operator, the rest are its sizes.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    return [
        # one token through a small projection whose int4 weights are stored rotated: latency is all of it
        {"name": "q4 int4 T1 2048x512", "op": "q4", "fmt": "int4", "rotated": True, "type": "bf16", "T": 1, "N": 2048,
         "K": 512, "pad": 0},
        # a decode batch of 8 through a large square projection: 36 MB of weights to stream
        {"name": "q4 int4 T8 8192x8192", "op": "q4", "fmt": "int4", "rotated": True, "type": "bf16", "T": 8, "N": 8192,
         "K": 8192, "pad": 0},
        # a larger batch with nothing round: odd rows, a K of 257 NVFP4 blocks, rows inside a wider buffer
        {"name": "q4 nvfp4 T37 5001x4112", "op": "q4", "fmt": "nvfp4", "rotated": False, "type": "f16", "T": 37,
         "N": 5001, "K": 4112, "pad": 24},
        # decode: four tokens, six experts each, gate|up with SwiGLU, rows gathered through the permutation
        {"name": "grouped decode gate|up", "op": "grouped", "type": "bf16", "E": 256, "T": 4, "top_k": 6, "N": 1024,
         "K": 2048, "act": "swiglu", "gather": True, "skew": False},
        # a prompt of 2048 tokens over 256 experts, gate|up with SwiGLU: the largest case
        {"name": "grouped prefill gate|up", "op": "grouped", "type": "bf16", "E": 256, "T": 2048, "top_k": 6, "N": 1024,
         "K": 2048, "act": "swiglu", "gather": True, "skew": False},
        # down projection with uneven loads (hot and empty experts), odd widths, rows already in expert order
        {"name": "grouped ragged down", "op": "grouped", "type": "f16", "E": 61, "T": 5003, "top_k": 1, "N": 1000,
         "K": 520, "act": "none", "gather": False, "skew": True},
        # routing of a small decode batch
        {"name": "permute T5", "op": "permute", "E": 256, "T": 5, "top_k": 6, "drop": 0.0},
        # routing of a long prompt batch with padded tokens (no expert) among it
        {"name": "permute T16384", "op": "permute", "E": 1000, "T": 16384, "top_k": 8, "drop": 0.1},
        # expert outputs back to three tokens, with the shared expert's output added
        {"name": "combine T3", "op": "combine", "type": "bf16", "T": 3, "top_k": 6, "H": 2048, "addend": True,
         "drop": 0.0},
        # the same for a long prompt, without a shared expert, some slots dropped
        {"name": "combine T8192", "op": "combine", "type": "f16", "T": 8192, "top_k": 6, "H": 2048, "addend": False,
         "drop": 0.1},
        # between two blocks at decode: fp32 residual, the branch added, the next block's input normalised
        {"name": "norm T4", "op": "norm", "type": "bf16", "res": "f32", "T": 4, "H": 2048, "post": False,
         "gate": "none", "weights": True},
        # the same for a prompt with the branch normalised and gated per element, residual in the model's type
        {"name": "norm T8192 gated", "op": "norm", "type": "bf16", "res": "bf16", "T": 8192, "H": 4096, "post": True,
         "gate": "token", "weights": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("q4", "q4", "grouped", "grouped", "permute", "combine", "norm"))
    if op == "q4":
        fmt = rng.choice(("int4", "int4", "nvfp4"))
        K = 128 * _log(rng, 1, 80) if fmt == "int4" else 16 * _log(rng, 1, 640)
        return {"op": op, "fmt": fmt, "rotated": fmt == "int4" and rng.random() < 0.6,
                "type": rng.choice(("bf16", "f16")), "T": _log(rng, 1, 64), "N": _log(rng, 17, 10000), "K": K,
                "pad": rng.choice((0, 0, 8, 40))}
    if op == "grouped":
        act = rng.choice(("none", "swiglu"))
        gather = rng.random() < 0.6
        return {"op": op, "type": rng.choice(("bf16", "f16")), "E": _log(rng, 1, 256), "T": _log(rng, 1, 2048),
                "top_k": rng.randint(1, 6) if gather else 1, "N": 2 * _log(rng, 8, 512) if act == "swiglu" else _log(rng, 9, 2048),
                "K": 8 * _log(rng, 4, 256), "act": act, "gather": gather, "skew": rng.random() < 0.5}
    if op == "permute":
        E = _log(rng, 8, 1024)
        return {"op": op, "E": E, "T": _log(rng, 1, 16384), "top_k": rng.randint(1, min(8, E)),
                "drop": rng.choice((0.0, 0.1, 0.5))}
    if op == "combine":
        return {"op": op, "type": rng.choice(("bf16", "f16")), "T": _log(rng, 1, 8192), "top_k": rng.randint(1, 8),
                "H": 8 * _log(rng, 8, 512) if rng.random() < 0.8 else _log(rng, 65, 4095), "addend": rng.random() < 0.5,
                "drop": rng.choice((0.0, 0.1))}
    return {"op": "norm", "type": rng.choice(("bf16", "f16")), "res": rng.choice(("f32", "same")), "T": _log(rng, 1, 8192),
            "H": 8 * _log(rng, 8, 512) if rng.random() < 0.8 else _log(rng, 65, 4095), "post": rng.random() < 0.5,
            "gate": rng.choice(("none", "row", "token")), "weights": rng.random() < 0.6}


# --------------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _activations(g, rows, cols, dtype, pad=0):
    """Hidden states of rms 1.26 with a few channels thirty times as large, as late blocks see; rows `pad`
    elements longer than used when pad > 0."""
    x = torch.randn((rows, cols + pad), generator=g, device=DEV) * 1.26
    hot = torch.randint(0, cols, (max(1, cols // 512),), generator=g, device=DEV)
    x[:, hot] *= 30.0
    return x.to(dtype)[:, :cols]


def _choices(g, T, E, k, skew):
    """k distinct experts per token, ascending, from random scores; skewed: some experts are hot, some idle."""
    score = torch.rand((T, E), generator=g, device=DEV)
    if skew:
        bias = torch.randn((E,), generator=g, device=DEV) * 1.5
        score = torch.log(score + 1e-6) * torch.exp(-bias)
        score = torch.where(bias < -2.0, score - 1e9, score)
    return score.topk(k, dim=1).indices.sort(dim=1).values.to(torch.int32)


def _order(ids, E):
    """Expert-major order of the flat pairs (stable), and the groups' offsets."""
    flat = ids.reshape(-1).long()
    perm = torch.sort(flat, stable=True).indices.to(torch.int32)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    return perm, offsets, int(counts.max())


def prepare(case, seed):
    g = _gen(seed)
    c, op = case, case["op"]
    s = {"case": c}
    if op == "q4":
        dt = TYPES[c["type"]]
        s["x"] = _activations(g, c["T"], c["K"], dt, c["pad"])
        s["codes"] = torch.randint(0, 256, (c["N"], c["K"] // 2), generator=g, device=DEV, dtype=torch.uint8)
        if c["fmt"] == "int4":
            u = torch.rand((c["N"], c["K"] // 128), generator=g, device=DEV)
            s["scales"] = (0.004 * (1 + u)).to(torch.bfloat16)
            s["tscale"] = None
        else:
            e = torch.randint(-4, 3, (c["N"], c["K"] // 16), generator=g, device=DEV)
            m = torch.randint(8, 16, (c["N"], c["K"] // 16), generator=g, device=DEV)
            s["scales"] = (m.float() * torch.exp2(e.float() - 3)).to(torch.float8_e4m3fn)
            s["tscale"] = torch.full((1,), 0.01, device=DEV)
    elif op == "grouped":
        dt = TYPES[c["type"]]
        P = c["T"] * c["top_k"]
        s["w"] = torch.empty((c["E"], c["N"], c["K"]), device=DEV, dtype=dt)
        s["w"].normal_(0, 0.02, generator=g)
        s["x"] = _activations(g, c["T"], c["K"], dt)
        k = min(c["top_k"], c["E"])
        ids = _choices(g, P // k if P % k == 0 else P, c["E"], k if P % k == 0 else 1, c["skew"])
        perm, s["offsets"], s["cap"] = _order(ids, c["E"])
        s["rows"] = perm if c["gather"] else None
    elif op == "permute":
        ids = _choices(g, c["T"], c["E"], c["top_k"], True)
        s["ids"] = torch.where(torch.rand((c["T"], 1), generator=g, device=DEV) < c["drop"], -1, ids).to(torch.int32)
    elif op == "combine":
        dt = TYPES[c["type"]]
        P = c["T"] * c["top_k"]
        s["o"] = _normal(g, (P, c["H"]), 1.0, dt)
        inv = torch.randperm(P, generator=g, device=DEV).to(torch.int32).reshape(c["T"], c["top_k"])
        s["inv"] = torch.where(torch.rand(inv.shape, generator=g, device=DEV) < c["drop"], -1, inv).to(torch.int32)
        w = torch.rand((c["T"], c["top_k"]), generator=g, device=DEV)
        s["w"] = w / w.sum(1, keepdim=True)
        s["addend"] = _normal(g, (c["T"], c["H"]), 1.0, dt) if c["addend"] else None
    else:
        dt = TYPES[c["type"]]
        rt = TYPES["f32"] if c["res"] == "f32" else dt
        T, H = c["T"], c["H"]
        s["x"] = _activations(g, T, H, rt)
        s["y"] = _normal(g, (T, H), 0.7, dt)
        s["gate"] = None if c["gate"] == "none" else _normal(g, (1 if c["gate"] == "row" else T, H), 1.0, dt)
        s["post_weight"] = (1 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(dt) if c["weights"] and c["post"] else None
        s["pre_weight"] = (1 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(dt) if c["weights"] else None
    return s


# ----------------------------------------------------------------------------------------------- plain forms

def _hadamard(n, dtype):
    i = torch.arange(n, device=DEV)
    a = i[:, None] & i[None, :]
    a = a ^ (a >> 4)
    a = a ^ (a >> 2)
    a = a ^ (a >> 1)
    return (1 - 2 * (a & 1)).to(dtype) / math.sqrt(n)


def _q4_weight(s, dtype):
    c = s["case"]
    codes = torch.stack((s["codes"] & 15, s["codes"] >> 4), dim=2).reshape(c["N"], c["K"]).long()
    if c["fmt"] == "int4":
        v = torch.where(codes > 7, codes - 16, codes).to(dtype)
        return v * s["scales"].to(dtype).repeat_interleave(128, dim=1)
    v = torch.tensor(E2M1, device=DEV, dtype=dtype)[codes]
    return v * s["scales"].to(dtype).repeat_interleave(16, dim=1)


def _q4_plain(s):
    c = s["case"]
    x = s["x"].float()
    if c["rotated"]:
        x = (x.reshape(c["T"], -1, 128) @ _hadamard(128, torch.float32)).reshape(c["T"], c["K"])
    y = x @ _q4_weight(s, torch.float32).t()
    if s["tscale"] is not None:
        y = y * s["tscale"]
    return y.to(s["x"].dtype)


def _grouped_plain(s):
    c = s["case"]
    P, E, cap = c["T"] * c["top_k"], c["E"], s["cap"]
    x = s["x"].float()
    if s["rows"] is not None:
        x = x[torch.div(s["rows"], c["top_k"], rounding_mode="floor").long()]
    off = s["offsets"].long()
    p = torch.arange(P, device=DEV)
    e = torch.searchsorted(off[1:], p, right=True)
    at = e * cap + p - off[e]
    padded = torch.zeros((E * cap, c["K"]), device=DEV).index_copy_(0, at, x).reshape(E, cap, c["K"])
    y = torch.bmm(padded, s["w"].float().transpose(1, 2)).reshape(E * cap, c["N"])[at]
    if c["act"] == "swiglu":
        gate, up = y[:, : c["N"] // 2], y[:, c["N"] // 2 :]
        y = gate / (1 + torch.exp(-gate)) * up
    return y.to(s["x"].dtype)


def _permute_plain(s):
    c = s["case"]
    flat = s["ids"].reshape(-1).long()
    E, P = c["E"], flat.numel()
    key = torch.where((flat < 0) | (flat >= E), E, flat)
    order = torch.sort(key, stable=True).indices
    counts = torch.zeros(E + 1, dtype=torch.int64, device=DEV).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = counts[:E].cumsum(0)
    live = torch.arange(P, device=DEV) < offsets[E]
    pos = torch.empty_like(order).scatter_(0, order, torch.arange(P, device=DEV))
    perm = torch.where(live, order, -1)
    inv = torch.where(key < E, pos, -1)
    return {"offsets": offsets.to(torch.int32), "perm": perm.to(torch.int32),
            "inv": inv.to(torch.int32).reshape(s["ids"].shape)}


def _combine_plain(s):
    inv = s["inv"].long()
    w = torch.where(inv < 0, 0.0, s["w"])
    rows = s["o"].float()[inv.clamp(min=0)]
    y = (rows * w[:, :, None]).sum(1)
    if s["addend"] is not None:
        y = y + s["addend"].float()
    return y.to(s["o"].dtype)


EPS, RES_SCALE, BRANCH_SCALE = 1e-6, 0.9, 1.25


def _norm_plain(s):
    x, y = s["x"].float(), s["y"].float()
    if s["case"]["post"]:
        y = y / torch.sqrt((y * y).mean(1, keepdim=True) + EPS)
        if s["post_weight"] is not None:
            y = y * s["post_weight"].float()
    if s["gate"] is not None:
        y = y / (1 + torch.exp(-s["gate"].float()))
    x = RES_SCALE * x + BRANCH_SCALE * y
    z = x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    if s["pre_weight"] is not None:
        z = z * s["pre_weight"].float()
    return {"x": x.to(s["x"].dtype), "z": z.to(s["y"].dtype)}


PLAIN = {"q4": _q4_plain, "grouped": _grouped_plain, "permute": _permute_plain, "combine": _combine_plain,
         "norm": _norm_plain}


# ------------------------------------------------------------------------------------------------------ run

def run(state):
    c = state["case"]
    if not own:
        return PLAIN[c["op"]](state)
    from bit_routed_expert_sigmoid_b200 import ops

    if c["op"] == "q4":
        return ops.q4_linear(state["x"], state["codes"], state["scales"], state["tscale"], fmt=c["fmt"],
                             rotated=c["rotated"])
    if c["op"] == "grouped":
        return ops.grouped_linear(state["x"], state["w"], state["offsets"], rows=state["rows"], row_div=c["top_k"],
                                  act=c["act"])
    if c["op"] == "permute":
        offsets, perm, inv = ops.expert_permute(state["ids"], c["E"])
        return {"offsets": offsets, "perm": perm, "inv": inv}
    if c["op"] == "combine":
        return ops.expert_combine(state["o"], state["inv"], state["w"], addend=state["addend"])
    x, z = ops.block_norm(state["x"], state["y"], post_norm=c["post"], post_weight=state["post_weight"],
                          gate=state["gate"], gate_act="sigmoid", res_scale=RES_SCALE, branch_scale=BRANCH_SCALE,
                          pre_weight=state["pre_weight"], eps=EPS)
    return {"x": x, "z": z}


# ---------------------------------------------------------------------------------------------------- work

def work(case):
    c, op = case, case["op"]
    if op == "q4":
        group = 2 / 128 if c["fmt"] == "int4" else 1 / 16
        w = c["N"] * c["K"] * (0.5 + group)
        return {"bytes": w + 2 * c["T"] * (c["N"] + c["K"]), "flops": 2 * c["T"] * c["N"] * c["K"]}
    if op == "grouped":
        P, E = c["T"] * c["top_k"], c["E"]
        # experts that at least one row goes to, for even loads (skewed loads reach fewer)
        k = min(c["top_k"], E)
        active = E * (1 - (1 - k / E) ** (P // k))
        out = c["N"] // 2 if c["act"] == "swiglu" else c["N"]
        rows = c["T"] if c["gather"] else P
        return {"bytes": 2 * (active * c["N"] * c["K"] + rows * c["K"] + P * out) + 4 * (E + 1 + P),
                "flops": 2 * P * c["N"] * c["K"]}
    if op == "permute":
        return {"bytes": 4 * (3 * c["T"] * c["top_k"] + c["E"] + 1), "flops": 0}
    if op == "combine":
        P = c["T"] * c["top_k"]
        live = P * (1 - c["drop"])
        return {"bytes": 2 * c["H"] * (live + c["T"] * (2 if c["addend"] else 1)) + 8 * P, "flops": 2 * live * c["H"]}
    n, r = c["T"] * c["H"], 4 if c["res"] == "f32" else 2
    gate = {"none": 0, "row": c["H"], "token": n}[c["gate"]]
    return {"bytes": n * (2 * r + 4) + 2 * gate + (2 * c["H"] * (2 if c["post"] else 1) if c["weights"] else 0),
            "flops": 10 * n}


# ---------------------------------------------------------------------------------------------------- exact

def exact(case, seed):
    s, c, op = prepare(case, seed), case, case["op"]
    f64 = torch.float64
    if op == "q4":
        w = _exact_q4(s)
        x = s["x"].to(f64)
        if c["rotated"]:                     # W blockdiag(Hn) against blockdiag(Hn) x, by doubling from the 1 x 1 matrix
            h = torch.ones((1, 1), dtype=f64, device=DEV)
            while h.shape[0] < 128:
                h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
            x = torch.einsum("tsk,jk->tsj", x.unflatten(1, (-1, 128)), h / math.sqrt(128.0)).flatten(1)
        return torch.einsum("tk,nk->tn", x, w)
    if op == "grouped":
        off = s["offsets"].tolist()
        x = s["x"].to(f64)
        if s["rows"] is not None:
            x = x[(s["rows"] // c["top_k"]).long()]
        y = torch.empty((c["T"] * c["top_k"], c["N"]), dtype=f64, device=DEV)
        for e in range(c["E"]):
            if off[e + 1] > off[e]:
                y[off[e] : off[e + 1]] = x[off[e] : off[e + 1]] @ s["w"][e].to(f64).mT
        if c["act"] == "swiglu":
            gate, up = y.chunk(2, dim=1)
            y = gate * torch.sigmoid(gate) * up
        return y
    if op == "permute":
        return None
    if op == "combine":
        y = torch.zeros((c["T"], c["H"]), dtype=f64, device=DEV)
        for k in range(c["top_k"]):
            t = (s["inv"][:, k] >= 0).nonzero()[:, 0]
            y[t] += s["w"][t, k].to(f64)[:, None] * s["o"].index_select(0, s["inv"][t, k]).to(f64)
        return y if s["addend"] is None else y + s["addend"].to(f64)
    x, y = s["x"].to(f64), s["y"].to(f64)
    if c["post"]:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
        y = y if s["post_weight"] is None else y * s["post_weight"].to(f64)
    if s["gate"] is not None:
        y = y * torch.sigmoid(s["gate"].to(f64))
    x = RES_SCALE * x + BRANCH_SCALE * y
    z = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return {"x": x, "z": z if s["pre_weight"] is None else z * s["pre_weight"].to(f64)}


def _exact_q4(s):
    c = s["case"]
    lo, hi = (s["codes"] % 16).to(torch.int64), (s["codes"] // 16).to(torch.int64)
    w = torch.empty((c["N"], c["K"]), dtype=torch.float64, device=DEV)
    if c["fmt"] == "int4":
        w[:, 0::2], w[:, 1::2] = ((lo + 8) % 16 - 8).double(), ((hi + 8) % 16 - 8).double()
        return (w.unflatten(1, (-1, 128)) * s["scales"].double()[:, :, None]).flatten(1)
    for half, code in ((0, lo), (1, hi)):    # sign, two exponent bits (bias 1), one fraction bit
        ex, m = (code >> 1) & 3, (code & 1).double()
        v = torch.where(ex == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(ex.double() - 1))
        w[:, half::2] = torch.where(code > 7, -v, v)
    return (w.unflatten(1, (-1, 16)) * s["scales"].double()[:, :, None]).flatten(1) * s["tscale"].double()
