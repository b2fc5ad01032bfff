"""Operators before, beside and behind the MoE layer, as cases to time and to compare.

Six kinds of case:

  norm      the residual's addition and the RMS norm ahead of the layer, rows and their MXFP8 form
  normgrad  its gradients
  dispatch  token rows that are in MXFP8 already, in expert order
  product   matrix products grouped by expert, ragged row counts
  prodgrad  its two gradients, by the rows and by the weights
  adamw     an AdamW step over many tensors, states in 32 or in 8 bits

With `own` false, `run` computes them from elementary torch operations in 32 bits; with `own` true it calls the library.
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
KINDS = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a few fp32 rows of a mid-size width, with the residual
        {"name": "norm_f32_37x1408", "op": "norm", "rows": 37, "d": 1408, "dtype": "f32", "residual": True, "codes": False},
        # the rows of 8 ranks x 4096 tokens ahead of a DeepSeek-V3-shaped layer in MXFP8
        {"name": "norm_mx_share", "op": "norm", "rows": 32768, "d": 7168, "dtype": "bf16", "residual": True, "codes": True},
        # the same layer's training step
        {"name": "normgrad_bf16_share", "op": "normgrad", "rows": 32768, "d": 7168, "dtype": "bf16", "residual": True},
        # a decoding batch of the share: 64 tokens of each of 8 ranks
        {"name": "dispatch_decode_share", "op": "dispatch", "R": 8, "T": 64, "d": 7168, "E": 256, "E_local": 32, "k": 8,
         "drop": 0.0, "skew": 0.0},
        # the whole share, uneven experts
        {"name": "dispatch_share", "op": "dispatch", "R": 8, "T": 4096, "d": 7168, "E": 256, "E_local": 32, "k": 8,
         "drop": 0.0, "skew": 0.5},
        # one token's six rows on a mid-size layer's experts: latency counts
        {"name": "product_one_token", "op": "product", "groups": 64, "rows": 6, "behind": 0, "K": 2048, "N": 1408,
         "dtype": "bf16", "layout": 0, "skew": 0.0},
        # a decoding batch of the share: some 16 rows an expert, the weights' bytes count
        {"name": "product_decode_share", "op": "product", "groups": 32, "rows": 509, "behind": 3, "K": 7168, "N": 2048,
         "dtype": "bf16", "layout": 0, "skew": 0.0},
        # a prompt of the share through the wide side of its experts, uneven
        {"name": "product_share", "op": "product", "groups": 32, "rows": 32749, "behind": 19, "K": 2048, "N": 7168,
         "dtype": "bf16", "layout": 0, "skew": 0.5},
        # fp32 gradients of a tiny layer, an odd number of rows
        {"name": "prodgrad_f32_tiny", "op": "prodgrad", "groups": 8, "rows": 509, "behind": 3, "K": 128, "N": 256,
         "dtype": "f32", "layout": 0, "skew": 1.0, "dw": "f32"},
        # a training step of the share with half its tokens
        {"name": "prodgrad_bf16_share", "op": "prodgrad", "groups": 32, "rows": 16381, "behind": 3, "K": 7168, "N": 2048,
         "dtype": "bf16", "layout": 0, "skew": 0.5, "dw": "bf16"},
        # the small fp32 tensors of a model: norm weights, routers, biases
        {"name": "adamw_f32_small", "op": "adamw", "count": 61, "total": 260000, "even": False, "param": "f32", "grad": "f32",
         "master": False, "states": 32},
        # the experts of a mid-size layer: 64 x (1408 x 2048) three times, bf16 weights with fp32 masters, 8-bit states
        {"name": "adamw_mx_experts", "op": "adamw", "count": 3, "total": 3 * 64 * 1408 * 2048, "even": True, "param": "bf16",
         "grad": "bf16", "master": True, "states": 8},
    ]


MOST_VALUES = 32768 * 7168           # values of the share's token rows
MOST_WEIGHTS = 32 * 7168 * 2048      # values of one of its weight tensors
MOST_FLOPS = 2 * 32768 * 7168 * 2048
MOST_PAIRS = 8 * 4096


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "normgrad", "dispatch", "product", "product", "prodgrad", "adamw"])
    while True:
        if op in ("norm", "normgrad"):
            dtype = rng.choice(["f32", "bf16"])
            codes = op == "norm" and rng.random() < 0.5
            unit = 128 if codes else 4 if dtype == "f32" else 8
            c = {"op": op, "rows": spread(1, 32768), "d": unit * spread(1, 8192 // unit), "dtype": dtype,
                 "residual": rng.random() < 0.7}
            if op == "norm":
                c["codes"] = codes
            if c["rows"] * c["d"] * (2 if dtype == "f32" else 1) <= MOST_VALUES:
                return c
        elif op == "dispatch":
            E = rng.choice([8, 16, 32, 64, 96, 128, 256])
            El = max(1, E // rng.choice([1, 1, 2, 4, 8]))
            c = {"op": op, "R": rng.choice([1, 1, 2, 3, 4, 8]), "T": spread(1, 4096), "d": 128 * spread(1, 56), "E": E,
                 "E_local": El, "k": rng.randint(1, 8), "drop": rng.choice([0.0, 0.0, 0.05, 0.3]),
                 "skew": rng.choice([0.0, 0.0, 0.5, 1.0])}
            if c["R"] * c["T"] * c["k"] * El // E <= MOST_PAIRS:
                return c
        elif op in ("product", "prodgrad"):
            dtype = rng.choice(["f32", "bf16", "bf16", "bf16"])
            unit = 4 if dtype == "f32" else 8
            c = {"op": op, "groups": spread(1, 256), "rows": spread(1, 32768), "behind": rng.choice([0, 0, 1, 37]),
                 "K": unit * spread(2, 7168 // unit), "N": unit * spread(2, 7168 // unit), "dtype": dtype,
                 "layout": rng.randint(0, 1), "skew": rng.choice([0.0, 0.5, 1.0])}
            if op == "prodgrad":
                c["dw"] = rng.choice([dtype, "f32"])
            flops = 2 * c["rows"] * c["K"] * c["N"] * (2 if op == "prodgrad" else 1) * (10 if dtype == "f32" else 1)
            top = -(-c["rows"] // c["groups"]) * (4 if c["skew"] else 2) * c["groups"]       # rows of the plain form, about
            if flops <= MOST_FLOPS and c["groups"] * c["K"] * c["N"] <= MOST_WEIGHTS // 2 and top * c["K"] <= MOST_VALUES:
                return c
        else:
            param = rng.choice(["f32", "bf16"])
            return {"op": op, "count": spread(1, 61), "total": spread(61, 1 << 28), "even": False, "param": param,
                    "grad": rng.choice([param, "f32"]), "master": param == "bf16" and rng.random() < 0.7,
                    "states": rng.choice([32, 8])}


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["rows"] * c["d"]
        esz = 4 if c["dtype"] == "f32" else 2
        # x and y, residual and sum, codes with scales written, read back, and their values
        return {"bytes": n * (esz * (4 if c["residual"] else 2) + (2 * (1 + 1 / 32) + 2 if c["codes"] else 0)) + 4 * c["d"],
                "flops": 4 * n}
    if c["op"] == "normgrad":
        n = c["rows"] * c["d"]
        return {"bytes": n * (4 if c["dtype"] == "f32" else 2) * (4 if c["residual"] else 3) + 8 * c["d"], "flops": 10 * n}
    if c["op"] == "dispatch":
        tokens = c["R"] * c["T"]
        pairs = tokens * c["k"] * c["E_local"] / c["E"] * (1 - c["drop"])
        return {"bytes": (min(tokens, pairs) + pairs) * c["d"] * (1 + 1 / 32) + pairs * 8, "flops": 0}
    if c["op"] in ("product", "prodgrad"):
        esz = 4 if c["dtype"] == "f32" else 2
        live = min(c["groups"], c["rows"])
        w = live * c["K"] * c["N"]
        flops = 2 * c["rows"] * c["K"] * c["N"]
        if c["op"] == "product":
            return {"bytes": (c["rows"] * (c["K"] + c["N"]) + w) * esz, "flops": flops}
        dw = c["groups"] * c["K"] * c["N"] * (4 if c["dw"] == "f32" else 2)
        return {"bytes": (c["rows"] * (2 * c["K"] + c["N"]) + w) * esz + dw, "flops": 2 * flops}
    p, g = (4 if c[k] == "f32" else 2 for k in ("param", "grad"))
    read_p = not c["master"]
    state = 2 * 2 * 4 if c["states"] == 32 else 2 * (2 * (1 + 1 / 32) + (1 + 1 / 32) + 2)     # 8 bits: read back as values
    return {"bytes": c["total"] * (g + p * (2 if read_p else 1) + (8 if c["master"] else 0) + state), "flops": 15 * c["total"]}


# ------------------------------------------------------------------------------------------------ inputs
def _rows(n, d, dtype, g, scale=1.0):
    return (torch.randn(n, d, generator=g, device=DEV) * scale).to(KINDS[dtype])


def _counts(c, g):
    """Rows of each group: how many there are goes by the sizes alone, which group has them by the seed."""
    G, rows = c["groups"], c["rows"]
    same = torch.Generator(device=DEV)
    same.manual_seed(rows + 7 * G)
    if rows <= G:
        n = (torch.arange(G, device=DEV) < rows).long()
    else:
        p = torch.softmax(torch.randn(G, generator=same, device=DEV) * 0.2 - c["skew"] * torch.log1p(torch.arange(G, device=DEV).float()), 0)
        n = torch.floor(p * rows).long()
        n[0] += rows - n.sum()
    return n[torch.randperm(G, generator=g, device=DEV)]


def _sizes(c):
    """Values of each tensor of an AdamW step."""
    if c["even"]:
        return [c["total"] // c["count"]] * c["count"]
    r = random.Random(c["count"] + 7 * c["total"])
    w = [math.exp(r.gauss(0, 1.5)) for _ in range(c["count"])]
    return [max(1, int(c["total"] * x / sum(w))) for x in w]


def _choices(c, g):
    """Distinct experts per token by noisy popularity, dropped pairs and a padded tail of -1."""
    R, T, E, El, k = c["R"], c["T"], c["E"], c["E_local"], c["k"]
    same = torch.Generator(device=DEV)
    same.manual_seed(R * T + 7 * E + k)
    score = torch.randn(R, T, E, generator=same, device=DEV) - c["skew"] * torch.log1p(torch.arange(E, device=DEV).float())
    idx = torch.topk(score, k, dim=-1).indices
    home = torch.randperm(E, generator=same, device=DEV)[:El]
    names = torch.randperm(E, generator=g, device=DEV)
    e2l = torch.full((E,), -1, dtype=torch.int32, device=DEV)
    e2l[names[home]] = torch.randperm(El, generator=g, device=DEV).int()
    idx = names[idx].to(torch.int32)
    if c["drop"] > 0:
        idx[torch.rand(R, T, k, generator=same, device=DEV) < c["drop"] / 2] = -1
        idx[:, T - int(T * c["drop"] / 2):] = -1
    return idx, e2l


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"case": c}
    if c["op"] in ("norm", "normgrad"):
        s["gamma"] = 1 + 0.1 * torch.randn(c["d"], generator=g, device=DEV)
        if c["op"] == "norm":
            s["x"] = _rows(c["rows"], c["d"], c["dtype"], g)
            s["residual"] = _rows(c["rows"], c["d"], c["dtype"], g, 3.0) if c["residual"] else None
        else:
            s["h"] = _rows(c["rows"], c["d"], c["dtype"], g, 3.0)
            s["dy"] = _rows(c["rows"], c["d"], c["dtype"], g)
            s["dh"] = _rows(c["rows"], c["d"], c["dtype"], g) if c["residual"] else None
        return s
    if c["op"] == "dispatch":
        R, T, d = c["R"], c["T"], c["d"]
        s["idx"], s["e2l"] = _choices(c, g)
        s["xq"], s["xs"] = [], []
        for _ in range(R):
            q, sc = _nearest8(_rows(T, d, "bf16", g).float())
            s["xq"].append(q)
            s["xs"].append(sc.view(T, d // 128, 4).transpose(0, 1).contiguous())
        flat = s["idx"].reshape(-1).long()
        loc = torch.where(flat >= 0, s["e2l"].long()[flat.clamp(min=0)], -1)
        s["N"] = int((loc >= 0).sum())
        # the layout that the layer's own call makes of these choices: rows of an expert in ascending (rank, token, j) order
        order = torch.argsort(torch.where(loc >= 0, loc, c["E_local"]), stable=True)[:s["N"]]
        tok = order // c["k"]
        s["pull_src"] = torch.stack((tok // T, tok % T), 1).int() if s["N"] else torch.zeros(1, 2, dtype=torch.int32, device=DEV)
        return s
    if c["op"] in ("product", "prodgrad"):
        n = _counts(c, g)
        s["offsets"] = torch.cat((n.new_zeros(1), torch.cumsum(n, 0))).int()
        s["live"] = torch.nonzero(n)[:, 0]
        s["cap"] = int(n.max())
        G, K, N = c["groups"], c["K"], c["N"]
        total = c["rows"] + c["behind"]
        s["x"] = _rows(total, K, c["dtype"], g)
        s["w"] = torch.empty(G, *((N, K) if c["layout"] == 0 else (K, N)), dtype=KINDS[c["dtype"]], device=DEV)
        for i in range(0, G, 8):
            s["w"][i:i + 8] = torch.randn(s["w"][i:i + 8].shape, generator=g, device=DEV) * K ** -0.5
        if c["op"] == "prodgrad":
            s["dy"] = _rows(total, N, c["dtype"], g)
        return s
    # AdamW: tensors of one kind lie in one buffer, each from a multiple of 128 values on
    sizes = _sizes(c)
    starts, at = [], 0
    for n in sizes:
        starts.append(at)
        at += -(-n // 128) * 128
    inside = torch.zeros(at, dtype=torch.bool, device=DEV)
    tensor = torch.zeros(at, dtype=torch.uint8, device=DEV)
    for i, (a, n) in enumerate(zip(starts, sizes)):
        inside[a:a + n] = True
        tensor[a:a + -(-n // 128) * 128] = i

    def values(scale):
        return torch.randn(at, generator=g, device=DEV) * scale * inside

    s["starts"], s["sizes"], s["total"] = starts, sizes, at
    p = values(0.02)
    s["param"] = p.to(KINDS[c["param"]])
    s["master"] = p if c["master"] else None
    size = torch.exp(torch.randn(at, generator=g, device=DEV))                # a value's typical gradient: over some powers of ten
    s["grad"] = (values(1e-3) * size).to(KINDS[c["grad"]])
    m, v = values(3e-4) * size, (1e-3 * size) ** 2 * inside
    if c["states"] == 32:
        s["m"], s["v"] = m, v
    else:
        half = torch.full((at,), 1 << 15, dtype=torch.int32, device=DEV)
        s["m"], s["ms"] = _rounded8(m, half, False)
        s["v"], s["vs"] = _rounded8(torch.sqrt(v), half, True)
    s["tensor"] = tensor
    s["seed"] = int(seed) * 1000003 + 12345
    return s


HYPER = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.1, "step": 1000}


# ------------------------------------------------------------------------------------------------ plain forms
def _blocks(v):
    """Blocks of 32 of the last axis and each one's largest magnitude."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    return b, b.abs().amax(-1, keepdim=True)


def _power(e):
    """2^e in fp32 for whole e in [-127, 127], by its bits (torch.ldexp is a unit off for some exponents on the GPU, and what is
    next to a border then falls on its other side)."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).int().view(torch.float32)


def _nearest8(v):
    """MXFP8 of fp32 rows: E4M3 codes and E8M0 scale codes of blocks of 32, scale 2^(floor(log2 max) - 8), nearest even, at
    most 448."""
    b, top = _blocks(v)
    e = torch.where(top > 0, (torch.frexp(top).exponent - 9).clamp(-127, 127), torch.full_like(top, -127, dtype=torch.int32))
    y = b * _power(-e)
    step = _power(torch.frexp(y).exponent.clamp(min=-5) - 4)       # E4M3's step at |y|
    q = (torch.round(y / step) * step).clamp(-448, 448)
    return q.to(torch.float8_e4m3fn).reshape(v.shape).view(torch.uint8), (e + 127).to(torch.uint8)[..., 0]


def _values8(codes, scales):
    """fp32 values of codes [..., K] and of one scale code for 32 of them."""
    v = codes.view(torch.float8_e4m3fn).float()
    return (v.reshape(*v.shape[:-1], -1, 32) * _power(scales[..., None].int() - 127)).reshape(v.shape)


def _rounded8(v, r16, root):
    """MXFP8 of an optimiser's state, rounded up with the probability of what is cut off (r16: 16 random bits a value): the
    smallest scale that keeps the block's largest magnitude within 448; a positive root takes the smallest code at least."""
    b, top = _blocks(v)
    e = (torch.frexp(top).exponent - 9).clamp(-127, 126)
    e = e + (top > 448.0 * _power(e)).int()
    e = torch.where(top > 0, e, torch.full_like(e, -127))
    y = (b * _power(-e)).abs().reshape(-1)
    part = (r16 << 4).reshape(-1)
    normal = ((y.view(torch.int32) + part) >> 20) - (120 << 3)
    small = ((y * 2.0 ** 29).int() + part) >> 20
    code = torch.where(y >= 2.0 ** -6, normal, small).clamp(max=126)
    if root:
        code = torch.where((y > 0) & (code == 0), 1, code)
    code = code + (torch.signbit(v.reshape(-1)) & (code > 0)).int() * 128
    return code.to(torch.uint8), (e + 127).to(torch.uint8).reshape(-1)


def _mix(z):
    """A mixing of 32 bits: two rounds of shift, exclusive or, and a product with an odd constant (the golden ratio's and
    the square root of 3's fractions)."""
    z = z ^ (z >> 16)
    z = (z * 0x9E3779B9) & 0xFFFFFFFF
    z = z ^ (z >> 15)
    z = (z * 0xBB67AE85) & 0xFFFFFFFF
    return z ^ (z >> 16)


def _bits(s, which):
    """32 random bits a value: of the seed, the step, the tensor, the value's place in it, and which of two words."""
    seed, step = s["seed"], HYPER["step"]
    head = _mix((_mix((_mix(seed & 0xFFFFFFFF) + (seed >> 32)) & 0xFFFFFFFF) + step) & 0xFFFFFFFF)
    keys = [_mix((_mix((_mix((head + i) & 0xFFFFFFFF) + 0) & 0xFFFFFFFF) + 1 + which) & 0xFFFFFFFF) for i in range(len(s["sizes"]))]
    key = torch.tensor(keys, dtype=torch.int64, device=DEV)[s["tensor"].int()]
    first = torch.tensor(s["starts"], dtype=torch.int64, device=DEV)[s["tensor"].int()]
    return _mix((torch.arange(s["total"], device=DEV) - first + key) & 0xFFFFFFFF)


def _norm(s):
    c = s["case"]
    x = s["x"].float()
    h = x if s["residual"] is None else x + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * s["gamma"]
    out = {"y": y.to(s["x"].dtype)}
    if c["residual"]:
        out["h"] = h.to(s["x"].dtype)
    if c["codes"]:
        out["codes"] = _values8(*_nearest8(y)).to(torch.bfloat16)
    return out


def _norm_grad(s):
    h, dy = s["h"].float(), s["dy"].float()
    rstd = torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6)
    u = dy * s["gamma"]
    dx = rstd * (u - h * (rstd.square() * (u * h).mean(-1, keepdim=True)))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["h"].dtype), "dgamma": (dy * h * rstd).sum(0)}


def _places(s):
    """Each row's place in a batch of `cap` rows for each group that has any."""
    c = s["case"]
    off = s["offsets"].long()
    row = torch.arange(c["rows"], device=DEV)
    group = torch.searchsorted(off[1:], row, right=True)
    batch = torch.zeros(c["groups"], dtype=torch.long, device=DEV)
    batch[s["live"]] = torch.arange(s["live"].numel(), device=DEV)
    return batch[group] * s["cap"] + row - off[group]


def _spread(rows, place, s):
    pad = torch.zeros(s["live"].numel() * s["cap"], rows.shape[1], device=DEV)
    pad[place] = rows.float()
    return pad.reshape(-1, s["cap"], rows.shape[1])


def _product(s):
    c = s["case"]
    place = _places(s)
    w = s["w"][s["live"]].float()
    w = w.transpose(1, 2) if c["layout"] == 0 else w
    y = torch.bmm(_spread(s["x"][:c["rows"]], place, s), w)
    return {"y": y.flatten(0, 1)[place].to(s["x"].dtype)}


def _product_grad(s):
    c = s["case"]
    place = _places(s)
    w = s["w"][s["live"]].float()
    w = w if c["layout"] == 0 else w.transpose(1, 2)
    x, dy = _spread(s["x"][:c["rows"]], place, s), _spread(s["dy"][:c["rows"]], place, s)
    dx = torch.bmm(dy, w).flatten(0, 1)[place]
    a, b = (dy, x) if c["layout"] == 0 else (x, dy)
    dw = torch.zeros(s["w"].shape, dtype=KINDS[c["dw"]], device=DEV)
    dw[s["live"]] = torch.bmm(a.transpose(1, 2), b).to(dw.dtype)
    return {"dx": dx.to(s["x"].dtype), "dw": dw}


def _adamw(s):
    c, y = s["case"], HYPER
    p = s["param"].float() if s["master"] is None else s["master"]
    g = s["grad"].float()
    if c["states"] == 32:
        m, v = s["m"], s["v"]
    else:
        m, v = _values8(s["m"], s["ms"]), _values8(s["v"], s["vs"]).square()
    m = y["beta1"] * m + (1 - y["beta1"]) * g
    v = y["beta2"] * v + (1 - y["beta2"]) * g * g
    away = m / (1 - y["beta1"] ** y["step"]) / (torch.sqrt(v / (1 - y["beta2"] ** y["step"])) + y["eps"])
    p = p * (1 - y["lr"] * y["weight_decay"]) - y["lr"] * away
    if s["master"] is not None:
        s["master"].copy_(p)
        s["param"].copy_(p)
    elif c["param"] == "bf16":
        s["param"].copy_(((p.view(torch.int32) + (_bits(s, 1) & 0xFFFF).int()) & -65536).view(torch.float32))
    else:
        s["param"].copy_(p)
    if c["states"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return _step_outputs(s, s["m"], s["v"])
    r = _bits(s, 0)
    s["m"], s["ms"] = _rounded8(m, (r & 0xFFFF).int(), False)
    s["v"], s["vs"] = _rounded8(torch.sqrt(v), (r >> 16).int(), True)
    return _step_outputs(s, _values8(s["m"], s["ms"]).to(torch.bfloat16), _values8(s["v"], s["vs"]).to(torch.bfloat16))


def _step_outputs(s, m, v):
    out = {"param": s["param"], "m": m, "v": v}
    if s["master"] is not None:
        out["master"] = s["master"]
    return out


def _dispatch(s):
    """Codes as E4M3 elements and their blocks' scale codes, moved as they are."""
    at = s["pull_src"][:s["N"]].long()
    at = at[:, 0] * s["case"]["T"] + at[:, 1]
    return {"codes": torch.cat(s["xq"])[at].view(torch.float8_e4m3fn), "scales": torch.cat(s["xs"], 1)[:, at]}


def _plain(s):
    return {"norm": _norm, "normgrad": _norm_grad, "dispatch": _dispatch, "product": _product, "prodgrad": _product_grad,
            "adamw": _adamw}[s["case"]["op"]](s)


# ------------------------------------------------------------------------------------------------ the library's calls
def _kept(s, name, make):
    """Buffers and descriptors that a program makes once."""
    if name not in s:
        s[name] = make()
    return s[name]


def _own(s):
    from mixture_experts_layer_histogram_amd import moe
    c = s["case"]
    code = {"f32": moe.MOE_F32, "bf16": moe.MOE_BF16}
    if c["op"] == "norm":
        rows, d = c["rows"], c["d"]
        n, y, h, q, sc, values = _kept(s, "buffers", lambda: (
            moe.Norm(rows, d, code[c["dtype"]], 1e-6), torch.empty_like(s["x"]),
            torch.empty_like(s["x"]) if c["residual"] else None,
            torch.empty(rows, d, dtype=torch.uint8, device=DEV) if c["codes"] else None,
            torch.empty(d // 128, rows, 4, dtype=torch.uint8, device=DEV) if c["codes"] else None,
            torch.empty(rows, d, dtype=torch.bfloat16, device=DEV) if c["codes"] else None))
        moe.moe_norm(n, s["x"], s["residual"], s["gamma"], h, y, q, sc)
        out = {"y": y}
        if c["residual"]:
            out["h"] = h
        if c["codes"]:
            moe.moe_mx_dequantize(q, sc, moe.MOE_MXFP8, rows, d, values, moe.MOE_BF16)
            out["codes"] = values
        return out
    if c["op"] == "normgrad":
        def make():
            n = moe.Norm(c["rows"], c["d"], code[c["dtype"]], 1e-6)
            return (n, torch.empty_like(s["h"]), torch.empty_like(s["gamma"]),
                    torch.empty(moe.moe_norm_backward_workspace_bytes(n), dtype=torch.uint8, device=DEV))
        n, dx, dgamma, ws = _kept(s, "buffers", make)
        moe.moe_norm_backward(n, s["dy"], s["h"], s["gamma"], s["dh"], dx, dgamma, ws)
        return {"dx": dx, "dgamma": dgamma}
    if c["op"] == "dispatch":
        def make():
            sh = moe.Shape(c["R"], c["T"], c["d"], c["E"], c["k"], 128, moe.MOE_MXFP8)
            p = moe.Placement(s["e2l"].data_ptr(), c["E_local"])
            i32 = dict(dtype=torch.int32, device=DEV)
            ws = torch.empty(moe.moe_workspace_bytes(sh, p), dtype=torch.uint8, device=DEV)
            offsets = torch.empty(c["E_local"] + 1, **i32)
            src = torch.empty(max(1, s["N"]), 2, **i32)
            moe.moe_layout_choices(sh, p, None, s["idx"], torch.empty(c["E"], **i32), offsets, src,
                                   torch.empty(c["R"], c["T"], c["k"], **i32), ws)
            most = moe.moe_max_pairs(sh, p)
            return (sh, p, src, offsets, ws, torch.empty(max(1, s["N"]), c["d"], dtype=torch.uint8, device=DEV),
                    torch.empty(c["d"] // 128, most, 4, dtype=torch.uint8, device=DEV))
        sh, p, src, offsets, ws, xe, xes = _kept(s, "buffers", make)
        moe.moe_dispatch_pull_codes(sh, p, s["xq"], s["xs"], src, offsets, xe, xes, ws)
        return {"codes": xe[:s["N"]].view(torch.float8_e4m3fn), "scales": xes[:, :s["N"]]}
    if c["op"] == "product":
        g, y = _kept(s, "buffers", lambda: (
            moe.Gemm(c["rows"] + c["behind"], c["groups"], c["K"], c["N"], code[c["dtype"]], c["layout"]),
            torch.empty(c["rows"] + c["behind"], c["N"], dtype=s["x"].dtype, device=DEV)))
        moe.moe_grouped_gemm(g, s["x"], s["w"], s["offsets"], y)
        return {"y": y[:c["rows"]]}
    if c["op"] == "prodgrad":
        def make():
            total = c["rows"] + c["behind"]
            forward = moe.Gemm(total, c["groups"], c["K"], c["N"], code[c["dtype"]], c["layout"])
            return (forward, moe.Gemm(total, c["groups"], c["N"], c["K"], code[c["dtype"]], 1 - c["layout"]),
                    torch.empty_like(s["x"]), torch.empty(s["w"].shape, dtype=KINDS[c["dw"]], device=DEV),
                    torch.empty(moe.moe_grouped_gemm_wgrad_workspace_bytes(forward), dtype=torch.uint8, device=DEV))
        g, back, dx, dw, ws = _kept(s, "buffers", make)
        moe.moe_grouped_gemm(back, s["dy"], s["w"], s["offsets"], dx)
        moe.moe_grouped_gemm_wgrad(g, s["x"], s["dy"], s["offsets"], dw, code[c["dw"]], ws)
        return {"dx": dx[:c["rows"]], "dw": dw}

    def make():
        eight = c["states"] == 8
        tensors = []
        for a, n in zip(s["starts"], s["sizes"]):
            b = a + -(-n // 128) * 128
            tensors.append(moe.AdamWTensor(
                s["param"][a:b], s["grad"][a:b], n, code[c["param"]], code[c["grad"]], s["m"][a:b], s["v"][a:b],
                s["ms"][a // 32:b // 32] if eight else None, s["vs"][a // 32:b // 32] if eight else None,
                s["master"][a:b] if s["master"] is not None else None, HYPER["weight_decay"]))
        step = moe.AdamW(HYPER["lr"], HYPER["beta1"], HYPER["beta2"], HYPER["eps"], HYPER["step"],
                         moe.MOE_MXFP8 if eight else moe.MOE_F32, 1 if eight or (c["param"] == "bf16" and not c["master"]) else 0,
                         s["seed"])
        values = [torch.empty(s["total"], dtype=torch.bfloat16, device=DEV) for _ in range(2)] if eight else None
        return step, moe.adamw_table(tensors), values
    step, table, values = _kept(s, "buffers", make)
    moe.moe_adamw(step, table)
    if c["states"] == 32:
        return _step_outputs(s, s["m"], s["v"])
    moe.moe_mx_dequantize(s["m"], s["ms"], moe.MOE_MXFP8, s["total"] // 128, 128, values[0], moe.MOE_BF16)
    moe.moe_mx_dequantize(s["v"], s["vs"], moe.MOE_MXFP8, s["total"] // 128, 128, values[1], moe.MOE_BF16)
    return _step_outputs(s, *values)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------------ 64 bits
def _elements(codes):
    """What E4M3 codes stand for, in 64 bits, by their fields."""
    c = codes.long()
    field, part = (c >> 3) & 15, (c & 7).double() / 8
    size = torch.where(field > 0, (1 + part) * torch.exp2(field.double() - 7), part * 2.0 ** -6)
    return torch.where(c >= 128, -size, size)


def _e4m3(v, part, unit):
    """v in E4M3 with a block's unit, `part` of a step added before what is left of a step is cut off (None: nearest even)."""
    y = v.abs().unflatten(-1, (-1, 32)) / unit
    step = torch.clamp(torch.exp2(torch.frexp(y).exponent.double() - 4), min=2.0 ** -9)
    q = torch.round(y / step) if part is None else torch.floor(y / step + part.reshape(y.shape))
    return (torch.clamp(q * step, max=448) * unit).flatten(-2) * torch.sign(v)


def _unit(v, most):
    """The scale of each block of 32: at most 2^-8 of the largest magnitude, twice that where it would pass `most`."""
    top = v.abs().unflatten(-1, (-1, 32)).max(-1, keepdim=True).values
    unit = torch.exp2((torch.frexp(top).exponent.double() - 9).clamp(-127, 127))
    return torch.where(top / unit > most, 2 * unit, unit)


def exact(case, seed):
    """The definitions in 64 bits."""
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "norm":
        out = {"y": [], "h": [], "codes": []}
        for i in range(0, c["rows"], 4096):
            t = s["x"][i:i + 4096].double()
            if c["residual"]:
                t = t + s["residual"][i:i + 4096].double()
            length = torch.linalg.vector_norm(t, dim=1, keepdim=True) / math.sqrt(c["d"])
            out["h"].append(t.float() if c["dtype"] == "bf16" else t)
            out["y"].append(t / torch.sqrt(length ** 2 + 1e-6) * s["gamma"].double())
            if c["codes"]:
                out["codes"].append(_e4m3(out["y"][-1], None, _unit(out["y"][-1], 512)))
        return {k: torch.cat(v).double() for k, v in out.items() if v and (k != "h" or c["residual"])}
    if c["op"] == "normgrad":
        dx, dgamma = [], torch.zeros(c["d"], dtype=torch.double, device=DEV)
        for i in range(0, c["rows"], 4096):
            h, dy = s["h"][i:i + 4096].double(), s["dy"][i:i + 4096].double()
            q = (h * h).sum(1, keepdim=True) / c["d"] + 1e-6
            u = dy * s["gamma"].double()
            r = u / torch.sqrt(q) - h * ((u * h).sum(1, keepdim=True) / c["d"] / q ** 1.5)
            dx.append(r + s["dh"][i:i + 4096].double() if c["residual"] else r)
            dgamma += (dy * h / torch.sqrt(q)).sum(0)
        return {"dx": torch.cat(dx), "dgamma": dgamma}
    if c["op"] == "dispatch":
        rank, token = (s["pull_src"][:s["N"], i].long() for i in (0, 1))
        out = torch.empty(s["N"], c["d"], dtype=torch.double, device=DEV)
        for r in range(c["R"]):
            mine = rank == r
            out[mine] = _elements(s["xq"][r][token[mine]])
        return {"codes": out, "scales": None}
    if c["op"] in ("product", "prodgrad"):
        if work(case)["flops"] > 1.2e12:
            return None
        off = s["offsets"].tolist()
        rows, N, K = c["rows"], c["N"], c["K"]
        y = torch.zeros(rows, N if c["op"] == "product" else K, dtype=torch.double, device=DEV)
        dw = torch.zeros(s["w"].shape, dtype=torch.double, device=DEV) if c["op"] == "prodgrad" else None
        for i, (a, b) in enumerate(zip(off, off[1:])):
            if a == b:
                continue
            w = s["w"][i].double() if c["layout"] == 0 else s["w"][i].double().T
            x = s["x"][a:b].double()
            if c["op"] == "product":
                y[a:b] = x @ w.T
                continue
            dy = s["dy"][a:b].double()
            y[a:b] = dy @ w
            t = dy.T @ x
            dw[i] = t if c["layout"] == 0 else t.T
        return {"y": y} if dw is None else {"dx": y, "dw": dw}
    p = (s["param"] if s["master"] is None else s["master"]).double()
    g = s["grad"].double()
    if c["states"] == 32:
        m, v = s["m"].double(), s["v"].double()
    else:
        unit = [torch.exp2(s[k].double() - 127).repeat_interleave(32) for k in ("ms", "vs")]
        m, v = _elements(s["m"]) * unit[0], (_elements(s["v"]) * unit[1]) ** 2
    b1, b2, t = HYPER["beta1"], HYPER["beta2"], HYPER["step"]
    m += (1 - b1) * (g - m)
    v += (1 - b2) * (g * g - v)
    p -= HYPER["lr"] * HYPER["weight_decay"] * p
    p -= HYPER["lr"] * (m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + HYPER["eps"])
    out = {"param": p, "m": m, "v": v}
    if c["states"] == 8:
        r, v = _bits(s, 0), torch.sqrt(v)
        out["m"] = _e4m3(m, (r & 0xFFFF).double() / 65536, _unit(m, 448))
        unit = _unit(v, 448)
        up = _e4m3(v, (r >> 16).double() / 65536, unit).unflatten(-1, (-1, 32))
        out["v"] = torch.where((v.unflatten(-1, (-1, 32)) > 0) & (up == 0), 2.0 ** -9 * unit, up).flatten(-2)
    return out if s["master"] is None else dict(out, master=p)
