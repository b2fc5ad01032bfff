"""Operators of the MoE layer for given expert choices and for 4-bit expert weights, as cases to time and to compare.

Five kinds of case, one for each group of entry points:

  quantise  rows to MXFP4 (E2M1 elements, one E8M0 scale per 32 values) and back to values
  experts   the layer's share for given choices and gate weights, expert products in MXFP4
  sort      the layout of given choices and the token rows in expert order
  merge     expert rows back at their tokens, with the gate weights applied
  grad      the gradients of merge (rows and gate weights) and of sort (token rows)

A pair is one (rank, token, j) choice; it is local if its expert lives on this GPU, and a choice of -1 is no pair.
With `own` false, `run` computes the operators from elementary torch operations in 32 bits; with `own` true it calls the
library.
"""
import math

import torch

own = False

DEV = "cuda:0"


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token's activations as an odd fp32 row block (d of a mid-size layer's F: 11 K tiles)
        {"name": "quantise_f32_37x1408", "op": "quantise", "rows": 37, "K": 1408, "dtype": "f32"},
        # the down weights of a DeepSeek-V3-shaped share, quantised once after loading
        {"name": "quantise_bf16_share_w2", "op": "quantise", "rows": 32 * 7168, "K": 2048, "dtype": "bf16"},
        # one token answered by a mid-size layer: six experts' weights are read, latency counts
        {"name": "experts_one_token", "op": "experts", "R": 1, "T": 1, "d": 2048, "F": 1408, "E": 64, "E_local": 64,
         "k": 6, "drop": 0.0, "skew": 0.0},
        # a decoding batch of the share: 64 tokens of each of 8 ranks, some 16 rows per expert, the weights' bytes count
        {"name": "experts_decode_share", "op": "experts", "R": 8, "T": 64, "d": 7168, "F": 2048, "E": 256,
         "E_local": 32, "k": 8, "drop": 0.0, "skew": 0.0},
        # a prompt of the mid-size layer with a padded tail (its choices are -1), uneven experts
        {"name": "experts_prompt_mid", "op": "experts", "R": 1, "T": 4093, "d": 2048, "F": 1408, "E": 64,
         "E_local": 64, "k": 6, "drop": 0.05, "skew": 0.5},
        # the whole share: 32768 rows on 32 experts
        {"name": "experts_share", "op": "experts", "R": 8, "T": 4096, "d": 7168, "F": 2048, "E": 256, "E_local": 32,
         "k": 8, "drop": 0.0, "skew": 0.0},
        # a few fp32 tokens, some of them dropped
        {"name": "sort_f32_small", "op": "sort", "R": 1, "T": 256, "d": 128, "E": 8, "E_local": 8, "k": 2,
         "dtype": "f32", "drop": 0.1, "skew": 0.0},
        # the share's tokens
        {"name": "sort_bf16_share", "op": "sort", "R": 8, "T": 4096, "d": 7168, "E": 256, "E_local": 32, "k": 8,
         "dtype": "bf16", "drop": 0.0, "skew": 0.5},
        # one decoding step's rows back
        {"name": "merge_f32_decode", "op": "merge", "R": 1, "T": 61, "d": 2048, "E": 64, "E_local": 64, "k": 6,
         "dtype": "f32", "drop": 0.0, "skew": 0.0},
        # a mid-size training step's rows back, every expert local
        {"name": "merge_bf16_mid", "op": "merge", "R": 1, "T": 4096, "d": 2048, "E": 64, "E_local": 64, "k": 6,
         "dtype": "bf16", "drop": 0.0, "skew": 0.5},
        # fp32 gradients of a small layer
        {"name": "grad_f32_small", "op": "grad", "R": 2, "T": 129, "d": 1408, "E": 16, "E_local": 8, "k": 4,
         "dtype": "f32", "drop": 0.1, "skew": 0.0},
        # the share's training step
        {"name": "grad_bf16_share", "op": "grad", "R": 8, "T": 4096, "d": 7168, "E": 256, "E_local": 32, "k": 8,
         "dtype": "bf16", "drop": 0.0, "skew": 0.5},
    ]


MOST_PAIRS = 8 * 4096 * 8 * 32 // 256      # local pairs of the share
MOST_WEIGHTS = 32 * 7168 * 2048            # values of one of its weight tensors


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["quantise", "experts", "experts", "sort", "merge", "grad"])
    if op == "quantise":
        while True:
            c = {"op": op, "rows": spread(1, 32 * 7168), "K": 128 * spread(1, 56), "dtype": rng.choice(["f32", "bf16"])}
            if c["rows"] * c["K"] <= MOST_WEIGHTS // (2 if c["dtype"] == "f32" else 1):
                return c
    while True:
        E = rng.choice([8, 16, 32, 64, 96, 128, 256])
        El = max(1, E // rng.choice([1, 1, 2, 4, 8]))
        c = {"op": op, "R": rng.choice([1, 1, 2, 3, 4, 8]), "T": spread(1, 4096), "d": 128 * spread(1, 56), "E": E,
             "E_local": El, "k": rng.randint(1, 8), "drop": rng.choice([0.0, 0.0, 0.05, 0.3]),
             "skew": rng.choice([0.0, 0.0, 0.5, 1.0])}
        if op == "experts":
            c["F"] = 128 * spread(1, 16)
            if El * c["d"] * c["F"] > MOST_WEIGHTS or (c["skew"] > 0.5 and c["T"] * c["R"] > 4096):
                continue
        else:
            c["dtype"] = rng.choice(["f32", "bf16"])
        if c["R"] * c["T"] * c["k"] * El // E * (2 if c.get("dtype") == "f32" else 1) <= MOST_PAIRS:
            return c


def work(case):
    c = case
    if c["op"] == "quantise":
        n = c["rows"] * c["K"]
        esz = 4 if c["dtype"] == "f32" else 2
        # values in and out, codes and scales written by the one call and read by the other
        return {"bytes": n * (2 * esz + 2 * (0.5 + 1 / 32)), "flops": 0}
    tokens = c["R"] * c["T"]
    pairs = tokens * c["k"] * c["E_local"] / c["E"] * (1 - c["drop"])
    d = c["d"]
    if c["op"] == "experts":
        F = c["F"]
        weights = 3 * min(c["E_local"], pairs) * d * F * (0.5 + 1 / 32)
        return {"bytes": weights + tokens * d * 4 + tokens * c["k"] * 8, "flops": 6 * pairs * d * F}
    esz = 4 if c["dtype"] == "f32" else 2
    read = min(tokens, pairs)                      # tokens with a local pair
    if c["op"] == "sort":
        return {"bytes": (read + pairs) * d * esz + tokens * c["k"] * 8 + pairs * 8, "flops": 0}
    if c["op"] == "merge":
        return {"bytes": (pairs + tokens) * d * esz + tokens * c["k"] * 8, "flops": 2 * pairs * d}
    return {"bytes": (3 * pairs + read + tokens) * d * esz + tokens * c["k"] * 12, "flops": 4 * pairs * d}


# ------------------------------------------------------------------------------------------------ inputs
def _choices(c, g):
    """Distinct experts per token by noisy popularity, gate weights by a softmax, dropped pairs and a padded tail of -1.
    How many pairs an expert has goes by the sizes alone (so that outputs keep their shapes); which tokens and which
    experts they are goes by the seed."""
    R, T, E, El, k = c["R"], c["T"], c["E"], c["E_local"], c["k"]
    same = torch.Generator(device=DEV)
    same.manual_seed(R * T + 7 * E + k)
    score = torch.randn(R, T, E, generator=same, device=DEV) - c["skew"] * torch.log1p(torch.arange(E, device=DEV).float())
    top = torch.topk(score, k, dim=-1)
    idx, w = top.indices, torch.softmax(top.values, dim=-1)
    home = torch.randperm(E, generator=same, device=DEV)[:El]          # the local experts, an arbitrary subset
    names = torch.randperm(E, generator=g, device=DEV)
    e2l = torch.full((E,), -1, dtype=torch.int32, device=DEV)
    e2l[names[home]] = torch.randperm(El, generator=g, device=DEV).int()
    idx = names[idx].to(torch.int32)
    pad = int(T * c["drop"] / 2)
    if c["drop"] > 0:
        idx[torch.rand(R, T, k, generator=same, device=DEV) < c["drop"] / 2] = -1
        idx[:, T - pad:] = -1
    live = torch.arange(R * T, device=DEV).reshape(R, T)[:, :T - pad].reshape(-1)
    moved = torch.arange(R * T, device=DEV)
    moved[live] = live[torch.randperm(live.numel(), generator=g, device=DEV)]
    return idx.reshape(R * T, k)[moved].reshape(R, T, k), w.reshape(R * T, k)[moved].reshape(R, T, k), e2l


def _rows(n, d, dtype, g, scale=1.0):
    return (torch.randn(n, d, generator=g, device=DEV) * scale).to(torch.float32 if dtype == "f32" else torch.bfloat16)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"case": c}
    if c["op"] == "quantise":
        s["v"] = _rows(c["rows"], c["K"], c["dtype"], g, 0.02)
        return s
    R, T, d, E, El = c["R"], c["T"], c["d"], c["E"], c["E_local"]
    dtype = c.get("dtype", "bf16")
    s["idx"], s["w"], s["e2l"] = _choices(c, g)
    if c["op"] in ("experts", "sort"):
        s["x"] = [_rows(T, d, dtype, g) for _ in range(R)]
    lay = _layout(s["idx"], s["e2l"], El, E)
    n = lay["offsets"].tolist()
    s["N"] = n[-1]
    s["cap"] = max(1, max(b - a for a, b in zip(n, n[1:])))
    s["live"] = torch.tensor([e for e in range(El) if n[e + 1] > n[e]] or [0], dtype=torch.long, device=DEV)
    if c["op"] == "experts":
        F = c["F"]
        for name, rows, K in (("w1", F, d), ("w3", F, d), ("w2", d, F)):
            codes = torch.empty(El, rows, K // 2, dtype=torch.uint8, device=DEV)
            scales = torch.empty(K // 128, El * rows, 4, dtype=torch.uint8, device=DEV)
            for e in range(El):
                q, sc = _quantise(_rows(rows, K, "f32", g, K ** -0.5))
                codes[e] = _pack(q)
                scales[:, e * rows:(e + 1) * rows] = sc.view(rows, K // 128, 4).transpose(0, 1)
            s[name], s[name + "s"] = codes, scales
    if c["op"] in ("merge", "grad"):
        s["slot_of"] = lay["slot_of"]
        s["ye"] = _rows(max(1, s["N"]), d, dtype, g)
    if c["op"] == "grad":
        s["dy"] = [_rows(T, d, dtype, g) for _ in range(R)]
        s["dxe"] = _rows(max(1, s["N"]), d, dtype, g)
    return s


# ------------------------------------------------------------------------------------------------ plain forms
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)      # E2M1's, by code


def _quantise(v):
    """MXFP4 of the last axis in blocks of 32: codes 0..15 (sign in bit 3) and the scales' E8M0 codes.  A block's scale
    is 2^(floor(log2 max) - 2); a value takes the nearest magnitude, ties to the even code, at most 6."""
    b = v.float().reshape(v.shape[0], -1, 32)
    m = b.abs().amax(-1)
    e = (torch.frexp(m).exponent - 3).clamp(-127, 127)
    sc = torch.where(m > 0, e + 127, torch.zeros_like(e))
    y = torch.ldexp(b, -e[..., None]).abs()
    q = torch.zeros_like(y, dtype=torch.uint8)
    for i, mid in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        q += (y > mid) if i % 2 == 0 else (y >= mid)
    q += 8 * (torch.signbit(b) & (m[..., None] > 0)).to(torch.uint8)
    return q.reshape(v.shape), sc.to(torch.uint8)


def _pack(q):
    return q[:, 0::2] | (q[:, 1::2] << 4)


def _values(q, sc):
    """Codes (one a byte) and scale codes as fp32 values."""
    table = torch.tensor(MAGNITUDES + tuple(-x for x in MAGNITUDES), device=q.device)
    v = table[q.int()].reshape(q.shape[0], -1, 32)
    return torch.ldexp(v, sc.int()[..., None] - 127).reshape(q.shape)


def _weight(codes, scales, live):
    """fp32 values of the experts in use of a weight tensor [E_local][rows][K] held as packed codes and plane-wise scales."""
    El, rows, half = codes.shape
    codes = codes[live]
    q = torch.stack((codes & 15, codes >> 4), -1).reshape(-1, 2 * half)
    sc = scales.reshape(scales.shape[0], El, rows, 4)[:, live].permute(1, 2, 0, 3).reshape(q.shape[0], half // 16)
    return _values(q, sc).reshape(-1, rows, 2 * half)


def _layout(idx, e2l, El, E):
    """Rows of one expert in ascending (rank, token, j) order, experts in local order."""
    flat = idx.reshape(-1).long()
    some = flat >= 0
    at = flat.clamp(min=0)
    loc = torch.where(some, e2l.long()[at], torch.full_like(flat, -1))
    hot = (loc[:, None] == torch.arange(El, device=idx.device)).int()
    upto = torch.cumsum(hot, 0, dtype=torch.int32)
    total = upto[-1]
    ends = torch.cumsum(total, 0, dtype=torch.int32)
    offsets = torch.cat((torch.zeros_like(ends[:1]), ends))
    local = loc >= 0
    pick = loc.clamp(min=0)
    rank = upto.gather(1, pick[:, None])[:, 0] - 1
    slot = torch.where(local, offsets[pick] + rank, torch.full_like(rank, -1))
    counts = torch.zeros(E, dtype=torch.int32, device=idx.device).index_add_(0, at, some.int())
    return {"counts": counts, "offsets": offsets, "slot_of": slot.reshape(idx.shape).int(), "loc": loc, "rank": rank}


def _by_slot(slot, N, values):
    """values[p] of each local pair p at its slot."""
    out = torch.zeros(N + 1, dtype=values.dtype, device=values.device)     # the last place takes what is not local
    out[torch.where(slot >= 0, slot, torch.full_like(slot, N)).long()] = values
    return out[:N]


def _split(rows, c, dtype):
    return list(rows.to(torch.float32 if dtype == "f32" else torch.bfloat16).reshape(c["R"], c["T"], -1).unbind(0))


def _plain_sort(s):
    c = s["case"]
    lay = _layout(s["idx"], s["e2l"], c["E_local"], c["E"])
    P = s["idx"].numel()
    tok = _by_slot(lay["slot_of"].reshape(-1), s["N"], torch.arange(P, device=DEV) // c["k"])
    src = torch.stack((tok // c["T"], tok % c["T"]), 1).int()
    return lay, tok, src


def _plain_merge(ye, slot, w):
    """sum over j of w ye[slot], fp32; ye has a row of zeros behind the last for pairs that are not local."""
    flat = slot.reshape(-1, slot.shape[-1])
    at = torch.where(flat >= 0, flat, torch.full_like(flat, ye.shape[0] - 1)).long()
    y = torch.zeros(flat.shape[0], ye.shape[1], device=ye.device)
    for j in range(flat.shape[1]):
        row = ye[at[:, j]].float()
        y += row if w is None else row * torch.where(flat[:, j] >= 0, w.reshape(flat.shape)[:, j], torch.zeros(1, device=DEV))[:, None]
    return y


def _zero_row(t):
    return torch.cat((t, torch.zeros(1, t.shape[1], dtype=t.dtype, device=t.device)))


def _plain(s):
    c = s["case"]
    if c["op"] == "quantise":
        q, sc = _quantise(s["v"])
        return {"values": _values(q, sc).to(s["v"].dtype)}
    N = s["N"]
    if c["op"] == "sort":
        lay, tok, src = _plain_sort(s)
        return {"counts": lay["counts"], "offsets": lay["offsets"], "slot_of": lay["slot_of"], "pull_src": src,
                "xe": torch.cat(s["x"])[tok]}
    if c["op"] == "merge":
        return {"y": _split(_plain_merge(_zero_row(s["ye"]), s["slot_of"], s["w"]), c, c["dtype"])}
    if c["op"] == "grad":
        slot = s["slot_of"].reshape(-1)
        P, k = slot.numel(), c["k"]
        dy = torch.cat(s["dy"]).float()
        pair = _by_slot(slot, N, torch.arange(P, device=DEV))
        dye = dy[pair // k] * s["w"].reshape(-1)[pair][:, None]
        dw = torch.zeros(P, device=DEV)
        dw[pair] = (dy[pair // k] * s["ye"][:N].float()).sum(-1)
        dx = _plain_merge(_zero_row(s["dxe"]), s["slot_of"], None)
        return {"dye": dye.to(s["ye"].dtype), "dw": dw.reshape(s["w"].shape), "dx": _split(dx, c, c["dtype"])}
    lay, tok, _ = _plain_sort(s)
    El, d, cap, live = c["E_local"], c["d"], s["cap"], s["live"]
    xq = _values(*_quantise(torch.cat(s["x"])[tok])) if N else torch.zeros(0, d, device=DEV)
    loc = _by_slot(lay["slot_of"].reshape(-1), N, lay["loc"])
    batch = torch.zeros(El, dtype=torch.long, device=DEV)
    batch[live] = torch.arange(live.numel(), device=DEV)
    place = batch[loc] * cap + torch.arange(N, device=DEV) - lay["offsets"].long()[loc]
    pad = torch.zeros(live.numel() * cap, d, device=DEV)
    pad[place] = xq
    pad = pad.reshape(-1, cap, d)
    a = torch.bmm(pad, _weight(s["w1"], s["w1s"], live).transpose(1, 2))
    b = torch.bmm(pad, _weight(s["w3"], s["w3s"], live).transpose(1, 2))
    h = (a / (1 + torch.exp(-a)) * b).flatten(0, 1)
    hq = _values(*_quantise(h)).reshape(a.shape)
    ye = torch.bmm(hq, _weight(s["w2"], s["w2s"], live).transpose(1, 2)).flatten(0, 1)[place]
    return {"y": _split(_plain_merge(_zero_row(ye), lay["slot_of"], s["w"]), c, "bf16")}


# ------------------------------------------------------------------------------------------------ the library's calls
def _kept(s, name, make):
    """Buffers and descriptors that a program makes once."""
    if name not in s:
        s[name] = make()
    return s[name]


def _handle(moe, c, s, dtype):
    p = moe.Placement(s["e2l"].data_ptr(), c["E_local"])
    sh = moe.Shape(c["R"], c["T"], c["d"], c["E"], c["k"], c.get("F", 128), dtype)
    return sh, p


def _layout_buffers(moe, c, s, sh, p):
    i32 = dict(dtype=torch.int32, device=DEV)
    return {"counts": torch.empty(c["E"], **i32), "offsets": torch.empty(c["E_local"] + 1, **i32),
            "pull_src": torch.empty(max(1, s["N"]), 2, **i32), "slot_of": torch.empty(c["R"], c["T"], c["k"], **i32),
            "ws": torch.empty(moe.moe_workspace_bytes(sh, p), dtype=torch.uint8, device=DEV)}


def _own(s):
    from mixture_experts_layer_histogram_amd import moe
    c = s["case"]
    dtypes = {"f32": (moe.MOE_F32, torch.float32), "bf16": (moe.MOE_BF16, torch.bfloat16)}
    if c["op"] == "quantise":
        rows, K = c["rows"], c["K"]
        code = dtypes[c["dtype"]][0]
        q, sc, out = _kept(s, "buffers", lambda: (torch.empty(rows, K // 2, dtype=torch.uint8, device=DEV),
                                                  torch.empty(K // 128, rows, 4, dtype=torch.uint8, device=DEV),
                                                  torch.empty_like(s["v"])))
        moe.moe_mx_quantize_to(s["v"], code, rows, K, moe.MOE_MXFP4, q, sc)
        moe.moe_mx_dequantize(q, sc, moe.MOE_MXFP4, rows, K, out, code)
        return {"values": out}
    R, T, d, N = c["R"], c["T"], c["d"], max(1, s["N"])
    code, kind = dtypes[c.get("dtype", "bf16")]
    if c["op"] == "experts":
        code = moe.MOE_MXFP4
    sh, p = _kept(s, "handle", lambda: _handle(moe, c, s, code))
    if c["op"] == "sort":
        b = _kept(s, "buffers", lambda: dict(_layout_buffers(moe, c, s, sh, p), xe=torch.empty(N, d, dtype=kind, device=DEV)))
        moe.moe_layout_choices(sh, p, None, s["idx"], b["counts"], b["offsets"], b["pull_src"], b["slot_of"], b["ws"])
        moe.moe_dispatch_pull(sh, p, s["x"], b["pull_src"], b["offsets"], b["xe"], b["ws"])
        return {"counts": b["counts"], "offsets": b["offsets"], "slot_of": b["slot_of"], "pull_src": b["pull_src"][:s["N"]],
                "xe": b["xe"][:s["N"]]}
    if c["op"] == "merge":
        y = _kept(s, "buffers", lambda: [torch.empty(T, d, dtype=kind, device=DEV) for _ in range(R)])
        moe.moe_combine_merge(sh, p, s["ye"], s["slot_of"], s["w"], y)
        return {"y": y}
    if c["op"] == "grad":
        b = _kept(s, "buffers", lambda: {"dye": torch.empty_like(s["ye"]), "dw": torch.empty_like(s["w"]),
                                         "dx": [torch.empty(T, d, dtype=kind, device=DEV) for _ in range(R)]})
        moe.moe_combine_merge_backward(sh, p, s["dy"], s["ye"], s["slot_of"], s["w"], b["dye"], b["dw"])
        moe.moe_dispatch_pull_backward(sh, p, s["dxe"], s["slot_of"], b["dx"])
        return {"dye": b["dye"][:s["N"]], "dw": b["dw"], "dx": b["dx"]}
    b = _kept(s, "buffers", lambda: dict(
        _layout_buffers(moe, c, s, sh, p), xe=torch.empty(moe.moe_max_pairs(sh, p), d // 2, dtype=torch.uint8, device=DEV),
        xes=torch.empty(d // 128, moe.moe_max_pairs(sh, p), 4, dtype=torch.uint8, device=DEV),
        ye=torch.empty(N, d, dtype=torch.bfloat16, device=DEV),
        y=[torch.empty(T, d, dtype=torch.bfloat16, device=DEV) for _ in range(R)],
        scales=moe.MXScales(*(s[n].data_ptr() for n in ("w1s", "w3s", "w2s")))))
    moe.moe_forward_choices(sh, p, None, s["idx"], s["w"], s["x"], s["w1"], s["w3"], s["w2"], b["xe"], b["ye"], b["y"],
                            b["counts"], b["offsets"], b["pull_src"], b["slot_of"], b["ws"], w_scales=b["scales"],
                            xe_scales=b["xes"])
    return {"y": b["y"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------------ 64 bits
def _nearest(v):
    """The values that v takes in MXFP4, in 64 bits: the step of E2M1 at |y| is half a unit below 2, then 1, then 2."""
    v = v.double()
    b = v.unflatten(-1, (-1, 32))
    top = b.abs().max(-1, keepdim=True).values
    unit = torch.exp2((torch.floor(torch.log2(top.clamp(min=2.0 ** -1000))) - 2).clamp(-127, 127))
    y = b / unit
    size = y.abs()
    step = torch.where(size < 2, 0.5, torch.where(size < 4, 1.0, 2.0)).double()
    q = torch.minimum(torch.round(size / step) * step, torch.tensor(6.0, dtype=torch.double, device=v.device))
    return (torch.sign(y) * q * unit).flatten(-2)


def _decoded(codes, scales, e):
    """Expert e's weights in 64 bits."""
    rows, half = codes.shape[1:]
    low, high = (codes[e] & 15).long(), (codes[e] >> 4).long()
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.double, device=DEV)
    v = torch.empty(rows, 2 * half, dtype=torch.double, device=DEV)
    v[:, 0::2], v[:, 1::2] = table[low], table[high]
    unit = torch.exp2(scales[:, e * rows:(e + 1) * rows].permute(1, 0, 2).reshape(rows, -1).double() - 127)
    return v * unit.repeat_interleave(32, 1)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "quantise":
        return {"values": torch.cat([_nearest(v) for v in s["v"].split(1 << 14)])}
    k, T, N = c["k"], c["T"], s["N"]
    if c["op"] in ("sort", "experts"):
        flat = s["idx"].reshape(-1)
        loc = torch.where(flat < 0, -1, s["e2l"][flat.clamp(min=0).long()])
        pairs = torch.nonzero(loc >= 0)[:, 0]
        pairs = pairs[torch.argsort(loc[pairs], stable=True)]
        rows = torch.cat(s["x"]).double()
        if c["op"] == "sort":
            return {"counts": None, "offsets": None, "slot_of": None, "pull_src": None, "xe": rows[pairs // k]}
        y = torch.zeros(c["R"] * T, c["d"], dtype=torch.double, device=DEV)
        gate = s["w"].reshape(-1).double()
        for e in range(c["E_local"]):
            mine = pairs[loc[pairs] == e]
            if not mine.numel():
                continue
            x = _nearest(rows[mine // k])
            a, b = (x @ _decoded(s[n], s[n + "s"], e).T for n in ("w1", "w3"))
            out = _nearest(a * torch.sigmoid(a) * b) @ _decoded(s["w2"], s["w2s"], e).T
            y.index_add_(0, mine // k, out * gate[mine, None])
        return {"y": list(y.reshape(c["R"], T, -1).unbind(0))}
    slot = s["slot_of"].reshape(-1).long()
    pairs = torch.nonzero(slot >= 0)[:, 0]
    at = slot[pairs]
    gate = s["w"].reshape(-1).double()

    def back(rows, g):
        y = torch.zeros(c["R"] * T, c["d"], dtype=torch.double, device=DEV)
        for p in pairs.split(1 << 15):
            y.index_add_(0, p // k, rows[slot[p]].double() * (g[p, None] if g is not None else 1.0))
        return list(y.reshape(c["R"], T, -1).unbind(0))

    if c["op"] == "merge":
        return {"y": back(s["ye"], gate)}
    dy = torch.cat(s["dy"]).double()
    dye = torch.zeros(N, c["d"], dtype=torch.double, device=DEV)
    dw = torch.zeros(slot.numel(), dtype=torch.double, device=DEV)
    dye[at] = dy[pairs // k] * gate[pairs, None]
    dw[pairs] = torch.einsum("nd,nd->n", dy[pairs // k], s["ye"][at].double())
    return {"dye": dye, "dw": dw.reshape(s["w"].shape), "dx": back(s["dxe"], None)}
