"""GPU parity of MXFP4: the codec bit for bit, and the expert path against its 64-bit formula.

Bars.  Codec: bit-exact.  Expert outputs: every element of ye lies within what its own
arithmetic allows, derived per element (_bound): the h codes that may legitimately differ
from the 64-bit h's -- those whose value lies closer to an E2M1 midpoint (or whose block
maximum lies closer to a power of two) than the fp32 error of h -- times W2, the fp32
accumulation of the down product, and one bf16 rounding (2^-8 of the value: half a step).
A dropped block, a wrong scale or nibble order moves outputs by tens of percent.
"""
import numpy as np
import pytest

from oracle import moe_oracle as O
from oracle import mx4_oracle as M4
from oracle import mx_oracle as M8
from mixture_experts_layer_histogram_amd import configs, inputs, moe

pytestmark = pytest.mark.gpu

GUARD = 0x5A


def _torch():
    import torch
    return torch


def _rowmajor(scales, rows, K):
    """Scale codes [rows][K/32] of the plane-wise device layout [K/128][rows][4]."""
    return scales.reshape(K // 128, rows, 4).transpose(1, 0, 2).reshape(rows, K // 32)


def _gpu_quantize(v, src, fmt=moe.MOE_MXFP4):
    """moe_mx_quantize_to of rows of fp32 values; codes and scales lie between guard bytes."""
    torch = _torch()
    rows, K = v.shape
    x = torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).cuda()
    if src == "bf16":
        x = x.to(torch.bfloat16)
        assert np.array_equal(x.float().cpu().numpy(), v, equal_nan=True), "inputs must be bf16 values"
    nb = rows * K // (2 if fmt == moe.MOE_MXFP4 else 1)
    q = torch.full((nb + 256,), GUARD, dtype=torch.uint8, device="cuda")
    s = torch.full((rows * K // 32 + 256,), GUARD, dtype=torch.uint8, device="cuda")
    moe.moe_mx_quantize_to(x, moe.MOE_BF16 if src == "bf16" else moe.MOE_F32, rows, K, fmt, q, s)
    q, s = q.cpu().numpy(), s.cpu().numpy()
    assert (q[nb:] == GUARD).all() and (s[rows * K // 32:] == GUARD).all()
    return q[:nb].reshape(rows, -1), _rowmajor(s[: rows * K // 32], rows, K)


def _bf16_values():
    return (np.arange(65536, dtype=np.uint32) << 16).view(np.float32).copy()


# --------------------------------------------------------------------------- codec
@pytest.mark.parametrize("order", ["natural", "shuffled", "near", "finite"])
def test_quantize_every_bf16_value(order):
    v = _bf16_values()
    if order == "finite":
        v[~np.isfinite(v)] = 0.0
    if order == "shuffled":                       # almost every block has an infinity, a NaN or a huge value
        v = v[np.random.default_rng(1).permutation(v.size)]
    elif order == "near":                         # blocks of neighbouring magnitudes
        v = v[np.argsort(np.abs(v), kind="stable")].reshape(-1, 32)
        v = v[np.random.default_rng(2).permutation(len(v))].reshape(-1)
    v = v.reshape(-1, 1024)
    codes, scales = _gpu_quantize(v, "bf16")
    rc, rs, _ = M4.quantize(v)
    assert np.array_equal(scales, rs)
    assert np.array_equal(M4.unpack(codes), rc)


@pytest.mark.parametrize("src", ["bf16", "f32"])
def test_quantize_midpoints_at_every_scale(src):
    """Values on and next to every midpoint, blocks scaled by every power of two of the type."""
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.5, 0.5, 1.0, 3.0, 0.125, 0.0])
    if src == "f32":
        m32 = mids.astype(np.float32)
        base = np.concatenate([mids, np.nextafter(m32, np.float32(0)), np.nextafter(m32, np.float32(9))])[:31]
    else:
        base = np.concatenate([mids, mids[:7] * (1 + 2.0 ** -7), mids[:7] * (1 - 2.0 ** -7)])[:31]
    rng = np.random.default_rng(3)
    blocks = []
    for e in range(-149, 126):
        b = np.concatenate([[4.0 + rng.integers(0, 4)], rng.permutation(np.resize(base, 31))])
        blocks.append(np.ldexp(b * np.where(rng.random(32) < 0.5, -1.0, 1.0), e))
    blocks += [np.zeros(32)] * ((-len(blocks)) % 4)
    v = np.array(blocks).astype(np.float32).reshape(-1, 128)
    if src == "bf16":
        v = inputs.f32_to_bf16_bits(v).astype(np.uint32)
        v = (v << 16).view(np.float32).reshape(-1, 128)
    codes, scales = _gpu_quantize(v, src)
    rc, rs, _ = M4.quantize(v)
    assert np.array_equal(scales, rs)
    assert np.array_equal(M4.unpack(codes), rc)


@pytest.mark.parametrize("rows,K", [(1, 128), (1, 7168), (31, 384), (32, 512), (33, 640), (65, 1408), (257, 128)])
@pytest.mark.parametrize("src", ["bf16", "f32"])
def test_quantize_dequantize_shapes(rows, K, src):
    torch = _torch()
    rng = np.random.default_rng(rows * K)
    v = rng.standard_normal((rows, K)).astype(np.float32)
    v[rng.random((rows, K // 32)).repeat(32, 1) < 0.1] = 0.0          # whole zero blocks
    if src == "bf16":
        v = (inputs.f32_to_bf16_bits(v).astype(np.uint32) << 16).view(np.float32).reshape(rows, K)
    v[rows // 2, 5], v[0, K - 1] = np.nan, -np.inf
    for fmt in (moe.MOE_MXFP4, moe.MOE_MXFP8):
        w = v if fmt == moe.MOE_MXFP4 else np.nan_to_num(v, nan=0.0, neginf=0.0)
        codes, scales = _gpu_quantize(w, src, fmt)
        rc, rs, want = M4.quantize(w) if fmt == moe.MOE_MXFP4 else M8.quantize(w)
        assert np.array_equal(M4.unpack(codes) if fmt == moe.MOE_MXFP4 else codes, rc) and np.array_equal(scales, rs)
        planes = torch.from_numpy(np.ascontiguousarray(rs.reshape(rows, K // 128, 4).transpose(1, 0, 2))).cuda()
        for code, kind in ((moe.MOE_BF16, torch.bfloat16), (moe.MOE_F32, torch.float32)):
            out = torch.full((rows * K + 64,), 7.0, dtype=kind, device="cuda")
            moe.moe_mx_dequantize(torch.from_numpy(codes.copy()).cuda(), planes, fmt, rows, K, out, code)
            assert (out[rows * K:] == 7.0).all()
            assert np.array_equal(out[: rows * K].double().cpu().numpy().reshape(rows, K), want, equal_nan=True)


def test_more_rows_than_a_launch_has_workgroups():
    """134 million rows of 128: workgroups take several blocks of rows (checked around the seam and at the end)."""
    torch = _torch()
    rows, K = (1 << 22) * 32 + 37, 128
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    places = [slice(0, 40), slice((1 << 22) * 32 - 40, rows)]
    g = torch.Generator(device="cuda").manual_seed(3)
    for p in places:
        x[p] = torch.randn(x[p].shape, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.full((rows, K // 2), GUARD, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, 4), GUARD, dtype=torch.uint8, device="cuda")
    moe.moe_mx_quantize_to(x, moe.MOE_BF16, rows, K, moe.MOE_MXFP4, q, s)
    values = []
    for p in places:
        codes, sc, val = M4.quantize(x[p].double().cpu().numpy())
        assert np.array_equal(M4.unpack(q[p].cpu().numpy()), codes) and np.array_equal(s[p].cpu().numpy(), sc)
        values.append(val)
    assert not q[40:(1 << 22) * 32 - 40].any() and not s[40:(1 << 22) * 32 - 40].any()
    x.fill_(float("nan"))
    moe.moe_mx_dequantize(q, s, moe.MOE_MXFP4, rows, K, x, moe.MOE_BF16)
    for p, val in zip(places, values):
        assert np.array_equal(x[p].double().cpu().numpy(), val)
    assert not x[40:(1 << 22) * 32 - 40].any()


@pytest.mark.parametrize("fmt", [moe.MOE_MXFP4, moe.MOE_MXFP8])
def test_dequantize_every_code_at_every_scale(fmt):
    torch = _torch()
    if fmt == moe.MOE_MXFP4:
        q = M4.unpack(np.arange(256, dtype=np.uint8)[None])[0]                 # every byte: 512 codes
        elem, stored = M4.e2m1_decode(q), np.arange(256, dtype=np.uint8)
    else:
        stored = np.arange(256, dtype=np.uint8)
        elem = M8.e4m3_decode(stored)
    K = elem.size
    codes = np.tile(stored, (256, 1))
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], K // 32, axis=1)
    planes = torch.from_numpy(np.ascontiguousarray(scales.reshape(256, K // 128, 4).transpose(1, 0, 2))).cuda()
    with np.errstate(over="ignore"):
        want = torch.from_numpy((elem[None] * M4.scale_value(scales[:, :1])).astype(np.float32))   # exact, or infinite
    for code, kind in ((moe.MOE_F32, torch.float32), (moe.MOE_BF16, torch.bfloat16)):
        out = torch.empty(256, K, dtype=kind, device="cuda")
        moe.moe_mx_dequantize(torch.from_numpy(codes).cuda(), planes, fmt, 256, K, out, code)
        assert torch.equal(torch.nan_to_num(out.cpu().float(), nan=12345.0),
                           torch.nan_to_num(want.to(kind).float(), nan=12345.0))


# --------------------------------------------------------------------------- expert products
def _cfg(name, **kw):
    base = dict(R=1, T=64, d=256, E=8, E_local=8, k=2, F=256, dtype="mxfp4")
    base.update(kw)
    return configs.DSV3_MX.scaled(name=name, **base)


CASES = {
    "one-token": _cfg("mx4 one token", T=1, d=256, F=128),
    "one-token-wide": _cfg("mx4 one token d1408", T=1, d=1408, F=640, E=16, E_local=16, k=6),
    "k1-one-expert": _cfg("mx4 one expert", T=7, d=128, F=128, E=1, E_local=1, k=1),
    "half-tails": _cfg("mx4 half tails", R=2, T=45, d=384, F=1408, E=4, E_local=2, k=2),
    "rows-33": _cfg("mx4 rows 33", T=33, d=640, F=384, E=1, E_local=1, k=1),
    "rows-64": _cfg("mx4 rows 64", T=64, d=512, F=256, E=1, E_local=1, k=1),
    "rows-129": _cfg("mx4 rows 129", T=129, d=256, F=512, E=1, E_local=1, k=1),
    "rows-257": _cfg("mx4 rows 257", T=257, d=1152, F=128, E=2, E_local=2, k=2),
    "several-tiles": _cfg("mx4 several tiles", R=2, T=600, d=1024, F=512, E=16, E_local=8, k=4),
    "skew": _cfg("mx4 skew", R=2, T=256, d=768, F=384, E=32, E_local=8, k=4, load="skew"),
}


def _problem(cfg, seed=0, mutate=None):
    from mixture_experts_layer_histogram_amd.device import DeviceProblem
    inp = inputs.make_inputs(cfg, seed=seed)
    if mutate:
        mutate(inp)
    return inp, DeviceProblem(cfg, inp)


def _bound(x, w1, w3, w2):
    """(ye, per-element allowance without the bf16 rounding) of one expert in 64 bits.  The MFMA adds
    64 exact products at a time to an fp32 accumulator: K / 64 roundings, each at most 2^-23 of the
    running sum of magnitudes (a truncating adder's step), and the scale product; exp and the quotient of
    silu: (|a| + 8) 2^-22 relative."""
    a, b = x @ w1.T, x @ w3.T
    ax, aw1, aw3 = np.abs(x), np.abs(w1), np.abs(w3)
    n = x.shape[1] / 64 + 4
    da, db = n * 2.0 ** -23 * (ax @ aw1.T), n * 2.0 ** -23 * (ax @ aw3.T)
    h = O.silu(a) * b
    dh = 1.1 * da * np.abs(b) + np.abs(O.silu(a)) * db + (np.abs(a) + 8) * 2.0 ** -22 * np.abs(h) + 2.0 ** -130
    _, sc, hq = M4.quantize(h)
    scale = np.repeat(M4.scale_value(sc), 32, axis=-1)
    y, dy = np.abs(h) / scale, dh / scale
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    steps = np.array([0.5, 0.5, 0.5, 0.5, 1.0, 1.0, 2.0])
    near = np.abs(y[..., None] - mids) <= dy[..., None]
    slack = (near * steps).sum(-1) * scale
    hb = np.abs(h).reshape(*h.shape[:-1], -1, 32)
    top = hb.max(-1)
    dtop = np.take_along_axis(dh.reshape(hb.shape), hb.argmax(-1)[..., None], -1)[..., 0]
    _, e_lo = np.frexp(np.maximum(top - dtop, 0))
    _, e_hi = np.frexp(top + dtop)
    moved = np.repeat(e_lo != e_hi, 32, axis=-1)                 # the block's scale may differ: up to 2 units either side
    slack = np.where(moved, 8 * scale, slack)
    aw2 = np.abs(w2)
    acc = (w2.shape[1] / 64 + 4) * 2.0 ** -23 * ((np.abs(hq) + slack) @ aw2.T)
    return hq @ w2.T, slack @ aw2.T + acc


def _weights64(P):
    """The device's packed weights in 64 bits, and that they are the oracle's quantisation."""
    out = []
    for w, q, s in zip((P.w1, P.w3, P.w2), P.wq, P.ws_codes):
        El, rows, K = w.shape
        v = w.float().cpu().numpy().astype(np.float64).reshape(El * rows, K)
        codes, sc, val = M4.quantize(v)
        assert np.array_equal(M4.unpack(q.cpu().numpy().reshape(El * rows, K // 2)), codes)
        assert np.array_equal(_rowmajor(s.cpu().numpy().reshape(-1), El * rows, K), sc)
        out.append(val.reshape(El, rows, K))
    return out


def _check_rows(P, ye, x64, w):
    """Every row of ye (device, bf16) within its bound; returns the 64-bit rows and their allowance."""
    off = P.offsets.cpu().numpy()
    N = int(off[-1])
    ref, allowed = np.zeros((N, x64.shape[-1])), np.zeros((N, x64.shape[-1]))
    src = P.pull_src.cpu().numpy()
    got = ye[:N].double().cpu().numpy()
    for l in range(len(off) - 1):
        a, b = int(off[l]), int(off[l + 1])
        if a == b:
            continue
        rows = M4.quantize(x64[src[a:b, 0], src[a:b, 1]])[2]
        ref[a:b], allow = _bound(rows, w[0][l], w[1][l], w[2][l])
        allowed[a:b] = allow
        err = np.abs(got[a:b] - ref[a:b])
        lim = allow + (np.abs(ref[a:b]) + allow) * 2.0 ** -8 + 1e-38
        assert (err <= lim).all(), (l, float((err / lim).max()), np.argwhere(err > lim)[:4].tolist())
    return ref, allowed


def _check_merged(P, ref, allowed, wgt):
    """y of expert rows in fp32: the rows' allowance under the weights, at most k fused multiply-adds, and
    one bf16 rounding."""
    slot, w = P.slot_of.cpu().numpy(), wgt.double().cpu().numpy()
    k = slot.shape[-1]
    at = np.where(slot >= 0, slot, 0)
    w = np.where(slot >= 0, w, 0.0)[..., None]
    want = (w * ref[at]).sum(-2)
    room = (np.abs(w) * allowed[at]).sum(-2) + k * 2.0 ** -24 * (np.abs(w) * (np.abs(ref[at]) + allowed[at])).sum(-2)
    for r, t in enumerate(P.y):
        err = np.abs(t.double().cpu().numpy() - want[r])
        lim = room[r] + (np.abs(want[r]) + room[r]) * 2.0 ** -8 + 1e-38
        assert (err <= lim).all(), (r, float((err / lim).max()))


def _rows32(P):
    """The shapes whose expert rows moe_forward_choices keeps in fp32."""
    return P.nmax * P.cfg.d * 4 <= 16 << 20


@pytest.mark.parametrize("name", sorted(CASES))
def test_expert_rows_within_their_bounds(name):
    torch = _torch()
    cfg = CASES[name]
    print(f"[mx4] {cfg.name}", flush=True)
    inp, P = _problem(cfg)
    P.xe.fill_(GUARD)
    P.ye.fill_(3.0)
    P.xe_scales.fill_(GUARD)
    P.forward()
    assert P.status() == 0
    torch.cuda.synchronize()
    N = int(P.offsets[-1])
    x64 = np.stack([P.rows_f64(t) for t in P.x]).reshape(cfg.R, cfg.T, cfg.d)
    src = P.pull_src.cpu().numpy()[:N]
    codes, sc, _ = M4.quantize(x64[src[:, 0], src[:, 1]])
    assert np.array_equal(M4.unpack(P.xe[:N].cpu().numpy()), codes)
    assert np.array_equal(P.xe_scales[:, :N].permute(1, 0, 2).reshape(N, -1).cpu().numpy(), sc)
    assert (P.xe[N:] == GUARD).all() and (P.xe_scales[:, N:] == GUARD).all() and (P.ye[N:] == 3.0).all()
    w = _weights64(P)
    ref, allowed = _check_rows(P, P.ye, x64, w)
    err = np.linalg.norm(P.ye[:N].double().cpu().numpy() - ref) / np.linalg.norm(ref)
    print(f"[mx4] {cfg.name}: N {N}, relative error {err:.2e}", flush=True)
    assert err <= 5e-3                      # the header's figure
    # the fused path gives the same bits, and the path for given choices too, or rounds once
    y = [t.clone() for t in P.y]
    for t in P.y:
        t.fill_(float("nan"))
    P.forward_fused()
    assert P.status() == 0 and all(torch.equal(a, b) for a, b in zip(y, P.y))
    idx, wgt, lay = P.topk_idx.clone(), P.topk_w.clone(), P.slot_of.clone()
    for t in P.y:
        t.fill_(float("nan"))
    P.ye.fill_(float("nan"))
    P.forward_choices(idx, wgt)
    assert P.status() == 0 and torch.equal(lay, P.slot_of)
    if _rows32(P):
        assert torch.isnan(P.ye).all()
        _check_merged(P, ref, allowed, wgt)
    else:
        assert all(torch.equal(a, b) for a, b in zip(y, P.y))


def _check_some_rows(P, ye, rows, w):
    """The given rows of ye within their bounds."""
    off = P.offsets.cpu().numpy()
    src = P.pull_src.cpu().numpy()
    for l in range(len(off) - 1):
        r = rows[(rows >= off[l]) & (rows < off[l + 1])]
        if not len(r):
            continue
        x = np.stack([P.x[src[i, 0]][src[i, 1]].double().cpu().numpy() for i in r])
        ref, allow = _bound(M4.quantize(x)[2], w[0][l], w[1][l], w[2][l])
        err = np.abs(ye[r].double().cpu().numpy() - ref)
        lim = allow + (np.abs(ref) + allow) * 2.0 ** -8 + 1e-38
        assert (err <= lim).all(), (l, float((err / lim).max()), r[np.argwhere(err > lim)[:4, 0]].tolist())


def _push(P, idx, wgt):
    """The choices' layer with the push fused into the down product; the merged rows."""
    torch = _torch()
    w1, w3, w2 = P.weights()
    for t in P.recv:
        t.fill_(float("nan"))
    moe.moe_layout_choices(P.shape, P.placement, P.ex, idx, P.counts, P.offsets, P.pull_src, P.slot_of, P.ws)
    P.dispatch()
    moe.moe_expert_ffn_push(P.shape, P.placement, P.ex, P.xe, P.offsets, w1, w3, w2, P.pull_src, P.slot_of, P.recv, P.ws,
                            w_scales=P.w_scales, xe_scales=P.xe_scales)
    y = [torch.full_like(t, float("nan")) for t in P.y]
    moe.moe_weighted_merge(P.shape, P.placement, P.slot_of, wgt, P.recv, y)
    return y


@pytest.mark.parametrize("T,d,F,E,k", [(26000, 512, 1024, 4, 1), (140000, 256, 128, 4, 1), (9000, 1152, 896, 8, 4)])
def test_many_tiles_a_workgroup(T, d, F, E, k):
    """Three and more tiles a workgroup, whole and partial ones in turn, of one, two and several stages, with
    half stages and half columns: the next tile's fills run under the last one's stores."""
    torch = _torch()
    cfg = _cfg(f"mx4 many tiles T{T} d{d} F{F} E{E} k{k}", T=T, d=d, F=F, E=E, E_local=E, k=k)
    print(f"[mx4] {cfg.name}", flush=True)
    inp, P = _problem(cfg)
    P.ye.fill_(float("nan"))
    P.forward()
    assert P.status() == 0
    off = P.offsets.cpu().numpy()
    N = int(off[-1])
    assert N == T * k and torch.isfinite(P.ye[:N]).all()
    edges = np.concatenate([np.concatenate([np.arange(a, b, 256), np.arange(a, b, 256) + 255]) for a, b in zip(off, off[1:])])
    rows = np.unique(np.concatenate([edges[edges < N][:: max(1, len(edges) // 400)], [0, N - 1],
                                     np.random.default_rng(3).integers(0, N, 200)]))
    _check_some_rows(P, P.ye, rows, _weights64(P))
    y = [t.clone() for t in P.y]
    for _ in range(3):                        # the same bits whatever the timing, and through the fused push
        P.ye.fill_(float("nan"))
        P.forward_choices(P.topk_idx.clone(), P.topk_w.clone())
        assert all(torch.equal(a, b) for a, b in zip(y, P.y))
    assert all(torch.equal(a, b) for a, b in zip(y, _push(P, P.topk_idx.clone(), P.topk_w.clone())))


@pytest.mark.parametrize("d", [384, 2176, 7168, 8320])
def test_gather_of_more_rows_than_workgroups(d):
    """Codes and scales bit for bit where workgroups take several rows, and rows wider than a wave holds."""
    torch = _torch()
    cfg = _cfg(f"mx4 gather d{d}", T=3000, d=d, F=128, E=5, E_local=4, k=2)
    print(f"[mx4] {cfg.name}", flush=True)
    inp, P = _problem(cfg)
    P.xe.fill_(GUARD)
    P.xe_scales.fill_(GUARD)
    P.layout()
    P.dispatch()
    assert P.status() == 0
    N = int(P.offsets[-1])
    assert 4096 < N < P.nmax
    codes, sc, _ = M4.quantize(P.rows_f64(P.x[0]).reshape(cfg.T, d))
    src = P.pull_src.cpu().numpy()[:N, 1]
    assert np.array_equal(M4.unpack(P.xe[:N].cpu().numpy()), codes[src])
    assert np.array_equal(P.xe_scales[:, :N].permute(1, 0, 2).reshape(N, -1).cpu().numpy(), sc[src])
    assert (P.xe[N:] == GUARD).all() and (P.xe_scales[:, N:] == GUARD).all()


def test_few_and_many_rows_in_one_call():
    """Experts of 100, 33, 32, 31, 1 and 0 rows where few are expected: each of the two product kernels
    takes its own."""
    torch = _torch()
    cfg = _cfg("mx4 few and many rows", T=100, d=640, F=384, E=16, E_local=16, k=2)
    inp, P = _problem(cfg)
    idx = np.full((1, 100, 2), -1, dtype=np.int32)
    idx[0, :, 0] = 0
    for e, (a, b) in enumerate([(0, 33), (33, 65), (65, 96), (96, 97)], start=1):
        idx[0, a:b, 1] = e
    idx = torch.from_numpy(idx).cuda()
    wgt = torch.rand(1, 100, 2, device="cuda") - 0.5
    P.ye.fill_(3.0)
    pushed = _push(P, idx, wgt)[0]
    P.ffn()
    assert P.status() == 0 and P.counts.tolist() == [100, 33, 32, 31, 1] + [0] * 11
    N = int(P.offsets[-1])
    assert (P.ye[N:] == 3.0).all()
    x64 = P.rows_f64(P.x[0]).reshape(1, cfg.T, cfg.d)
    ref, allowed = _check_rows(P, P.ye, x64, _weights64(P))
    moe.moe_combine_merge(P.shape, P.placement, P.ye, P.slot_of, wgt, P.y)
    assert torch.equal(P.y[0], pushed)
    P.forward_choices(idx, wgt)
    assert _rows32(P)
    _check_merged(P, ref, allowed, wgt)


def test_tokens_without_a_value_stay_apart():
    """A NaN, an infinity or both in a token's row makes that token NaN and touches no other."""
    torch = _torch()
    cfg = _cfg("mx4 non-finite tokens", T=70, d=512, F=256, E=4, E_local=4, k=2)
    inp, P = _problem(cfg)
    P.forward()
    P.forward_choices(P.topk_idx.clone(), P.topk_w.clone())
    clean = P.y[0].clone()
    x = P.x[0].clone()
    P.x[0][3, 17] = float("nan")
    P.x[0][40, 511] = float("inf")
    P.x[0][69, 0], P.x[0][69, 1] = float("-inf"), float("nan")
    P.forward_choices(P.topk_idx.clone(), P.topk_w.clone())
    bad = [3, 40, 69]
    assert torch.isnan(P.y[0][bad]).all()
    good = [t for t in range(70) if t not in bad]
    assert torch.equal(P.y[0][good], clean[good])
    P.x[0].copy_(x)
    P.forward_choices(P.topk_idx.clone(), P.topk_w.clone())
    assert torch.equal(P.y[0], clean)


def test_zero_and_extreme_rows():
    """Rows of zeros give zeros; rows at the ends of bf16's range keep their scales."""
    torch = _torch()
    cfg = _cfg("mx4 extreme rows", T=8, d=256, F=128, E=2, E_local=2, k=1)
    inp, P = _problem(cfg)
    P.x[0][0] = 0.0
    P.x[0][1] *= 2.0 ** -120
    P.x[0][2] *= 2.0 ** 60
    P.forward()
    assert (P.y[0][0] == 0).all()
    x64 = P.rows_f64(P.x[0]).reshape(1, 8, 256)
    codes = M4.quantize(x64[0])[0]
    src = P.pull_src.cpu().numpy()[:, 1]
    assert np.array_equal(M4.unpack(P.xe.cpu().numpy()), codes[src])
    assert torch.isfinite(P.y[0][[0, 1, 3, 4, 5, 6, 7]]).all()


def test_no_local_rows_and_all_dropped():
    torch = _torch()
    cfg = _cfg("mx4 nothing", T=5, d=256, F=128, E=8, E_local=2, k=2)
    inp, P = _problem(cfg)
    P.forward_choices(torch.full((1, 5, 2), -1, dtype=torch.int32, device="cuda"), torch.ones(1, 5, 2, device="cuda"))
    assert P.status() == 0 and (P.y[0] == 0).all() and (P.offsets == 0).all() and (P.slot_of == -1).all()
    away = torch.tensor([[[6, 7]] * 5], dtype=torch.int32, device="cuda")        # experts 0 and 1 are local
    P.forward_choices(away, torch.ones(1, 5, 2, device="cuda"))
    assert P.status() == 0 and (P.y[0] == 0).all()
    assert P.counts.tolist() == [0, 0, 0, 0, 0, 0, 5, 5]


def test_graph_replays_and_two_streams():
    torch = _torch()
    cfg = CASES["half-tails"]
    inp, A = _problem(cfg, seed=1)
    _, B = _problem(cfg, seed=2)
    for P in (A, B):
        P.forward()
    ch = [(P.topk_idx.clone(), P.topk_w.clone()) for P in (A, B)]
    for P, c in zip((A, B), ch):
        P.forward_choices(*c)
    want = [[t.clone() for t in P.y] for P in (A, B)]
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        A.forward_choices(*ch[0])
    for i in range(3):
        for P in (A, B):
            for t in P.y:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        other = torch.cuda.Stream()
        B.forward_choices(*ch[1], stream=other)
        torch.cuda.synchronize()
        for P, w in zip((A, B), want):
            assert all(torch.equal(a, b) for a, b in zip(P.y, w)), i


@pytest.mark.parametrize("T", [9, 300])
def test_two_graphs_over_one_workspace(T):
    """Two captured layers with choices of their own over the same buffers, replayed in turn with eager
    calls between: every call leaves its own result, whatever the tables held."""
    torch = _torch()
    cfg = _cfg(f"mx4 two graphs T{T}", T=T, d=512, F=384, E=12, E_local=6, k=3)
    inp, P = _problem(cfg)
    rng = np.random.default_rng(5)
    ch = []
    for drop in (0.0, 0.3, 1.0):
        idx = np.argsort(rng.random((1, T, 12)), -1)[..., :3].astype(np.int32)
        idx[rng.random(idx.shape) < drop] = -1
        ch.append((torch.from_numpy(idx).cuda(), torch.rand(1, T, 3, device="cuda")))
    want = []
    for c in ch:
        P.forward_choices(*c)
        want.append(P.y[0].clone())
    assert not torch.equal(want[0], want[1]) and (want[2] == 0).all()
    graphs = []
    s = torch.cuda.Stream()
    for c in ch[:2]:
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            P.forward_choices(*c)
        graphs.append(g)
    for i in (0, 1, 1, 2, 0, 2, 1):
        P.y[0].fill_(float("nan"))
        if i < 2:
            graphs[i].replay()
        else:
            P.forward_choices(*ch[2])
        torch.cuda.synchronize()
        assert torch.equal(P.y[0], want[i]), i
