"""GPU parity of the layer for given choices and gate weights: the layout bit for bit, the rows
back at their tokens and the gradients against their formulas in 64 bits and against
differences, and all of them together under a router of another kind.

Bars (derived): a merged value is an fp32 chain of at most k fused multiply-adds, each off by at
most 2^-24 of the running sum, which is at most S = sum |w ye|, then one rounding to the row
type (2^-8 of the value in bf16, none in fp32); a row gradient is one product and one rounding;
a weight gradient is a sum of d products in fp32, each lane at most d / 64 + 6 additions long.
"""
import numpy as np
import pytest

from oracle import moe_oracle as O
from oracle import moe_oracle_bwd as OB
from oracle import mx4_oracle as M4
from mixture_experts_layer_histogram_amd import configs, inputs, moe

pytestmark = pytest.mark.gpu

KIND = {"f32": moe.MOE_F32, "bf16": moe.MOE_BF16, "mxfp8": moe.MOE_MXFP8, "mxfp4": moe.MOE_MXFP4}
HALF = {"f32": 0.0, "bf16": 2.0 ** -8}


def _torch():
    import torch
    return torch


def _choices(rng, R, T, E, k, drop):
    idx = np.stack([np.stack([rng.permutation(E)[:k] for _ in range(T)]) for _ in range(R)]).astype(np.int32)
    idx[rng.random(idx.shape) < drop] = -1
    return idx


def _e2l(rng, E, El):
    e2l = np.full(E, -1, dtype=np.int32)
    e2l[rng.permutation(E)[:El]] = np.arange(El, dtype=np.int32)
    return e2l


class Layer:
    """Device buffers of a layout of given choices (no weights)."""

    def __init__(self, R, T, d, E, El, k, dtype, e2l, F=128):
        torch = _torch()
        self.e2l = torch.from_numpy(e2l).cuda()
        self.shape = moe.Shape(R, T, d, E, k, F, KIND[dtype])
        self.pl = moe.Placement(self.e2l.data_ptr(), El)
        n = moe.moe_max_pairs(self.shape, self.pl)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.counts, self.offsets = torch.full((E,), -7, **i32), torch.full((El + 1,), -7, **i32)
        self.pull_src, self.slot_of = torch.full((n, 2), -7, **i32), torch.full((R, T, k), -7, **i32)
        self.ws = torch.full((moe.moe_workspace_bytes(self.shape, self.pl),), 0xA5, dtype=torch.uint8, device="cuda")
        self.nmax = n

    def layout(self, idx, **kw):
        t = idx if not isinstance(idx, np.ndarray) else _torch().from_numpy(idx).cuda()
        moe.moe_layout_choices(self.shape, self.pl, None, t, self.counts, self.offsets, self.pull_src, self.slot_of, self.ws, **kw)
        return moe.moe_read_status(self.ws)


SHAPES = [  # R, T, E, El, k, drop
    (1, 1, 1, 1, 1, 0.0), (1, 1, 8, 8, 2, 0.0), (1, 1, 8, 3, 8, 0.5), (1, 63, 8, 8, 2, 0.1), (2, 65, 16, 5, 4, 0.3),
    (3, 128, 64, 64, 6, 0.0), (1, 200, 256, 32, 8, 0.02), (8, 67, 96, 96, 16, 0.2), (1, 1000, 1024, 1024, 3, 0.0),
    (5, 300, 7, 1, 5, 0.9), (2, 70, 12, 12, 12, 0.0), (1, 4097, 32, 8, 4, 0.05), (2, 33, 8, 4, 2, 1.0),
]


@pytest.mark.parametrize("R,T,E,El,k,drop", SHAPES)
def test_layout_of_choices(R, T, E, El, k, drop):
    print(f"[choices] layout R{R} T{T} E{E}/{El} k{k} drop {drop}", flush=True)
    rng = np.random.default_rng(T * 31 + E)
    idx, e2l = _choices(rng, R, T, E, k, drop), _e2l(rng, E, El)
    L = Layer(R, T, 128, E, El, k, "bf16", e2l)
    assert L.layout(idx) == 0
    ref = M4.layout(idx, e2l, El)
    N = len(ref["pull_src"])
    for n in ("counts", "offsets", "slot_of"):
        assert np.array_equal(getattr(L, n).cpu().numpy(), ref[n]), n
    got = L.pull_src.cpu().numpy()
    assert np.array_equal(got[:N], ref["pull_src"]) and (got[N:] == -7).all()


def test_layout_equals_the_routed_layout():
    """The choices that moe_layout takes, given: every output and every table behind it the same."""
    torch = _torch()
    from mixture_experts_layer_histogram_amd.device import DeviceProblem
    cfg = configs.MID.scaled(name="choices R2 T333 E64/16 k6", R=2, T=333, d=256, F=128, E=64, E_local=16, k=6)
    P = DeviceProblem(cfg, inputs.make_inputs(cfg, seed=3))
    P.layout()
    P.dispatch()
    keep = {n: getattr(P, n).clone() for n in ("counts", "offsets", "slot_of", "xe")}
    N = int(P.offsets[-1])
    src = P.pull_src[:N].clone()
    for n in keep:
        getattr(P, n).zero_()
    P.ws.fill_(0x33)
    moe.moe_layout_choices(P.shape, P.placement, P.ex, P.topk_idx, P.counts, P.offsets, P.pull_src, P.slot_of, P.ws)
    P.dispatch()
    assert P.status() == 0 and torch.equal(P.pull_src[:N], src)
    for n, v in keep.items():
        m = N if n == "xe" else len(v)
        assert torch.equal(getattr(P, n)[:m], v[:m]), n


@pytest.mark.parametrize("what", ["too large", "too small", "twice", "last pair"])
@pytest.mark.parametrize("T", [1, 64, 300])
def test_bad_choices_are_refused_on_the_device(what, T):
    rng = np.random.default_rng(5)
    idx, e2l = _choices(rng, 2, T, 16, 4, 0.0), _e2l(rng, 16, 16)
    L = Layer(2, T, 128, 16, 16, 4, "bf16", e2l)
    bad = idx.copy()
    if what == "too large":
        bad[0, 0, 0] = 16
    elif what == "too small":
        bad[1, T // 2, 3] = -2
    elif what == "twice":
        bad[1, T - 1, 2] = bad[1, T - 1, 0]
    else:
        bad[1, T - 1, 3] = 2 ** 31 - 1
    assert L.layout(bad) == -1
    assert (L.offsets == 0).all() and (L.slot_of == -1).all()
    assert (L.pull_src == -7).all()
    assert L.layout(idx) == 0                             # the next call is not affected
    assert np.array_equal(L.slot_of.cpu().numpy(), M4.layout(idx, e2l, 16)["slot_of"])
    dup = idx.copy()
    dup[0, 0, :2] = -1                                    # -1 twice is no expert twice
    assert L.layout(dup) == 0


@pytest.mark.parametrize("R,T,E,El,k,drop", [(8, 8192, 16, 8, 9, 0.1), (3, 7000, 256, 32, 6, 0.02),
                                              (64, 513, 1024, 1000, 16, 0.0)])
def test_layout_of_many_choices(R, T, E, El, k, drop):
    """Many workgroups, tokens across the groups and blocks they split the pairs at (k does not divide 64), and
    more pairs than the workgroups hold in registers (more than 524288); slots by a stable sort."""
    print(f"[choices] layout R{R} T{T} E{E}/{El} k{k}", flush=True)
    rng = np.random.default_rng(11)
    idx = np.argsort(rng.random((R * T, E), dtype=np.float32), axis=1)[:, :k].astype(np.int32).reshape(R, T, k)
    idx[rng.random(idx.shape) < drop] = -1
    e2l = _e2l(rng, E, El)
    L = Layer(R, T, 128, E, El, k, "bf16", e2l)
    assert L.layout(idx) == 0
    flat = idx.reshape(-1)
    l = np.where(flat >= 0, e2l[flat], -1)
    local = np.flatnonzero(l >= 0)
    order = local[np.argsort(l[local], kind="stable")]
    slot = np.full(flat.shape, -1, dtype=np.int32)
    slot[order] = np.arange(len(order), dtype=np.int32)
    assert np.array_equal(L.slot_of.cpu().numpy().reshape(-1), slot)
    assert np.array_equal(L.counts.cpu().numpy(), np.bincount(flat[flat >= 0], minlength=E))
    assert np.array_equal(L.offsets.cpu().numpy(), np.concatenate([[0], np.cumsum(np.bincount(l[local], minlength=El))]))
    src = L.pull_src.cpu().numpy()[:len(order)]
    assert np.array_equal(src[:, 0], order // (T * k)) and np.array_equal(src[:, 1], order // k % T)
    # one bad choice anywhere refuses all of it: across a group's edge, across a block's, in the last token
    for at in (63 // k, 4096 // k, (R * T * k // 2) // k, R * T - 1):
        bad = idx.reshape(-1, k).copy()
        bad[at] = np.arange(k)
        bad[at, k - 1] = bad[at, 0]
        assert L.layout(bad.reshape(R, T, k)) == -1, at
        assert (L.slot_of == -1).all() and (L.offsets == 0).all()
    bad = idx.copy()
    bad[R - 1, T - 1, k - 1] = E
    assert L.layout(bad) == -1
    assert L.layout(idx) == 0 and np.array_equal(L.slot_of.cpu().numpy().reshape(-1), slot)


MOVES = [  # R, T, d, E, El, k, drop, dtype
    (1, 1, 64, 4, 4, 1, 0.0, "bf16"), (1, 1, 4, 4, 4, 2, 0.0, "f32"), (1, 3, 12, 8, 3, 8, 0.4, "f32"),
    (2, 65, 128, 16, 16, 4, 0.2, "bf16"), (1, 130, 2048, 64, 64, 6, 0.0, "bf16"), (3, 50, 7168, 32, 8, 8, 0.1, "bf16"),
    (1, 64, 1408, 16, 8, 16, 0.1, "f32"), (2, 40, 2052, 8, 8, 3, 0.0, "f32"), (1, 37, 8256, 4, 4, 4, 0.0, "bf16"),
    (1, 9, 512, 16, 4, 4, 1.0, "bf16"), (1, 2100, 192, 12, 12, 5, 0.05, "bf16"),
    (1, 2060, 2176, 8, 8, 3, 0.1, "bf16"), (2, 1040, 1032, 8, 4, 2, 0.1, "f32"), (1, 2050, 8256, 4, 4, 2, 0.0, "bf16"),
]


def _move_inputs(R, T, d, E, El, k, drop, dtype):
    torch = _torch()
    rng = np.random.default_rng(d + T)
    idx, e2l = _choices(rng, R, T, E, k, drop), _e2l(rng, E, El)
    L = Layer(R, T, d, E, El, k, dtype, e2l, F=64 if dtype == "bf16" else 4)
    assert L.layout(idx) == 0
    g = torch.Generator(device="cuda")
    g.manual_seed(d * T)
    kind = torch.float32 if dtype == "f32" else torch.bfloat16
    N = int(L.offsets[-1])
    ye = torch.randn(N + 3, d, generator=g, device="cuda").to(kind)
    ye[N:] = float("nan")                                 # rows behind the last are not read
    w = torch.randn(R, T, k, generator=g, device="cuda")
    w[L.slot_of < 0] = float("nan")                       # nor the weights of pairs that are not local
    dy = [torch.randn(T, d, generator=g, device="cuda").to(kind) for _ in range(R)]
    return L, N, ye, w, dy, kind


def _n64(t):
    return t.double().cpu().numpy()


def _merge_ref(ye, slot, w):
    w = None if w is None else np.where(slot >= 0, w, 0.0)
    return M4.merge(ye, slot, w), M4.merge(np.abs(ye), slot, None if w is None else np.abs(w))


@pytest.mark.parametrize("R,T,d,E,El,k,drop,dtype", MOVES)
def test_merge_and_gradients(R, T, d, E, El, k, drop, dtype):
    torch = _torch()
    print(f"[choices] moves R{R} T{T} d{d} E{E}/{El} k{k} drop {drop} {dtype}", flush=True)
    L, N, ye, w, dy, kind = _move_inputs(R, T, d, E, El, k, drop, dtype)
    slot, y64, w64 = L.slot_of.cpu().numpy(), _n64(ye[:N]), _n64(w)
    u = 2.0 ** -24
    # rows back
    y = [torch.full((T, d), 9.0, dtype=kind, device="cuda") for _ in range(R)]
    moe.moe_combine_merge(L.shape, L.pl, ye, L.slot_of, w, y)
    ref, mag = _merge_ref(y64, slot, w64)
    got = np.stack([_n64(t) for t in y])
    lim = (k + 1) * u * mag
    assert (np.abs(got - ref) <= lim + HALF[dtype] * (np.abs(ref) + lim)).all()
    none = (slot < 0).all(-1)
    assert (got[none] == 0).all()
    # gradient of the rows and of the weights
    dye = torch.full((N + 3, d), 9.0, dtype=kind, device="cuda")
    dw = torch.full((R, T, k), 9.0, device="cuda")
    moe.moe_combine_merge_backward(L.shape, L.pl, dy, ye, L.slot_of, w, dye, dw)
    assert (dye[N:] == 9.0).all()
    dy64 = np.stack([_n64(t) for t in dy])
    src = L.pull_src.cpu().numpy()[:N]
    gate = np.zeros(N)
    gate[slot[slot >= 0]] = w64[slot >= 0]
    want = gate[:, None] * dy64[src[:, 0], src[:, 1]]
    assert (np.abs(_n64(dye[:N]) - want) <= (u + HALF[dtype]) * np.abs(want) * (1 + u) + 1e-40).all()
    dots = (dy64[src[:, 0], src[:, 1]] * y64).sum(-1)
    size = (np.abs(dy64[src[:, 0], src[:, 1]]) * np.abs(y64)).sum(-1)
    dwg = _n64(dw)
    back = np.zeros(N)
    back[slot[slot >= 0]] = dwg[slot >= 0]
    assert (np.abs(back - dots) <= (d / 64 + 16) * u * size).all()
    assert (dwg[slot < 0] == 0).all()
    # gradient of the pull
    dx = [torch.full((T, d), 9.0, dtype=kind, device="cuda") for _ in range(R)]
    moe.moe_dispatch_pull_backward(L.shape, L.pl, ye, L.slot_of, dx)
    ref, mag = _merge_ref(y64, slot, None)
    got = np.stack([_n64(t) for t in dx])
    lim = (k + 1) * u * mag
    assert (np.abs(got - ref) <= lim + HALF[dtype] * (np.abs(ref) + lim)).all() and (got[none] == 0).all()
    # the same bits again
    again = torch.empty_like(dye)
    dw2 = torch.empty_like(dw)
    moe.moe_combine_merge_backward(L.shape, L.pl, dy, ye, L.slot_of, w, again, dw2)
    assert torch.equal(again[:N], dye[:N]) and torch.equal(dw, dw2)


def test_gradients_against_differences():
    """L = <dy, merge(ye, w)> is linear in ye and in w: L(w + D) - L(w - D) = 2 <dw, D> for any D, up to the
    fp32 roundings of the two forwards."""
    torch = _torch()
    L, N, ye, w, dy, _ = _move_inputs(2, 40, 256, 8, 8, 3, 0.2, "f32")
    ye = ye[:N].contiguous()
    w = torch.nan_to_num(w)
    dye, dw = torch.empty_like(ye), torch.empty_like(w)
    moe.moe_combine_merge_backward(L.shape, L.pl, dy, ye, L.slot_of, w, dye, dw)
    dy64 = np.stack([_n64(t) for t in dy])
    slot = L.slot_of.cpu().numpy()

    def loss(rows, gate):
        y = [torch.empty(40, 256, device="cuda") for _ in range(2)]
        moe.moe_combine_merge(L.shape, L.pl, rows, L.slot_of, gate, y)
        out = np.stack([_n64(t) for t in y])
        mag = M4.merge(np.abs(_n64(rows)), slot, np.abs(_n64(gate)))
        return (dy64 * out).sum(), 4 * 2.0 ** -24 * (np.abs(dy64) * mag).sum()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for _ in range(3):
        D = torch.randint(-4, 5, w.shape, generator=g, device="cuda").float()
        (a, ea), (b, eb) = loss(ye, w + D), loss(ye, w - D)
        # w +- D round once more in fp32
        extra = 2 * 2.0 ** -24 * float(((w.abs() + D.abs()) * dw.abs()).sum().double())
        assert abs((a - b) / 2 - (_n64(dw) * _n64(D)).sum()) <= ea + eb + extra + 1e-5 * np.abs(_n64(dw) * _n64(D)).sum()
        D = torch.randint(-4, 5, ye.shape, generator=g, device="cuda").float()
        (a, ea), (b, eb) = loss(ye + D, w), loss(ye - D, w)
        extra = 2 * 2.0 ** -24 * float(((ye.abs() + D.abs()) * dye.abs()).sum().double())
        assert abs((a - b) / 2 - (_n64(dye) * _n64(D)).sum()) <= ea + eb + extra + 1e-5 * np.abs(_n64(dye) * _n64(D)).sum()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "mxfp8"])
def test_forward_choices_is_the_forward_bit_for_bit(dtype):
    torch = _torch()
    from mixture_experts_layer_histogram_amd.device import DeviceProblem
    cfg = configs.MID.scaled(name=f"forward_choices {dtype}", R=2, T=150, d=512, F=256, E=16, E_local=8, k=4, dtype=dtype)
    P = DeviceProblem(cfg, inputs.make_inputs(cfg, seed=1))
    P.forward()
    assert P.status() == 0
    y, idx, w = [t.clone() for t in P.y], P.topk_idx.clone(), P.topk_w.clone()
    for t in P.y:
        t.fill_(float("nan"))
    P.ye.fill_(float("nan"))
    P.forward_choices(idx, w)
    assert P.status() == 0 and all(torch.equal(a, b) for a, b in zip(y, P.y))
    # dropped pairs: the token's other experts, and a padded token gives zeros
    idx[0, 0, 1:] = -1
    idx[1, 5] = -1
    P.forward_choices(idx, w)
    assert P.status() == 0 and (P.y[1][5] == 0).all()
    s = int(P.slot_of[0, 0, 0])
    want = torch.zeros(cfg.d, device="cuda") if s < 0 else (P.ye[s].float() * w[0, 0, 0])
    assert torch.equal(P.y[0][0], want.to(P.y[0].dtype))
    assert torch.equal(P.y[0][1:], y[0][1:]) and torch.equal(P.y[1][:5], y[1][:5])


def _train_step(P, idx, w, dy):
    """Forward and gradients of the bf16 layer for given choices, from the library's calls."""
    torch = _torch()
    P.forward_choices(idx, w)
    a, b = moe.moe_backward_rows_info(P.shape, P.placement)
    dw = torch.empty_like(w)
    moe.moe_combine_merge_backward(P.shape, P.placement, dy, P.ye, P.slot_of, w, P.bws[a:], dw)
    moe.moe_expert_ffn_backward(P.shape, P.placement, P.xe, P.offsets, P.w1, P.w3, P.w2, P.ws, P.dw1, P.dw3, P.dw2, P.bws)
    moe.moe_dispatch_pull_backward(P.shape, P.placement, P.bws[b:], P.slot_of, P.dx)
    return dw


def _train_problem(seed=4):
    torch = _torch()
    from mixture_experts_layer_histogram_amd.device import DeviceProblem
    cfg = configs.MID.scaled(name="train choices R2 T200 d384 F320 E16/8 k4", R=2, T=200, d=384, F=320, E=16, E_local=8, k=4)
    inp = inputs.make_inputs(cfg, seed=seed)
    P = DeviceProblem(cfg, inp)
    P.alloc_backward()
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    dy = [torch.randn(cfg.T, cfg.d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(cfg.R)]
    return cfg, inp, P, dy


def test_training_step_under_the_softmax_router_is_moe_backward():
    """With the choices and gates of moe_layout the chain of calls gives moe_backward's dx and weight
    gradients bit for bit."""
    torch = _torch()
    cfg, inp, P, dy = _train_problem()
    P.forward()
    P.dy = dy
    moe.moe_backward(P.shape, P.placement, dy, P.xe, P.ye, P.w1, P.w3, P.w2, P.topk_idx, P.topk_w, P.offsets, P.pull_src,
                     P.slot_of, P.ws, P.recv, P.dx, P.dlogits, P.dw1, P.dw3, P.dw2, P.bws)
    want = [t.clone() for t in (*P.dx, P.dw1, P.dw3, P.dw2)]
    dl = torch.stack(P.dlogits)
    idx, w = P.topk_idx.clone(), P.topk_w.clone()
    for t in (*P.dx, P.dw1, P.dw3, P.dw2):
        t.fill_(float("nan"))
    dw = _train_step(P, idx, w, dy)
    assert all(torch.equal(a, b) for a, b in zip(want, (*P.dx, P.dw1, P.dw3, P.dw2)))
    # the logit gradient from the weights' gradient by the softmax rule
    z = w * (dw - (w * dw).sum(-1, keepdim=True))
    mine = torch.zeros_like(dl).scatter_(-1, idx.long(), z)
    scale = (w.abs() * dw.abs()).sum(-1, keepdim=True)
    assert ((mine - dl).abs() <= 1e-4 * scale + 1e-12).all()


def test_training_step_under_a_sigmoid_router():
    """Gates sigmoid(logits) of the k best by a biased score, some pairs dropped: the gradients of the step
    against the 64-bit formulas (bars: 2e-2 of a row's largest value, as for moe_backward)."""
    torch = _torch()
    cfg, inp, P, dy = _train_problem(seed=9)
    logits = torch.stack(P.logits).double()
    bias = 0.05 * torch.cos(torch.arange(cfg.E, device="cuda").double())
    idx = torch.topk(torch.sigmoid(logits) + bias, cfg.k, dim=-1).indices
    w = torch.sigmoid(logits).gather(-1, idx).float().contiguous()
    idx = idx.int().contiguous()
    idx[:, ::7, 2] = -1
    idx[1, -20:] = -1                                     # a padded tail
    dw = _train_step(P, idx, w, dy)
    assert P.status() == 0
    n = lambda t: t.double().cpu().numpy()                # noqa: E731
    x = np.stack([n(t) for t in P.x])
    dy64 = np.stack([n(t) for t in dy])
    lay = M4.layout(idx.cpu().numpy(), P.e2l.cpu().numpy(), cfg.E_local)
    slot, src, off = lay["slot_of"], lay["pull_src"], lay["offsets"]
    N = len(src)
    assert N > 300
    rows, dyr = x[src[:, 0], src[:, 1]], dy64[src[:, 0], src[:, 1]]
    gate = np.zeros(N)
    gate[slot[slot >= 0]] = n(w)[slot >= 0]
    dxe, ye = np.zeros_like(rows), np.zeros_like(rows)
    w1, w3, w2 = n(P.w1), n(P.w3), n(P.w2)
    for l in range(cfg.E_local):
        r = slice(off[l], off[l + 1])
        a, b = rows[r] @ w1[l].T, rows[r] @ w3[l].T
        h = O.silu(a) * b
        ye[r] = h @ w2[l].T
        do = gate[r, None] * dyr[r]
        dh = do @ w2[l]
        da, db = dh * b * OB.silu_grad(a), dh * O.silu(a)
        dxe[r] = da @ w1[l] + db @ w3[l]
        for got, ref in ((P.dw1[l], da.T @ rows[r]), (P.dw3[l], db.T @ rows[r]), (P.dw2[l], do.T @ h)):
            top = np.abs(ref).max(-1)
            assert (np.abs(n(got) - ref).max(-1) <= 2e-2 * top + 1e-30).all()
    dx = M4.merge(dxe, slot, None)
    got = np.stack([n(t) for t in P.dx])
    assert (np.abs(got - dx).max(-1) <= 2e-2 * np.abs(dx).max(-1) + 1e-30).all()
    dwr = np.where(slot >= 0, (dyr * ye).sum(-1)[np.maximum(slot, 0)], 0.0)
    size = np.where(slot >= 0, (np.linalg.norm(dyr, axis=-1) * np.linalg.norm(ye, axis=-1))[np.maximum(slot, 0)], 0.0)
    assert (np.abs(n(dw) - dwr) <= 2e-2 * size + 1e-30).all()


def test_chain_captured_and_replayed():
    torch = _torch()
    cfg, inp, P, dy = _train_problem(seed=2)
    P.forward()
    idx, w = P.topk_idx.clone(), P.topk_w.clone()
    dw = _train_step(P, idx, w, dy)
    want = [t.clone() for t in (*P.y, *P.dx, P.dw1, P.dw3, P.dw2, dw)]
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        dw = _train_step(P, idx, w, dy)
    for i in range(3):
        for t in (*P.y, *P.dx, P.dw1, P.dw3, P.dw2, dw):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (*P.y, *P.dx, P.dw1, P.dw3, P.dw2, dw))), i


def test_rows_past_4_gib():
    """320000 rows of 14 KiB (4.6 GB): slots whose byte offsets pass 32 bits, checked at both ends."""
    torch = _torch()
    T, d, k = 40000, 7168, 8
    idx = torch.stack([torch.randperm(8, device="cuda") for _ in range(16)]).int().repeat(T // 16, 1).reshape(1, T, 8).contiguous()
    L = Layer(1, T, d, 8, 8, k, "bf16", np.arange(8, dtype=np.int32), F=64)
    assert L.layout(idx) == 0
    N = T * k
    assert int(L.offsets[-1]) == N
    x = [torch.randn(T, d, device="cuda").to(torch.bfloat16)]
    xe = torch.empty(N, d, dtype=torch.bfloat16, device="cuda")
    moe.moe_dispatch_pull(L.shape, L.pl, x, L.pull_src, L.offsets, xe, L.ws)
    w = torch.rand(1, T, k, device="cuda")
    y = [torch.empty_like(x[0])]
    moe.moe_combine_merge(L.shape, L.pl, xe, L.slot_of, w, y)
    for t in (0, 1, T // 2, T - 1):
        s = L.slot_of[0, t].long()
        assert int(s.max()) >= 7 * T
        assert torch.equal(xe[s], x[0][t].expand(k, d))
        ref = x[0][t].double() * w[0, t].double().sum()
        assert ((y[0][t].double() - ref).abs() <= (2.0 ** -8 + 9 * 2.0 ** -24) * ref.abs() * (1 + 2.0 ** -8)).all()
    dxe, dw = torch.empty_like(xe), torch.empty_like(w)
    moe.moe_combine_merge_backward(L.shape, L.pl, x, xe, L.slot_of, w, dxe, dw)
    for t in (0, T - 1):
        s = L.slot_of[0, t].long()
        assert torch.equal(dxe[s], (x[0][t].float() * w[0, t][:, None]).to(torch.bfloat16))
    # every pair of a token holds the token's own row: its weight gradients are |x|^2 all
    assert torch.allclose(dw, x[0].double().square().sum(-1)[None, :, None].expand_as(w).float(), rtol=1e-4)


def test_more_tokens_than_a_launch_has_waves():
    """17 million tokens of one 16-byte vector: waves take several tokens.  One term a token, so the merge and
    the row gradient are single products, and a weight's gradient four products and their sum."""
    torch = _torch()
    T = 17_000_000
    shape, pl = moe.Shape(1, T, 4, 4, 1, 128, moe.MOE_F32), moe.Placement(1, 4)
    g = torch.Generator(device="cuda").manual_seed(7)
    ye, dy = (torch.randn(T, 4, device="cuda", generator=g) for _ in range(2))
    w = torch.randn(T, device="cuda", generator=g)
    slot = torch.randperm(T, device="cuda", generator=g).to(torch.int32)
    slot[:: 1000] = -1
    local = slot >= 0
    at = slot[local].long()
    y, dx = (torch.full((T, 4), float("nan"), device="cuda") for _ in range(2))
    moe.moe_combine_merge(shape, pl, ye, slot, w, [y])
    assert torch.equal(y[local], w[local, None] * ye[at]) and (y[~local] == 0).all()
    moe.moe_dispatch_pull_backward(shape, pl, ye, slot, [dx])
    assert torch.equal(dx[local], ye[at]) and (dx[~local] == 0).all()
    dye, dw = torch.full((T, 4), 9.0, device="cuda"), torch.full((T,), float("nan"), device="cuda")
    moe.moe_combine_merge_backward(shape, pl, [dy], ye, slot, w, dye, dw)
    assert torch.equal(dye[at], w[local, None] * dy[local]) and (dw[~local] == 0).all()
    assert int((dye == 9.0).all(1).sum()) == T - int(local.sum())
    terms = dy[local].double() * ye[at].double()
    assert ((dw[local].double() - terms.sum(1)).abs() <= 4 * 2.0 ** -24 * terms.abs().sum(1)).all()
