"""GPU tests of calls at the edges of what the header allows, for given choices and MXFP4 experts."""
import numpy as np
import pytest

from oracle import mx4_oracle as M4
from oracle import mx_oracle_bwd as QB
from mixture_experts_layer_histogram_amd import configs, inputs, moe
from tests.mx4_packed import Packed
from tests.test_gpu_mx4 import _bound, _cfg, _check_merged, _check_rows, _problem, _push, _torch, _weights64
from tests.test_gpu_mx_bwd import DL_TOL, DX_FRO, DX_ROW, W_TOL

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,most", [(40, 3000), (200, 3000)])
def test_every_call_in_a_workspace_made_for_more_tokens(T, most):
    """The workspace of `most` tokens is smaller than that of T, which has room for fp32 rows.  Every call takes it, the
    rows are bf16 in ye, y is moe_forward's, and nothing behind its end is written.  With the shape's own
    workspace the rows stay in fp32 and ye is left alone."""
    torch = _torch()
    cfg = _cfg(f"mx4 workspace for {most} tokens, T{T}", T=T, d=1024, F=256, E=16, E_local=16, k=4)
    inp, P = _problem(cfg)
    own = P.ws
    many = moe.Shape(1, most, cfg.d, cfg.E, cfg.k, cfg.F, P.shape.dtype)
    size = moe.moe_workspace_bytes(many, P.placement)
    if T == 200:
        assert size < own.numel()
    wide = torch.full((max(size, own.numel()) + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    P.ws = wide[:size]
    if size > own.numel():                     # as small as the calls take: without the fp32 rows
        P.ws = wide[:own.numel() - P.nmax * cfg.d * 4]
    end = P.ws.numel()
    P.forward()
    assert P.status() == 0
    y, rows = [t.clone() for t in P.y], P.ye.clone()
    N = int(P.offsets[-1])
    idx, w = P.topk_idx.clone(), P.topk_w.clone()
    P.forward_fused()
    assert P.status() == 0 and torch.equal(y[0], P.y[0])
    assert torch.equal(y[0], _push(P, idx, w)[0])
    P.ye.fill_(float("nan"))
    P.y[0].fill_(float("nan"))
    P.forward_choices(idx, w)
    assert P.status() == 0 and torch.equal(y[0], P.y[0]) and torch.equal(rows[:N], P.ye[:N])
    assert (wide[end:] == 0x5A).all()
    P.ws = own
    P.ye.fill_(float("nan"))
    P.forward_choices(idx, w)
    assert P.status() == 0 and torch.isnan(P.ye).all() and not torch.equal(y[0], P.y[0])
    P.ye.copy_(rows)
    x64 = P.rows_f64(P.x[0]).reshape(1, cfg.T, cfg.d)
    _check_merged(P, *_check_rows(P, P.ye, x64, _weights64(P)), w)


@pytest.mark.parametrize("T", [40, 1100])
def test_gate_gradient_over_mxfp4_experts(T):
    """Staged calls write ye at every size, and the gradient of the gates reads it with a bf16 shape; the MXFP4
    shape is refused (at T = 40 moe_forward_choices leaves ye as it was, at 1100 it writes it)."""
    torch = _torch()
    cfg = _cfg(f"mx4 gate gradient T{T}", R=2, T=T, d=1024, F=256, E=16, E_local=8, k=4)
    inp, P = _problem(cfg)
    P.forward()
    idx, w = P.topk_idx.clone(), P.topk_w.clone()
    P.ye.fill_(float("nan"))
    P.forward_choices(idx, w)
    N = int(P.offsets[-1])
    assert bool(torch.isnan(P.ye[:N]).any()) == (T == 40)
    g = torch.Generator(device="cuda").manual_seed(T)
    dy = [torch.randn(T, cfg.d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    dye, dw = torch.full_like(P.ye, 9.0), torch.full_like(w, float("nan"))
    args = (dy, P.ye, P.slot_of, w, dye, dw)
    with pytest.raises(moe.MoEError):
        moe.moe_combine_merge_backward(P.shape, P.placement, *args)
    moe.moe_layout_choices(P.shape, P.placement, P.ex, idx, P.counts, P.offsets, P.pull_src, P.slot_of, P.ws)
    P.dispatch()
    P.ffn()
    rows = moe.Shape(2, T, cfg.d, cfg.E, cfg.k, cfg.F, moe.MOE_BF16)
    moe.moe_combine_merge_backward(rows, P.placement, *args)
    slot = P.slot_of.long()
    ye, dy64 = P.ye.double(), torch.stack(dy).double()[:, :, None]
    at = torch.where(slot >= 0, slot, 0)
    want = (dy64 * ye[at]).sum(-1)
    size = (dy64.abs() * ye[at].abs()).sum(-1)
    local = slot >= 0
    # d products and their sum in fp32, d / 64 + 6 additions to a lane
    assert ((dw.double() - want).abs() <= (cfg.d / 64 + 16) * 2.0 ** -24 * size)[local].all() and (dw[~local] == 0).all()
    step = w.double()[local][:, None] * dy64.expand(-1, -1, cfg.k, -1)[local]
    assert ((dye[slot[local]].double() - step).abs() <= (2.0 ** -8 + 2.0 ** -23) * step.abs()).all()
    assert (dye[N:] == 9.0).all()


@pytest.mark.parametrize("T", [5, 4300])
def test_rows_wider_than_the_gather_keeps_in_lds(T):
    """d = 524288: the scale words of four rows pass 64 KiB, so they go straight to memory, a row for a workgroup
    at a time (more rows than workgroups: 4300).  Codes bit for bit, and the layer of the few within its bounds."""
    torch = _torch()
    d = 1 << 19
    rows = torch.randn(7, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(torch.bfloat16)
    P = Packed(T, d, 128, 1, 1, seed=2, x=rows[torch.arange(T, device="cuda") % 7].contiguous())
    print(f"[edges] d {d} T {T}", flush=True)
    idx = torch.zeros(1, T, 1, dtype=torch.int32, device="cuda")
    P.layout(idx)
    P.xe.fill_(0x5A)
    P.xe_scales.fill_(0x5A)
    P.dispatch()
    assert P.status() == 0
    codes, sc, val = M4.quantize(rows.double().cpu().numpy())
    codes = torch.from_numpy(M4.pack(codes)).cuda()
    planes = torch.from_numpy(np.ascontiguousarray(sc.reshape(7, d // 128, 4).transpose(1, 0, 2))).cuda()
    for t in range(0, T, 700):
        n = min(700, T - t)
        assert torch.equal(P.xe[t:t + n], codes.repeat(100, 1)[:n])
        assert torch.equal(P.xe_scales[:, t:t + n], planes.repeat(1, 100, 1)[:, :n])
    if T > 32:
        return
    w = torch.rand(1, T, 1, device="cuda") + 0.5
    P.forward_choices(idx, w)
    assert P.status() == 0
    ref, allow = _bound(val[:T], *P.weights64(0))
    _check_merged(P, ref, allow, w)


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (1028, "f32")])
@pytest.mark.parametrize("T,k,drop", [(1, 1, 0.0), (3, 3, 0.5), (6656, 1, 0.0), (6657, 1, 0.0), (3700, 2, 0.02), (8192, 1, 0.0),
                                      (8193, 1, 0.0), (5000, 2, 0.2), (9000, 4, 0.05)])
def test_dispatch_of_any_number_of_rows(T, k, drop, d, dtype):
    """Row counts on both sides of those at which the gather's waves take one row or two, and grids bounded by the
    pairs there can be: every row the token's own, rows behind the last untouched."""
    torch = _torch()
    E = 8
    code, kind = {"f32": (moe.MOE_F32, torch.float32), "bf16": (moe.MOE_BF16, torch.bfloat16)}[dtype]
    g = torch.Generator(device="cuda").manual_seed(T + k)
    idx = torch.rand(1, T, E, device="cuda", generator=g).topk(k, -1).indices.int().contiguous()
    idx[torch.rand(1, T, k, device="cuda", generator=g) < drop] = -1
    e2l = torch.arange(E, dtype=torch.int32, device="cuda")
    shape, pl = moe.Shape(1, T, d, E, k, 64, code), moe.Placement(e2l.data_ptr(), E)
    n = moe.moe_max_pairs(shape, pl)
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, offsets = torch.empty(E, **i32), torch.empty(E + 1, **i32)
    src, slot = torch.empty(n, 2, **i32), torch.empty(1, T, k, **i32)
    ws = torch.empty(moe.moe_workspace_bytes(shape, pl), dtype=torch.uint8, device="cuda")
    moe.moe_layout_choices(shape, pl, None, idx, counts, offsets, src, slot, ws)
    x = torch.randn(T, d, device="cuda", generator=g).to(kind)
    xe = torch.full((n + 1, d), 9.0, dtype=kind, device="cuda")
    moe.moe_dispatch_pull(shape, pl, [x], src, offsets, xe, ws)
    N = int(offsets[-1])
    assert N == int((idx >= 0).sum())
    assert torch.equal(xe[:N], x[src[:N, 1].long()]) and (xe[N:] == 9.0).all()


def test_mxfp8_training_step_under_a_sigmoid_router(monkeypatch):
    """moe_backward_mx after moe_forward_choices: dx and the weight gradients for gates sigmoid(logits) of the k best by
    a biased score, some pairs dropped, against the MXFP8 backward oracle on the same choices (bars as for
    moe_backward_mx under the softmax router); the gates' gradient from moe_combine_merge_backward."""
    torch = _torch()
    from mixture_experts_layer_histogram_amd.device import DeviceProblem
    cfg = configs.MoEConfig("mxfp8 choices R2 T200 d256 F256 E16/8 k4", R=2, T=200, d=256, F=256, E=16, E_local=8, k=4,
                            dtype="mxfp8")
    inp = inputs.make_inputs(cfg, seed=5)
    bits, dy = inputs.make_dy(cfg, seed=5)
    P = DeviceProblem(cfg, inp)
    P.alloc_backward(bits)
    logits = torch.stack(P.logits).double()
    bias = 0.05 * torch.cos(torch.arange(cfg.E, device="cuda").double())
    idx = torch.topk(torch.sigmoid(logits) + bias, cfg.k, dim=-1).indices
    w = torch.sigmoid(logits).gather(-1, idx).float().contiguous()
    idx = idx.int().contiguous()
    idx[:, ::7, 2] = -1
    idx[1, -20:] = -1                                     # a padded tail
    P.forward_choices(idx, w)
    dye, dw = torch.empty_like(P.ye), torch.empty_like(w)
    moe.moe_combine_merge_backward(P.shape, P.placement, P.dy, P.ye, P.slot_of, w, dye, dw)
    P.prepare_backward_mx()
    P.topk_idx, P.topk_w = idx, w
    P.backward_mx()
    assert P.status() == 0
    ids, gates = idx.cpu().numpy(), w.double().cpu().numpy()
    lay = M4.layout(ids, inp.expert_to_local, cfg.E_local)
    monkeypatch.setattr(QB.O, "route", lambda *_: (ids, gates))
    monkeypatch.setattr(QB.O, "layout", lambda *_: lay)
    ref = QB.backward_q(inp.logits, inp.x_f32, inp.w1_f32, inp.w3_f32, inp.w2_f32, inp.expert_to_local, cfg.E_local, cfg.k,
                        dy)
    n = lambda t: t.double().cpu().numpy()                # noqa: E731
    slot = lay["slot_of"]
    assert np.array_equal(P.slot_of.cpu().numpy(), slot)
    has = (slot >= 0).any(-1)
    got = np.stack([n(t) for t in P.dx])
    assert has.sum() > 300 and (got[~has] == 0).all() and not has[1, -20:].any()
    row = np.abs(got - ref["dx"])[has].max(-1) / np.abs(ref["dx"][has]).max(-1)
    fro = np.linalg.norm((got - ref["dx"])[has]) / np.linalg.norm(ref["dx"][has])
    print(f"[edges] mxfp8 choices: dx row {row.max():.2e}, Frobenius {fro:.2e}", flush=True)
    assert row.max() <= DX_ROW and fro <= DX_FRO
    for key in ("dw1", "dw3", "dw2"):
        for l in range(cfg.E_local):
            top = np.abs(ref[key][l]).max(-1)
            assert (np.abs(n(getattr(P, key)[l]) - ref[key][l]).max(-1) <= W_TOL * top + 1e-30).all(), (key, l)
    at = np.maximum(slot, 0)
    want = np.where(slot >= 0, (dy[:, :, None] * ref["ye"][at]).sum(-1), 0.0)
    size = np.linalg.norm(dy, axis=-1)[:, :, None] * np.linalg.norm(ref["ye"][at], axis=-1)
    assert (np.abs(n(dw) - want) <= DL_TOL * size + 1e-30).all() and (n(dw)[slot < 0] == 0).all()
