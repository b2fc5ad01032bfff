"""GPU parity of the RMS norm and its gradients, and of the dispatch of quantised rows.

Bars.  2^-24 a rounding in fp32, finfo.eps / 2 for the one rounding to the row type (bf16: 2^-8 of the value at most).  A sum of
squares has positive terms, so it is off by at most as many roundings as the longest chain of additions: 32 fused ones in a
lane, 6 over the wave, 15 over the waves, one division, one addition: 55 of 2^-24; rstd by half of that, and two more for root and
reciprocal; with the residual's addition and two products, y by (55 / 2 + 5) * 2^-24 of its value: FWD below.  The gradients' sums have
terms of both signs: the same chains, of the sums of magnitudes.
"""
import numpy as np
import pytest

from oracle import more_oracle as M
from oracle import mx_oracle as M8
from mixture_experts_layer_histogram_amd import configs, inputs, moe
from tests.test_gpu_mx4 import GUARD, _rowmajor

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
FWD = 33 * U
BWD = 70 * U           # both sums (55 each, of which rstd takes half, three times) and some six products
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
EPS = 1e-6


def _torch():
    import torch
    return torch


def _kind(dtype):
    torch = _torch()
    return (moe.MOE_BF16, torch.bfloat16) if dtype == "bf16" else (moe.MOE_F32, torch.float32)


def _rows(rows, d, dtype, seed, scale=1.0):
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, d, generator=g, device="cuda") * scale).to(_kind(dtype)[1])


def _np(t):
    return t.double().cpu().numpy()


def _guarded(rows, d, kind, value=7.0):
    """A buffer of rows with one more behind them that has to stay as it is."""
    return _torch().full((rows + 1, d), value, dtype=kind, device="cuda")


def _check_codes(codes, scales, n, err):
    """Every code within half a step of the 64-bit value, and what `err` allows that value to be off before the rounding."""
    rows, d = n.shape
    v = M.state_values(codes, _rowmajor(scales, rows, d).reshape(-1)).reshape(rows, d)
    sc = _rowmajor(scales, rows, d).astype(np.float64)
    unit = np.where(sc > 0, np.exp2(sc - 127), 0).repeat(32, 1)
    top = np.abs(n).reshape(rows, -1, 32).max(-1).repeat(32, 1)
    assert ((unit == 0) == (top == 0)).all()
    some = top > 0
    # floor(log2 max) - 8, of a maximum that may be off by err
    assert (unit[some] <= 2.0 ** -8 * top[some] * (1 + err)).all() and (unit[some] * (1 + err) > 2.0 ** -9 * top[some] * (1 - err)).all()
    y = np.abs(n) / np.where(some, unit, 1)
    step = np.maximum(np.exp2(np.floor(np.log2(np.maximum(y * (1 + err), 2.0 ** -30))) - 3), 2.0 ** -9)
    allowed = np.where(y > 448, np.maximum(y - 448, 16), step / 2) * unit + err * np.abs(n)
    assert (np.abs(v - n) <= allowed * (1 + 1e-12)).all()


FWD_CASES = [(1, 4, "f32"), (3, 8, "bf16"), (37, 1408, "f32"), (1, 7168, "bf16"), (513, 128, "bf16"), (70, 132, "f32"),
             (5, 2056, "bf16"), (9, 8192, "f32"), (3, 8200, "bf16"), (2, 32768, "f32"), (2, 32768, "bf16"), (2, 16644, "f32"),
             (4100, 2048, "bf16"), (2051, 7168, "bf16"), (40000, 64, "f32")]


@pytest.mark.parametrize("rows,d,dtype", FWD_CASES)
@pytest.mark.parametrize("residual", [True, False])
def test_norm(rows, d, dtype, residual):
    torch = _torch()
    code, kind = _kind(dtype)
    x, res = _rows(rows, d, dtype, 1), _rows(rows, d, dtype, 2, 3.0) if residual else None
    gamma = 1 + 0.1 * torch.randn(d, device="cuda")
    h, y = _guarded(rows, d, kind), _guarded(rows, d, kind)
    codes = d % 128 == 0
    q = torch.full((rows + 1, d), GUARD, dtype=torch.uint8, device="cuda") if codes else None
    sc = torch.full((rows * d // 32 + 64,), GUARD, dtype=torch.uint8, device="cuda") if codes else None
    n = moe.Norm(rows, d, code, EPS)
    moe.moe_norm(n, x, res, gamma, h, y, q, sc)
    s, ref, _ = M.norm(_np(x), None if res is None else _np(res), _np(gamma), EPS)
    assert (np.abs(_np(h[:rows]) - s) <= (HALF[dtype] + U) * np.abs(s)).all()
    assert (np.abs(_np(y[:rows]) - ref) <= (HALF[dtype] + FWD) * np.abs(ref)).all()
    assert (h[rows] == 7).all() and (y[rows] == 7).all()
    if codes:
        assert (q[rows] == GUARD).all() and (sc[rows * d // 32:] == GUARD).all()
        _check_codes(q[:rows].cpu().numpy(), sc[: rows * d // 32].cpu().numpy(), ref, FWD)
    # each output alone, without gamma, and in place, has the same bits
    y2 = torch.empty_like(x)
    moe.moe_norm(n, x, res, gamma, None, y2)
    assert torch.equal(y2, y[:rows])
    ones = torch.ones_like(gamma)
    moe.moe_norm(n, x, res, ones, None, y2)
    y3 = torch.empty_like(x)
    moe.moe_norm(n, x, res, None, None, y3)
    assert torch.equal(y2, y3)
    if codes:
        q2, sc2 = torch.empty_like(q[:rows]), torch.empty_like(sc[: rows * d // 32])
        moe.moe_norm(n, x, res, gamma, None, None, q2, sc2)
        assert torch.equal(q2, q[:rows]) and torch.equal(sc2, sc[: rows * d // 32])
    a, b = x.clone(), None if res is None else res.clone()
    if residual:
        moe.moe_norm(n, a, b, gamma, b, a)
        assert torch.equal(b, h[:rows]) and torch.equal(a, y[:rows])
    else:
        moe.moe_norm(n, a, None, gamma, None, a)
        assert torch.equal(a, y[:rows])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_of_wild_rows(dtype):
    """A NaN or an infinity stays in its row (its squares' sum) and turns its blocks into NaN; rows of zeros are zeros;
    a row of which all but one value vanish; the largest values whose squares fp32 holds."""
    torch = _torch()
    code, kind = _kind(dtype)
    d = 256
    x = _rows(7, d, dtype, 5)
    x[0, 3] = float("nan")
    x[1, 200] = float("inf")
    x[2] = 0
    x[3] = 0
    x[3, 17] = -2.0
    x[4] *= 2.0 ** 58
    x[5] *= 2.0 ** -30
    y = torch.empty_like(x)
    q, sc = torch.empty(7, d, dtype=torch.uint8, device="cuda"), torch.empty(2, 7, 4, dtype=torch.uint8, device="cuda")
    moe.moe_norm(moe.Norm(7, d, code, EPS), x, None, None, None, y, q, sc)
    y = _np(y)
    words = _rowmajor(sc.cpu().numpy().reshape(-1), 7, d)
    assert np.isnan(y[0]).all() and (words[0] == 255).all() and (q[0] == 0).all()
    # 1 / inf = 0, and inf * 0 = NaN at the infinity itself
    assert np.isnan(y[1, 200]) and (np.delete(y[1], 200) == 0).all()
    assert words[1, 6] == 255 and (np.delete(words[1], 6) == 0).all() and (q[1] == 0).all()
    assert (y[2] == 0).all() and (words[2] == 0).all()
    s, ref, _ = M.norm(_np(x[3:]), None, None, EPS)
    assert (np.abs(y[3:] - ref) <= (HALF[dtype] + FWD) * np.abs(ref)).all()
    _check_codes(q[3:].cpu().numpy(), sc[:, 3:].contiguous().cpu().numpy().reshape(-1), ref, FWD)


@pytest.mark.parametrize("rows,d,dtype", [(1, 4, "f32"), (3, 8, "bf16"), (129, 2048, "f32"), (37, 1408, "bf16"), (4099, 128, "bf16"),
                                          (2, 2052, "f32"), (1500, 7168, "bf16"), (3, 32768, "bf16"), (3, 32768, "f32"),
                                          (2, 12296, "bf16"), (1025, 8192, "f32"), (5000, 512, "f32")])
@pytest.mark.parametrize("with_dh", [True, False])
def test_norm_backward(rows, d, dtype, with_dh):
    torch = _torch()
    code, kind = _kind(dtype)
    h, dy = _rows(rows, d, dtype, 1, 3.0), _rows(rows, d, dtype, 2)
    dh = _rows(rows, d, dtype, 3) if with_dh else None
    gamma = 1 + 0.1 * torch.randn(d, device="cuda")
    n = moe.Norm(rows, d, code, EPS)
    ws = torch.full((moe.moe_norm_backward_workspace_bytes(n) + 256,), GUARD, dtype=torch.uint8, device="cuda")
    dx, dgamma = _guarded(rows, d, kind), torch.full((d + 1,), 7.0, device="cuda")
    moe.moe_norm_backward(n, dy, h, gamma, dh, dx, dgamma, ws, ws.numel() - 256)
    rx, rg, bx, bg = M.norm_backward(_np(dy), _np(h), _np(gamma), None if dh is None else _np(dh), EPS)
    assert (np.abs(_np(dx[:rows]) - rx) <= HALF[dtype] * np.abs(rx) + BWD * bx).all()
    # a column's sum: rows of a workgroup in turn (1024 share the rows, or 4 waves each of them; at most 4 rows more each where they
    # are 512 or 256, for up to 2000 rows of more than 2048 values), their partial sums by
    # 16 waves, then those; each term is off by rstd's 55 / 2 + 2 and two products
    chain = rows / 1024 + 4 + 64 + 16 + 30 + 4
    assert (np.abs(_np(dgamma[:d]) - rg) <= chain * U * bg).all()
    assert (dx[rows] == 7).all() and dgamma[d] == 7 and (ws[-256:] == GUARD).all()
    # again, one at a time, in place: the same bits
    d2, g2 = torch.empty_like(h), torch.empty_like(gamma)
    moe.moe_norm_backward(n, dy, h, gamma, dh, d2, None)
    moe.moe_norm_backward(n, dy, h, gamma, dh, None, g2, ws)
    assert torch.equal(d2, dx[:rows]) and torch.equal(g2, dgamma[:d])
    for which in range(3 if with_dh else 2):
        bufs = [dy.clone(), h.clone(), None if dh is None else dh.clone()]
        moe.moe_norm_backward(n, bufs[0], bufs[1], gamma, bufs[2], bufs[which], None)
        assert torch.equal(bufs[which], dx[:rows])


def test_norm_backward_without_gamma_and_without_rows():
    torch = _torch()
    h, dy = _rows(5, 64, "f32", 1), _rows(5, 64, "f32", 2)
    n = moe.Norm(5, 64, moe.MOE_F32, EPS)
    a, b = torch.empty_like(h), torch.empty_like(h)
    moe.moe_norm_backward(n, dy, h, None, None, a, None)
    moe.moe_norm_backward(n, dy, h, torch.ones(64, device="cuda"), None, b, None)
    assert torch.equal(a, b)
    n0 = moe.Norm(0, 64, moe.MOE_F32, EPS)
    dgamma = torch.full((64,), 7.0, device="cuda")
    assert moe.moe_norm(n0, None, None, None, None, None) == 0
    moe.moe_norm_backward(n0, None, None, None, None, None, dgamma)
    assert (dgamma == 0).all()


# ------------------------------------------------------------------------------------------------ dispatch of codes
@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("R,T,d,E,El,k,drop", [(1, 1, 128, 4, 4, 2, 0), (3, 37, 1024, 16, 8, 4, 0.2), (2, 300, 7168, 16, 16, 2, 0),
                                               (8, 64, 2048, 64, 8, 8, 0.1), (1, 5000, 256, 8, 8, 6, 0)])
def test_dispatch_of_codes_equals_the_quantising_dispatch(fmt, R, T, d, E, El, k, drop):
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(T)
    code = moe.DTYPE_CODE[fmt]
    sh = moe.Shape(R, T, d, E, k, 128, code)
    e2l = torch.full((E,), -1, dtype=torch.int32, device="cuda")
    e2l[torch.randperm(E, generator=g, device="cuda")[:El]] = torch.arange(El, dtype=torch.int32, device="cuda")
    p = moe.Placement(e2l.data_ptr(), El)
    idx = torch.topk(torch.rand(R, T, E, generator=g, device="cuda"), k).indices.int()
    idx[torch.rand(R, T, k, generator=g, device="cuda") < drop] = -1
    x = [torch.randn(T, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(R)]
    nmax = moe.moe_max_pairs(sh, p)
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, offsets, slot = torch.empty(E, **i32), torch.empty(El + 1, **i32), torch.empty(R, T, k, **i32)
    src = torch.empty(nmax, 2, **i32)
    ws = torch.empty(moe.moe_workspace_bytes(sh, p), dtype=torch.uint8, device="cuda")
    moe.moe_layout_choices(sh, p, None, idx, counts, offsets, src, slot, ws)
    per = d if fmt == "mxfp8" else d // 2
    new = lambda *s: torch.full(s, GUARD, dtype=torch.uint8, device="cuda")      # noqa: E731
    xe, xes, ye, yes = new(nmax, per), new(d // 128, nmax, 4), new(nmax, per), new(d // 128, nmax, 4)
    moe.moe_dispatch_pull(sh, p, x, src, offsets, xe, ws, xe_scales=xes)
    xq, xs = [], []
    for t in x:
        xq.append(new(T, per))
        xs.append(new(d // 128, T, 4))
        moe.moe_mx_quantize_to(t, moe.MOE_BF16, T, d, code, xq[-1], xs[-1])
    moe.moe_dispatch_pull_codes(sh, p, xq, xs, src, offsets, ye, yes, ws)
    assert moe.moe_read_status(ws) == 0
    N = int(offsets[-1])
    assert N > 0 and torch.equal(ye[:N], xe[:N]) and torch.equal(yes[:, :N], xes[:, :N])
    assert (ye[N:] == GUARD).all() and (yes[:, N:] == GUARD).all()


def test_dispatch_of_codes_with_no_local_pair():
    torch = _torch()
    sh = moe.Shape(1, 16, 128, 4, 1, 128, moe.MOE_MXFP8)
    e2l = torch.tensor([-1, 0, -1, -1], dtype=torch.int32, device="cuda")
    p = moe.Placement(e2l.data_ptr(), 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    idx = torch.full((1, 16, 1), -1, **i32)
    src, offsets = torch.zeros(16, 2, **i32), torch.empty(2, **i32)
    ws = torch.empty(moe.moe_workspace_bytes(sh, p), dtype=torch.uint8, device="cuda")
    moe.moe_layout_choices(sh, p, None, idx, torch.empty(4, **i32), offsets, src, torch.empty(1, 16, 1, **i32), ws)
    u8 = dict(dtype=torch.uint8, device="cuda")
    xe, xes = torch.full((16, 128), GUARD, **u8), torch.full((1, 16, 4), GUARD, **u8)
    moe.moe_dispatch_pull_codes(sh, p, [torch.zeros(16, 128, **u8)], [torch.zeros(1, 16, 4, **u8)], src, offsets, xe, xes, ws)
    assert (xe == GUARD).all() and (xes == GUARD).all()


# ------------------------------------------------------------------------------------------------ the range that the header names
SPREAD = [1.0, 2e-18, 2e16, 1e-16, 3.0, 1e8, 2.0 ** -50]
RANGE = [(15, 4, "f32"), (15, 8, "bf16"), (9001, 64, "f32"), (29, 512, "bf16"), (4203, 2048, "bf16"), (29, 1408, "f32"), (15, 4096, "f32"), (1100, 7168, "bf16"),
         (15, 8200, "bf16"), (15, 32768, "f32")]


def _sized(rows, d, dtype, seed):
    """Rows of sizes in turn, side by side in a workgroup: from the smallest whose squares fp32 holds (a mean of 4e-36, of which each value's
    2^-150 is less than 2^-31) to values of 1e17, 32768 of which add up to less than 3.4e38."""
    torch = _torch()
    size = torch.tensor([SPREAD[i % len(SPREAD)] for i in range(rows)], device="cuda")
    return (_rows(rows, d, "f32", seed).clamp(-5, 5) * size[:, None]).to(_kind(dtype)[1])


@pytest.mark.parametrize("rows,d,dtype", RANGE)
def test_norm_without_eps_over_its_range(rows, d, dtype):
    torch = _torch()
    code, kind = _kind(dtype)
    x, res = _sized(rows, d, dtype, 1), _sized(rows, d, dtype, 2)
    gamma = 1 + 0.1 * torch.randn(d, device="cuda")
    h, y = torch.empty_like(x), torch.empty_like(x)
    q = torch.empty(rows, d, dtype=torch.uint8, device="cuda") if d % 128 == 0 else None
    sc = torch.empty(rows * d // 32, dtype=torch.uint8, device="cuda") if d % 128 == 0 else None
    moe.moe_norm(moe.Norm(rows, d, code, 0.0), x, res, gamma, h, y, q, sc)
    s, ref, _ = M.norm(_np(x), _np(res), _np(gamma), 0.0)
    assert (np.abs(_np(h) - s) <= (HALF[dtype] + U) * np.abs(s)).all()
    bad = ~(np.abs(_np(y) - ref) <= (HALF[dtype] + FWD) * np.abs(ref))
    assert not bad.any(), sorted({int(i) % len(SPREAD) for i in np.nonzero(bad)[0]})
    if q is not None:
        _check_codes(q.cpu().numpy(), sc.cpu().numpy(), ref, FWD)


@pytest.mark.parametrize("rows,d,dtype", RANGE)
def test_norm_gradients_without_eps_over_its_range(rows, d, dtype):
    torch = _torch()
    code, kind = _kind(dtype)
    h, dy, dh = _sized(rows, d, dtype, 1), _rows(rows, d, dtype, 2), _rows(rows, d, dtype, 3)
    gamma = 1 + 0.1 * torch.randn(d, device="cuda")
    n = moe.Norm(rows, d, code, 0.0)
    ws = torch.empty(moe.moe_norm_backward_workspace_bytes(n), dtype=torch.uint8, device="cuda")
    dx, dgamma = torch.empty_like(h), torch.empty(d, device="cuda")
    moe.moe_norm_backward(n, dy, h, gamma, dh, dx, dgamma, ws)
    rx, rg, bx, bg = M.norm_backward(_np(dy), _np(h), _np(gamma), _np(dh), 0.0)
    bad = ~(np.abs(_np(dx) - rx) <= HALF[dtype] * np.abs(rx) + BWD * bx)
    assert not bad.any(), sorted({int(i) % len(SPREAD) for i in np.nonzero(bad)[0]})
    chain = rows / 1024 + 4 + 64 + 16 + 30 + 4
    assert (np.abs(_np(dgamma) - rg) <= chain * U * bg).all()


@pytest.mark.parametrize("d,dtype", [(512, "bf16"), (2048, "bf16"), (4096, "bf16"), (8192, "bf16"), (16384, "bf16"), (32768, "bf16"),
                                     (512, "f32"), (2048, "f32"), (4096, "f32"), (8192, "f32"), (16384, "f32"), (32768, "f32")])
def test_rows_past_the_caches(d, dtype):
    """Rows of 256 MiB and more go past the caches: the same bits as in two calls that do not, with one, four, eight and sixteen waves a row,
    residual, codes and dh; gamma's gradient against 64 bits."""
    torch = _torch()
    code, kind = _kind(dtype)
    rows = (1 << 28) // (d * (2 if dtype == "bf16" else 4)) + 5
    half = rows // 2
    x, res = _rows(rows, d, dtype, 1), _rows(rows, d, dtype, 2)
    gamma = 1 + 0.1 * torch.randn(d, device="cuda")

    def forward(lo, hi):
        k = hi - lo
        h, y = _guarded(k, d, kind), _guarded(k, d, kind)
        q = torch.full((k + 1, d), GUARD, dtype=torch.uint8, device="cuda")
        sc = torch.full((k * d // 32 + 64,), GUARD, dtype=torch.uint8, device="cuda")
        moe.moe_norm(moe.Norm(k, d, code, EPS), x[lo:hi], res[lo:hi], gamma, h, y, q, sc)
        assert (h[k] == 7).all() and (y[k] == 7).all() and (q[k] == GUARD).all() and (sc[k * d // 32:] == GUARD).all()
        return h[:k], y[:k], q[:k], sc[:k * d // 32].view(d // 128, k, 4).transpose(0, 1)

    whole, parts = forward(0, rows), (forward(0, half), forward(half, rows))
    for i, t in enumerate(whole):
        assert torch.equal(t[:half], parts[0][i]) and torch.equal(t[half:], parts[1][i])
    h = whole[0]
    del parts, whole

    def backward(lo, hi, dgamma):
        n = moe.Norm(hi - lo, d, code, EPS)
        ws = torch.empty(moe.moe_norm_backward_workspace_bytes(n), dtype=torch.uint8, device="cuda")
        dx = _guarded(hi - lo, d, kind)
        moe.moe_norm_backward(n, x[lo:hi], h[lo:hi], gamma, res[lo:hi], dx, dgamma, ws)
        assert (dx[hi - lo] == 7).all()
        return dx[:hi - lo]

    dgamma = torch.empty(d, device="cuda")
    dx = backward(0, rows, dgamma)
    assert torch.equal(dx[:half], backward(0, half, None)) and torch.equal(dx[half:], backward(half, rows, None))
    ref, mag = torch.zeros(d, dtype=torch.double, device="cuda"), torch.zeros(d, dtype=torch.double, device="cuda")
    for lo in range(0, rows, 8192):
        a, b = h[lo:lo + 8192].double(), x[lo:lo + 8192].double()
        t = b * a / torch.sqrt((a * a).mean(-1, keepdim=True) + EPS)
        ref += t.sum(0)
        mag += t.abs().sum(0)
    # as in test_norm_backward, of the workgroups that share the rows: 1024, 512 with eight waves a row, 256 with sixteen
    chain = rows / (1024 if d <= 2048 else 512 if d <= 8192 else 256) + 4 + 64 + 16 + 30 + 4
    assert ((dgamma.double() - ref).abs() <= chain * U * mag).all()
