"""GPU parity of the AdamW step.

Bars.  States: bit for bit (the header's order of operations, each rounded once, and whole-number roundings).  The param: from the
states, away = lr * m' * rcp(root * c + eps): float32 factors of lr, by_m, by_r and eps, a root, five products and sums, and a
reciprocal of one unit: 16 roundings of 2^-24 of away at most; two of the kept part and one of the difference: 3 of |p| + |away|;
a param rounded to bf16 by half a step more, or by less than one where it is rounded stochastically.
"""
import numpy as np
import pytest

from oracle import more_oracle as M
from mixture_experts_layer_histogram_amd import moe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BETA1, BETA2, LR, EPS = 0.9, 0.999, 1e-3, 1e-8


def _torch():
    import torch
    return torch


def _np(t):
    return t.double().cpu().numpy()


def _pad(n):
    return -(-n // 128) * 128


class Tensor:
    """A tensor of n values with what its step reads and writes; buffers have guards behind them."""

    def __init__(self, n, param, grad, master, eight, seed, wd=0.1, zero=False):
        torch = _torch()
        g = torch.Generator(device="cuda").manual_seed(seed)
        kind = {"f32": torch.float32, "bf16": torch.bfloat16}
        self.n, self.eight, self.wd = n, eight, wd
        rand = lambda s: torch.randn(n + 16, generator=g, device="cuda") * s           # noqa: E731
        p, size = rand(0.02), torch.exp(rand(2.0))
        self.param, self.grad = p.to(kind[param]), (rand(1e-3) * size).to(kind[grad])
        self.master = p if master else None
        m, v = rand(3e-4) * size, (1e-3 * size) ** 2
        if zero:
            m, v = m * 0, v * 0
        if eight:
            nm = lambda t: np.pad(t[:n].cpu().numpy(), (0, _pad(n) - n))               # noqa: E731
            cm, sm = M.state_codes(nm(m), None, False)
            cv, sv = M.state_codes(np.sqrt(nm(v)), None, True)
            dev = lambda a: torch.from_numpy(np.concatenate([a, np.full(64, 0x5A, np.uint8)])).cuda()  # noqa: E731
            self.m, self.ms, self.v, self.vs = dev(cm), dev(sm), dev(cv), dev(sv)
        else:
            self.m, self.v, self.ms, self.vs = m, v, None, None
        self.kinds = (moe.DTYPE_CODE[param], moe.DTYPE_CODE[grad])

    def entry(self):
        return moe.AdamWTensor(self.param, self.grad, self.n, *self.kinds, self.m, self.v, self.ms, self.vs, self.master, self.wd)

    def copy(self):
        t = object.__new__(Tensor)
        t.__dict__.update({k: v.clone() if hasattr(v, "clone") else v for k, v in self.__dict__.items()})
        return t

    def same(self, o):
        return all(_torch().equal(a, b) for a, b in zip(self.buffers(), o.buffers()))

    def buffers(self):
        return [t for t in (self.param, self.master, self.m, self.v, self.ms, self.vs) if t is not None]

    def check(self, old, place, step, seed, stochastic, scale=1.0, lr=LR):
        n = self.n
        g = np.float32(_np(old.grad[:n])) * np.float32(scale)
        if self.eight:
            k = _pad(n)
            m = M.state_values(old.m[:k].cpu().numpy(), old.ms[:k // 32].cpu().numpy())[:n]
            v = np.float32(M.state_values(old.v[:k].cpu().numpy(), old.vs[:k // 32].cpu().numpy())[:n])
            v = v * v
        else:
            m, v = old.m[:n].cpu().numpy(), old.v[:n].cpu().numpy()
        m, v = M.moments(m, v, g, BETA1, BETA2)
        if self.eight:
            bits = M.random_bits(seed, step, place, k, 0)
            pad = lambda a: np.pad(a, (0, k - n))                                       # noqa: E731
            cm, sm = M.state_codes(pad(m), bits & np.uint64(0xFFFF) if stochastic else None, False)
            cv, sv = M.state_codes(pad(np.sqrt(v)), bits >> np.uint64(16) if stochastic else None, True)
            for got, want in ((self.m, cm), (self.ms, sm), (self.v, cv), (self.vs, sv)):
                got = got.cpu().numpy()
                assert np.array_equal(got[:want.size], want), np.nonzero(got[:want.size] != want)
                assert (got[want.size:] == 0x5A).all()
        else:
            assert np.array_equal(self.m[:n].cpu().numpy(), m) and np.array_equal(self.v[:n].cpu().numpy(), v)
            assert _torch().equal(self.m[n:], old.m[n:]) and _torch().equal(self.v[n:], old.v[n:])
        p0 = _np((old.param if old.master is None else old.master)[:n])
        p, away = M.adamw(p0, m, v, lr, BETA1, BETA2, EPS, step, self.wd)
        bar = 16 * U * away + 3 * U * (np.abs(p0) + away)
        if self.master is not None:
            got = _np(self.master[:n])
            assert (np.abs(got - p) <= bar).all()
            assert _torch().equal(self.param[:n], self.master[:n].to(_torch().bfloat16))
            assert _torch().equal(self.master[n:], old.master[n:])
        elif self.kinds[0] == moe.MOE_F32:
            assert (np.abs(_np(self.param[:n]) - p) <= bar).all()
        else:
            got = _np(self.param[:n])
            step_of = np.exp2(np.floor(np.log2(np.maximum(np.abs(p), 2.0 ** -126))) - 7)
            assert (np.abs(got - p) <= bar + step_of * (1.0 if stochastic else 0.5)).all()
        assert _torch().equal(self.param[n:], old.param[n:])


def _step(tensors, step, seed, eight, stochastic, **more):
    moe.moe_adamw(moe.AdamW(LR, BETA1, BETA2, EPS, step, moe.MOE_MXFP8 if eight else moe.MOE_F32, int(stochastic), seed, **more),
                  moe.adamw_table(t.entry() for t in tensors))


SIZES = [1, 3, 128, 129, 31, 4096, 2049, 70001]


@pytest.mark.parametrize("param,grad,master", [("f32", "f32", False), ("bf16", "bf16", True), ("bf16", "f32", True),
                                               ("bf16", "bf16", False), ("f32", "bf16", False)])
@pytest.mark.parametrize("eight,stochastic", [(False, False), (True, True), (True, False), (False, True)])
def test_step(param, grad, master, eight, stochastic):
    """Tensors of many sizes in one call, from states that live and from zeros, at the first and a later step."""
    for step, seed, zero in ((1, 0, True), (1000, (7 << 40) + 3, False)):
        ts = [Tensor(n, param, grad, master, eight, 10 + i, wd=0.1 * (i % 3), zero=zero) for i, n in enumerate(SIZES)]
        old = [t.copy() for t in ts]
        _step(ts, step, seed, eight, stochastic)
        for i, (t, o) in enumerate(zip(ts, old)):
            t.check(o, i, step, seed, stochastic)


@pytest.mark.parametrize("eight", [False, True])
def test_more_tensors_than_a_launch_takes(eight):
    """101 tensors, some of them empty, of mixed types: each as in a call of its own size (its place counts on over launches)."""
    ts = []
    for i in range(101):
        n = 0 if i % 17 == 5 else 1 + (i * 37) % 400
        ts.append(Tensor(n, ("f32", "bf16")[i % 2], ("f32", "bf16")[i // 2 % 2], i % 4 == 1, eight, i))
    old = [t.copy() for t in ts]
    _step(ts, 12, 5, eight, True)
    for i, (t, o) in enumerate(zip(ts, old)):
        if t.n:
            t.check(o, i, 12, 5, True)
        else:
            assert t.same(o)


@pytest.mark.parametrize("eight", [False, True])
def test_values_on_the_device(eight):
    """The rate, the step and the gradients' factor read on the device: as given on the host."""
    torch = _torch()
    a, b = (Tensor(5000, "bf16", "bf16", True, eight, 3, wd=0.0) for _ in range(2))
    old = a.copy()
    lr, step = torch.tensor([LR], device="cuda"), torch.tensor([77], dtype=torch.int64, device="cuda")
    scale = torch.tensor([0.25], device="cuda")
    _step([a], 77, 9, eight, True, grad_scale=scale.data_ptr())
    moe.moe_adamw(moe.AdamW(0.5, BETA1, BETA2, EPS, 0, moe.MOE_MXFP8 if eight else moe.MOE_F32, 1, 9, scale.data_ptr(),
                            lr.data_ptr(), step.data_ptr()), [b.entry()])
    assert a.same(b)
    a.check(old, 0, 77, 9, True, scale=0.25)


@pytest.mark.parametrize("stochastic", [True, False])
def test_blocks_of_very_different_values(stochastic):
    """Gradients over forty powers of ten in one block: codes below E4M3's smallest power of two, zeros, roots that take the smallest
    code, states below fp32's normal range, blocks of zeros, the largest values."""
    torch = _torch()
    for seed in range(3):
        t = Tensor(4096, "f32", "f32", False, True, 20 + seed, zero=seed == 0, wd=0.0)
        g = torch.Generator(device="cuda").manual_seed(seed)
        size = 10.0 ** (40 * torch.rand(4096, generator=g, device="cuda") - 34)
        t.grad[:4096] = torch.randn(4096, generator=g, device="cuda") * size
        t.grad[64:96] = 0
        t.grad[96:128] *= 1e-12
        t.grad[128:160] = 1e18 * torch.sign(t.grad[128:160])
        old = t.copy()
        moe.moe_adamw(moe.AdamW(LR, BETA1, BETA2, EPS, 5, moe.MOE_MXFP8, int(stochastic), seed), [t.entry()])
        t.check(old, 0, 5, seed, stochastic)


def test_wild_gradients():
    """NaN and infinite gradients: their values alone in fp32 states, their blocks in 8 bits, for good."""
    torch = _torch()
    for eight in (False, True):
        t = Tensor(256, "bf16", "f32", True, eight, 4)
        clean = t.copy()
        t.grad[5], t.grad[200] = float("nan"), float("inf")
        for step in (3, 4):
            _step([t], step, 1, eight, True)
            _step([clean], step, 1, eight, True)
            p, c = t.master[:256], clean.master[:256]
            hit = torch.zeros(256, dtype=torch.bool, device="cuda")
            hit[5] = hit[200] = True
            if eight and step == 4:                  # the blocks' states are NaN by then
                hit[:32] = hit[192:224] = True
            assert torch.isnan(p[hit]).all() and torch.equal(p[~hit], c[~hit])
            assert torch.isnan(t.param[:256][hit].float()).all()
            if eight:
                assert (t.ms[:8].cpu().numpy() == 255).tolist() == [True] + [False] * 5 + [True, False]
                assert (t.vs[:8].cpu().numpy() == 255).tolist() == [True] + [False] * 5 + [True, False]


def test_eight_bit_states_follow_fp32_states():
    """500 steps of the same gradients: the mean of many values' v stays within some hundredths of the fp32 one (rounded to
    nearest it would not move at all), and params stay close.

    The root r is rounded without bias, so its square gains the rounding's variance: with steps of t and a change of c, t^2 (c/t)
    (1 - c/t) <= t c.  t is r/8 to r/16, 0.0902 r on the mean over a power of two (1/8 / (2 ln 2)); c = 0.001 |g^2 - v| / (2 r)
    with E|g^2 - v| <= s^2, the gradients' square (0.97 of it at v = s^2, all of it at v = 0).  So each step adds at most 4.51e-5
    s^2, 500 of them that decay by 0.001 393 times that, 0.0177 s^2, and v has come to 0.394 s^2: at most 0.045 of it, upwards.
    Beside that mean, one value's v is off by about 500^1/2 roundings, each of at most a sixteenth with the chance of a step's
    change over it: 0.35 of its deviation; over 8192 values 5 * 0.35 / 90 = 0.02."""
    torch = _torch()
    n = 8192
    a, b = Tensor(n, "f32", "f32", False, False, 6, zero=True), Tensor(n, "f32", "f32", False, True, 6, zero=True)
    g = torch.Generator(device="cuda").manual_seed(8)
    for step in range(1, 501):
        grad = torch.randn(n + 16, generator=g, device="cuda") * 1e-3
        a.grad, b.grad = grad, grad
        _step([a], step, 0, False, False)
        _step([b], step, 11, True, True)
    va = _np(a.v[:n])
    vb = M.state_values(b.v[:n].cpu().numpy(), b.vs[:n // 32].cpu().numpy()) ** 2
    assert -0.02 < vb.mean() / va.mean() - 1 < 0.045 + 0.02
    moved = _np(a.param[:n]) - _np(b.param[:n])
    assert np.abs(moved).mean() < 500 * LR * 0.1


def test_a_step_of_millions():
    """So many values that a workgroup takes two parts of a tensor at a time, beside tensors that end in either."""
    ts = [Tensor(n, "bf16", "bf16", True, True, 30 + i) for i, n in enumerate((4300001, 1025, 2048, 1, 3073, 1024))]
    old = [t.copy() for t in ts]
    _step(ts, 5, 3, True, True)
    for i, (t, o) in enumerate(zip(ts, old)):
        t.check(o, i, 5, 3, True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_of_states_for_every_code_and_scale(dtype):
    """Rows of 128 go their own way in moe_mx_dequantize: the same bits as rows of 256, for all 256 codes under all 256 scales."""
    torch = _torch()
    kind, code = (torch.bfloat16, moe.MOE_BF16) if dtype == "bf16" else (torch.float32, moe.MOE_F32)
    codes = torch.arange(256, device="cuda").repeat(256, 1).to(torch.uint8)                        # [scale][code]
    scales = torch.arange(256, device="cuda").to(torch.uint8)
    wide, rows = torch.empty(256, 256, dtype=kind, device="cuda"), torch.empty(512, 128, dtype=kind, device="cuda")
    moe.moe_mx_dequantize(codes, scales.repeat_interleave(4).repeat(2).contiguous(), moe.MOE_MXFP8, 256, 256, wide, code)
    moe.moe_mx_dequantize(codes, scales.repeat_interleave(8).contiguous(), moe.MOE_MXFP8, 512, 128, rows, code)
    a, b = wide.reshape(-1).float(), rows.reshape(-1).float()
    nan = torch.isnan(a)
    assert torch.equal(nan, torch.isnan(b)) and torch.equal(a[~nan], b[~nan]) and int(nan.sum()) == 256 + 2 * 255


@pytest.mark.parametrize("param,grad,master", [("f32", "f32", False), ("bf16", "f32", True), ("bf16", "bf16", True), ("bf16", "bf16", False)])
@pytest.mark.parametrize("eight,stochastic", [(False, False), (False, True), (True, True), (True, False)])
def test_finite_gradients_whose_squares_pass_fp32(param, grad, master, eight, stochastic):
    """v and its root are infinite then, so the change is zero and the param decays only; fp32 states go on like that in later steps, a
    block of 8-bit roots with an infinity is NaN from the next step on.  Gradients just within the range beside them."""
    torch = _torch()
    big = torch.tensor([1e21, -1e30, 3e38, 7e20, -5e20, 1e21, 1e21], device="cuda")
    at = [0, 7, 33, 130, 131, 200, 299]
    for step, zero in ((1, True), (1000, False)):
        t = Tensor(300, param, grad, master, eight, 40, zero=zero)
        t.grad[at] = big.to(t.grad.dtype)
        old = t.copy()
        _step([t], step, 5, eight, stochastic)
        t.check(old, 0, step, 5, stochastic)
        again = t.copy()
        _step([t], step + 1, 5, eight, stochastic)
        if eight:
            lost = torch.zeros(300, dtype=torch.bool, device="cuda")
            for block in (0, 1, 4, 6, 9):
                lost[32 * block: 32 * block + 32] = True
            p = t.param[:300] if t.master is None else t.master[:300]
            assert torch.equal(torch.isnan(p), lost)
        else:
            t.check(again, 0, step + 1, 5, stochastic)

@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("eps", [2.0 ** -126, 2.0 ** -100, 2.0 ** 126])
def test_the_smallest_and_the_largest_eps(eight, eps):
    """Values without a gradient and without states do not move but by the decay; with one, the change is at most one unit's rounding of
    lr m' / (r' + eps) off (as in the bars above)."""
    t = Tensor(300, "f32", "f32", False, eight, 41, zero=True)
    t.grad[:200] = 0
    old = t.copy()
    moe.moe_adamw(moe.AdamW(LR, BETA1, BETA2, eps, 1, moe.MOE_MXFP8 if eight else moe.MOE_F32, 0, 0), [t.entry()])
    p0, got = _np(old.param[:300]), _np(t.param[:300])
    m, v = M.moments(np.zeros(300), np.zeros(300), _np(t.grad[:300]), BETA1, BETA2)
    p, away = M.adamw(p0, m, v, LR, BETA1, BETA2, eps, 1, t.wd)
    assert (away[:200] == 0).all() and (np.abs(got - p) <= 16 * U * away + 3 * U * (np.abs(p0) + away)).all()


def test_params_move_with_eight_bit_states_as_with_fp32_states():
    """500 steps of the same gradients, which move a param by 500^1/2 lr (m' adds up to the gradients, over their size).  What 8 bits add, of
    that: m's roundings have at most a variance of (|m| / 16)^2 and count ten times (1 / (1 - 0.9)), |m| is (0.1 / 1.9)^1/2 of the root:
    10 * 0.23 / 16 = 0.144; v is off by 0.35 of itself and 0.065 on the mean at most (above), its root by half of that: 0.21.  A param that
    stands still is off by 1, one that goes the other way by 2."""
    torch = _torch()
    n = 8192
    a, b = Tensor(n, "f32", "f32", False, False, 6, zero=True), Tensor(n, "f32", "f32", False, True, 6, zero=True)
    start = _np(a.param[:n])
    g = torch.Generator(device="cuda").manual_seed(8)
    for step in range(1, 501):
        grad = torch.randn(n + 16, generator=g, device="cuda") * 1e-3
        a.grad, b.grad = grad, grad
        _step([a], step, 0, False, False)
        _step([b], step, 11, True, True)
    pa, pb = _np(a.param[:n]), _np(b.param[:n])
    moved = np.abs(pa - start).mean()
    assert 10 * LR < moved < 25 * LR
    assert np.abs(pa - pb).mean() <= 0.36 * moved


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("grad", ["bf16", "f32"])
def test_the_random_bits_of_a_bf16_param(eight, grad):
    """A param without a master: its 16 random bits (a word of their own) are added to what bf16 cuts off.  The codes of both ends of what the
    param's bar allows before that; most values have one."""
    torch = _torch()
    step, seed, n = 9, (5 << 35) + 77, 50001
    ts = [Tensor(k, "bf16", grad, False, eight, 50 + i) for i, k in enumerate((3, n))]
    old = [t.copy() for t in ts]
    _step(ts, step, seed, eight, True)
    for place, (t, o) in enumerate(zip(ts, old)):
        k = t.n
        if eight:
            pad = _pad(k)
            m = M.state_values(o.m[:pad].cpu().numpy(), o.ms[:pad // 32].cpu().numpy())[:k]
            v = np.float32(M.state_values(o.v[:pad].cpu().numpy(), o.vs[:pad // 32].cpu().numpy())[:k]) ** 2
        else:
            m, v = o.m[:k].cpu().numpy(), o.v[:k].cpu().numpy()
        m, v = M.moments(m, v, _np(o.grad[:k]), BETA1, BETA2)
        p0 = _np(o.param[:k])
        p, away = M.adamw(p0, m, v, LR, BETA1, BETA2, EPS, step, t.wd)
        bar = 16 * U * away + 3 * U * (np.abs(p0) + away)
        sure = np.abs(p) > 4 * bar
        r16 = (M.random_bits(seed, step, place, k, 1) & np.uint64(0xFFFF)).astype(np.uint32)
        f = np.float32
        least = (np.nextafter(f(np.abs(p) - bar), f(0)).view(np.uint32) + r16) >> 16
        most = (np.nextafter(f(np.abs(p) + bar), f(np.inf)).view(np.uint32) + r16) >> 16
        got = t.param[:k].view(torch.int16).cpu().numpy().view(np.uint16).astype(np.uint32)
        assert ((got >> 15).astype(bool) == (p < 0))[sure].all()
        assert ((least <= (got & 0x7FFF)) & ((got & 0x7FFF) <= most))[sure].all()
        assert sure.mean() > 0.99 and (least == most)[sure].mean() > 0.99


def test_small_changes_of_a_bf16_param_add_up():
    """100 changes of lr = 1e-4 (a constant gradient) to params of 1, whose bf16 neighbour below is 2^-8 away: to nearest none would stay.  Each is a
    step with the chance 1e-4 * 2^8: 100 of them vary by 100 * 1e-4 * 2^-8, 0.0063 a value and 6.9e-5 for the mean of 8192, of which five are
    allowed (the rest, m' / (r' + eps) and bf16's smaller steps above 1, below a thousandth of the 0.01)."""
    torch = _torch()
    t = Tensor(8192, "bf16", "f32", False, False, 60, wd=0.0, zero=True)
    t.param[:] = 1.0
    t.grad[:] = 1.0
    for step in range(1, 101):
        moe.moe_adamw(moe.AdamW(1e-4, BETA1, BETA2, EPS, step, moe.MOE_F32, 1, 3), [t.entry()])
    moved = 1.0 - _np(t.param[:8192])
    assert abs(moved.mean() - 0.01) <= 5 * 6.9e-5 + 1e-5
