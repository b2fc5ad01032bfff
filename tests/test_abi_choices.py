"""Refusals of the entry points for given choices and MXFP4, before any HIP call (no GPU)."""
import ctypes

import pytest

from mixture_experts_layer_histogram_amd import moe

FAKE = 0x7F0000000000
BIG = 1 << 40


def _shape(**kw):
    d = dict(R=2, T=64, d=1024, E=16, k=4, F=512, dtype=moe.MOE_BF16)
    d.update(kw)
    return moe.Shape(d["R"], d["T"], d["d"], d["E"], d["k"], d["F"], d["dtype"])


def _tab(n=2, last=FAKE):
    return ctypes.cast((ctypes.c_void_p * n)(*([FAKE] * (n - 1) + [last])), ctypes.c_void_p)


def _call(name, shape, args, pl=None):
    return getattr(moe.lib(), name)(ctypes.byref(shape), ctypes.byref(pl or moe.Placement(FAKE, 8)), *args)


MX = moe.MXScales(FAKE, FAKE, FAKE)
# valid arguments after (shape, placement); TAB marks a rank table, WS a workspace pointer
CALLS = {
    "moe_layout_choices": [None, FAKE, FAKE, FAKE, FAKE, FAKE, "WS", BIG, None],
    "moe_combine_merge": ["ROW", FAKE, FAKE, "TAB", None],
    "moe_combine_merge_backward": ["TAB", "ROW", FAKE, FAKE, "ROW", FAKE, None],
    "moe_dispatch_pull_backward": ["ROW", FAKE, "TAB", None],
    "moe_forward_choices": [None, FAKE, FAKE, "TAB", "ROW", "ROW", "ROW", "MX", "ROW", "SC", "ROW", "TAB", FAKE, FAKE,
                            FAKE, FAKE, "WS", BIG, None],
}


def _fill(spec, at=None, value=None):
    out = []
    for i, a in enumerate(spec):
        v = {"TAB": _tab(), "ROW": FAKE, "WS": FAKE, "SC": FAKE}.get(a, a) if isinstance(a, str) and a != "MX" else a
        if a == "MX":
            v = ctypes.byref(MX)
        out.append(value if i == at else v)
    return out


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("dtype", [moe.MOE_F32, moe.MOE_BF16, moe.MOE_MXFP8, moe.MOE_MXFP4])
def test_missing_and_misaligned_pointers(name, dtype):
    spec, s = CALLS[name], _shape(dtype=dtype)
    stream = len(spec) - 1
    for i, a in enumerate(spec):
        if i == stream or a == BIG or (a is None and i == 0):
            continue
        mx_only = a in ("MX", "SC")
        if mx_only and dtype not in (moe.MOE_MXFP8, moe.MOE_MXFP4):
            continue
        if a == "WS":                       # checked after the pointers: everything else is valid here
            assert _call(name, s, _fill(spec, i, None)) == -1
            assert _call(name, s, _fill(spec, i, FAKE + 64)) == -2
            continue
        assert _call(name, s, _fill(spec, i, None)) == -1, (name, i)
        if a == "TAB":
            assert _call(name, s, _fill(spec, i, _tab(last=None))) == -1
            assert _call(name, s, _fill(spec, i, _tab(last=FAKE + 8))) == -2
        elif a == "ROW":
            assert _call(name, s, _fill(spec, i, FAKE + 8)) == -2
        elif a == "SC":
            assert _call(name, s, _fill(spec, i, FAKE + 2)) == -2
        elif a == "MX":
            assert _call(name, s, _fill(spec, i, ctypes.byref(moe.MXScales(FAKE, None, FAKE)))) == -1
            assert _call(name, s, _fill(spec, i, ctypes.byref(moe.MXScales(FAKE, FAKE, FAKE + 1)))) == -2


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("kw,El,code", [(dict(k=0), 8, -1), (dict(k=17), 8, -1), (dict(T=0), 8, -1), (dict(R=65), 8, -1),
                                        (dict(), 0, -1), (dict(), 17, -1), (dict(dtype=4), 8, -1),
                                        (dict(dtype=moe.MOE_MXFP4, d=1024 + 64), 8, -2),
                                        (dict(dtype=moe.MOE_MXFP4, F=512 + 64), 8, -2),
                                        (dict(dtype=moe.MOE_MXFP4, d=1 << 17, F=1 << 15), 8, -1),
                                        (dict(d=1000), 8, -2), (dict(dtype=moe.MOE_F32, d=130), 8, -2)])
def test_bad_shapes(name, kw, El, code):
    assert _call(name, _shape(**kw), _fill(CALLS[name]), moe.Placement(FAKE, El)) == code


def test_outputs_in_place_of_inputs():
    """A row moved onto rows that other tokens still read: the same pointer is refused."""
    s, other = _shape(), FAKE + (1 << 30)
    both = _tab(last=other)                                              # rank 0's rows are at FAKE
    assert _call("moe_combine_merge", s, [FAKE, FAKE, FAKE, both, None]) == -1
    assert _call("moe_combine_merge", s, [other, FAKE, FAKE, both, None]) == -1
    assert _call("moe_combine_merge_backward", s, [both, other + 64, FAKE, FAKE, other + 64, FAKE, None]) == -1
    assert _call("moe_dispatch_pull_backward", s, [other, FAKE, both, None]) == -1


def test_small_workspace_and_exec_knobs():
    for name in ("moe_layout_choices", "moe_forward_choices"):
        spec = list(CALLS[name])
        at = spec.index(BIG)
        assert _call(name, _shape(), _fill(spec, at, 1024)) == -3
        for ex in (moe.Exec(-1), moe.Exec(0, 0, 0, 1), moe.Exec(0, 0, 0, 0, 0, 1)):
            assert _call(name, _shape(), _fill(spec, 0, ctypes.byref(ex))) == -1
        assert _call(name, _shape(), _fill(spec), moe.Placement(None, 8)) == -1


def test_paths_that_mxfp4_does_not_have():
    s, p, L = _shape(dtype=moe.MOE_MXFP4), moe.Placement(FAKE, 8), moe.lib()
    S, P = ctypes.byref(s), ctypes.byref(p)
    t = _tab()
    assert moe.moe_ring_slot_bytes(s, moe.Exec(128)) == 0
    assert L.moe_backward_workspace_bytes(S, P) == 0
    assert L.moe_forward_persistent(S, P, None, t, t, FAKE, FAKE, FAKE, ctypes.byref(MX), FAKE, BIG, t, t, FAKE, FAKE,
                                    FAKE, FAKE, FAKE, FAKE, FAKE, BIG, None) == -6
    assert L.moe_forward_persistent_noalloc(S, P, None, t, t, FAKE, FAKE, FAKE, t, t, FAKE, FAKE, FAKE, FAKE, FAKE,
                                            FAKE, None, None) == -6
    assert L.moe_persistent_dispatch_ffn_combine(S, P, None, t, FAKE, FAKE, FAKE, ctypes.byref(MX), FAKE, BIG, FAKE,
                                                 FAKE, FAKE, t, FAKE, BIG, None) == -6
    assert L.moe_expert_ffn_push(S, P, None, t, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, ctypes.byref(MX), FAKE, FAKE, t,
                                 FAKE, BIG, None) == -6
    assert L.moe_backward(S, P, t, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, BIG, t, t, t, FAKE,
                          FAKE, FAKE, FAKE, BIG, None) == -6
    assert L.moe_backward_prepare_mx(S, P, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None) == -6
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert L.moe_backward_rows_info(S, P, ctypes.byref(a), ctypes.byref(b)) == -6
    # h is half a byte a value: the workspace is smaller than MXFP8's ...
    many, m8 = _shape(dtype=moe.MOE_MXFP4, T=4096), _shape(dtype=moe.MOE_MXFP8, T=4096)
    assert 0 < moe.moe_workspace_bytes(many, p) < moe.moe_workspace_bytes(m8, p)
    # ... but holds fp32 expert rows up to 16 MiB of them: 4096 rows of 1024, not 4104
    at, past = (moe.moe_workspace_bytes(_shape(dtype=moe.MOE_MXFP4, T=t), p) for t in (512, 513))
    assert at > (16 << 20) > past
    # and the calls it shares with MXFP8 need its scales
    assert L.moe_dispatch_pull(S, P, t, FAKE, FAKE, FAKE, None, FAKE, BIG, None) == -1
    assert L.moe_expert_ffn(S, P, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, BIG, None) == -1


def test_rows_info():
    s, p = _shape(), moe.Placement(FAKE, 8)
    a, b = moe.moe_backward_rows_info(s, p)
    size = 2 * 64 * 4 * 1024 * 2
    total = moe.lib().moe_backward_workspace_bytes(ctypes.byref(s), ctypes.byref(p))
    assert a % 256 == 0 and b % 256 == 0 and a + size <= total and b + size <= total and abs(a - b) >= size
    with pytest.raises(moe.MoEError):
        moe.moe_backward_rows_info(_shape(dtype=moe.MOE_F32), p)
    assert moe.lib().moe_backward_rows_info(ctypes.byref(s), ctypes.byref(p), None, ctypes.byref(ctypes.c_size_t())) == -1


@pytest.mark.parametrize("fmt", [moe.MOE_MXFP8, moe.MOE_MXFP4])
def test_codec_refusals(fmt):
    q, dq = moe.lib().moe_mx_quantize_to, moe.lib().moe_mx_dequantize
    assert q(FAKE, moe.MOE_BF16, 4, 128, moe.MOE_BF16, FAKE, FAKE, None) == -1       # no such format
    assert dq(FAKE, FAKE, moe.MOE_F32, 4, 128, FAKE, moe.MOE_BF16, None) == -1
    assert q(FAKE, moe.MOE_MXFP8, 4, 128, fmt, FAKE, FAKE, None) == -1
    assert dq(FAKE, FAKE, fmt, 4, 128, FAKE, moe.MOE_MXFP4, None) == -1
    for rows, K, code in ((-1, 128, -1), (4, 0, -1), (4, 64, -2), (4, 160, -2), (1 << 40, 128, -1)):
        assert q(FAKE, moe.MOE_BF16, rows, K, fmt, FAKE, FAKE, None) == code
        assert dq(FAKE, FAKE, fmt, rows, K, FAKE, moe.MOE_BF16, None) == code
    for bad in range(3):
        a = [FAKE] * 3
        a[bad] = None
        assert q(a[0], moe.MOE_F32, 4, 128, fmt, a[1], a[2], None) == -1
        assert dq(a[0], a[1], fmt, 4, 128, a[2], moe.MOE_F32, None) == -1
    assert q(FAKE + 8, moe.MOE_F32, 4, 128, fmt, FAKE, FAKE, None) == -2
    assert q(FAKE, moe.MOE_F32, 4, 128, fmt, FAKE + 8, FAKE, None) == -2
    assert dq(FAKE + 8, FAKE, fmt, 4, 128, FAKE, moe.MOE_F32, None) == -2
    assert dq(FAKE, FAKE, fmt, 4, 128, FAKE + 8, moe.MOE_F32, None) == -2
    assert dq(FAKE, FAKE + 2, fmt, 4, 128, FAKE, moe.MOE_F32, None) == -2
    assert q(FAKE, moe.MOE_BF16, 0, 128, fmt, FAKE, FAKE, None) == 0                 # nothing to do, nothing launched
    assert dq(FAKE, FAKE, fmt, 0, 128, FAKE, moe.MOE_BF16, None) == 0


@pytest.mark.parametrize("kw,El,Ts", [(dict(R=1, d=2048, F=1408, E=64, k=6), 64, (1, 128, 340, 341, 1024)),
                                      (dict(R=2, d=1024, F=512, E=16, k=4), 8, (1, 33, 512, 513, 4096)),
                                      (dict(R=8, d=7168, F=2048, E=256, k=8), 32, (1, 9, 10, 64, 4096))])
def test_a_workspace_for_more_tokens_serves_fewer(kw, El, Ts):
    """moe_workspace_bytes of T tokens suffices for every smaller T, although the fp32 rows make it smaller than
    those of some of them.  (The calls check the workspace before ye is found among the outputs.)"""
    other = FAKE + (1 << 40)

    def forward(T, ws_bytes):
        s = _shape(dtype=moe.MOE_MXFP4, T=T, **kw)
        t = (ctypes.c_void_p * s.R)(*[FAKE] * s.R)
        args = [None, FAKE, FAKE, t, FAKE, FAKE, FAKE, ctypes.byref(MX), other, FAKE, FAKE, t, FAKE, FAKE, FAKE, FAKE, FAKE,
                ws_bytes, None]
        return _call("moe_forward_choices", s, args, moe.Placement(FAKE, El))

    size = {T: moe.moe_workspace_bytes(_shape(dtype=moe.MOE_MXFP4, T=T, **kw), moe.Placement(FAKE, El)) for T in Ts}
    assert any(size[a] > size[b] for a in Ts for b in Ts if a < b)
    for T in Ts:
        for small in Ts:
            if small <= T:
                assert forward(small, size[T]) == -1, (small, T)            # not MOE_ENOSPC
        assert forward(T, 4096) == -3
    assert forward(Ts[-1], size[Ts[-1]] - 256) == -3 and forward(Ts[-1], size[Ts[0]]) == -3


def test_merge_backward_has_no_mxfp4_form():
    """moe_forward_choices in MXFP4 writes ye or not by its size, so the gradient that reads ye refuses the dtype."""
    args = [_tab(), FAKE + (1 << 40), FAKE, FAKE, FAKE + (2 << 40), FAKE, None]
    assert _call("moe_combine_merge_backward", _shape(dtype=moe.MOE_MXFP4), args) == -6


@pytest.mark.parametrize("fmt", [moe.MOE_MXFP8, moe.MOE_MXFP4])
@pytest.mark.parametrize("by", [1, 2, 3])
def test_quantize_to_asks_for_aligned_scales_in_both_formats(fmt, by):
    q = moe.lib().moe_mx_quantize_to
    assert q(FAKE, moe.MOE_BF16, 4, 128, fmt, FAKE, FAKE + by, None) == -2
    assert q(FAKE, moe.MOE_F32, 0, 128, fmt, FAKE, FAKE + by, None) == -2


@pytest.mark.parametrize("fmt", [moe.MOE_MXFP8, moe.MOE_MXFP4])
def test_codec_of_no_rows_takes_null_pointers(fmt):
    """An empty tensor has no address: no rows are done whatever the pointers, once the sizes and types are right."""
    L = moe.lib()
    for ptr in (None, FAKE, FAKE + 1):
        assert L.moe_mx_quantize_to(ptr, moe.MOE_BF16, 0, 128, fmt, ptr, ptr, None) == (-2 if ptr == FAKE + 1 else 0)
        assert L.moe_mx_dequantize(ptr, ptr, fmt, 0, 128, ptr, moe.MOE_F32, None) == (-2 if ptr == FAKE + 1 else 0)
    assert L.moe_mx_quantize_to(None, moe.MOE_BF16, 0, 64, fmt, None, None, None) == -2
    assert L.moe_mx_quantize_to(None, moe.MOE_BF16, 1, 128, fmt, None, None, None) == -1
    assert L.moe_mx_dequantize(None, None, fmt, 0, 128, None, fmt, None) == -1
