"""Refusals of the norm, the dispatch of codes, the grouped products and the AdamW step, before any HIP call (no GPU)."""
import ctypes

import pytest

from mixture_experts_layer_histogram_amd import moe

A = 0x7F0000000000                      # aligned addresses that nothing may reach
B, C, D, E = (A + (i << 32) for i in range(1, 5))
BIG = 1 << 40
INF, NAN = float("inf"), float("nan")


def _norm(rows=5, d=256, dtype=moe.MOE_BF16, eps=1e-6, **kw):
    a = dict(x=A, residual=None, gamma=None, h=None, y=B, codes=None, scales=None)
    a.update(kw)
    return moe.moe_norm(moe.Norm(rows, d, dtype, eps), *a.values(), stream=0, check=False)


def _norm_bwd(rows=5, d=256, dtype=moe.MOE_BF16, eps=1e-6, **kw):
    a = dict(dy=A, h=B, gamma=None, dh=None, dx=C, dgamma=D, ws=E, ws_bytes=BIG)
    a.update(kw)
    return moe.moe_norm_backward(moe.Norm(rows, d, dtype, eps), *a.values(), stream=0, check=False)


@pytest.mark.parametrize("call", [_norm, _norm_bwd])
@pytest.mark.parametrize("kw,code", [(dict(rows=-1), -1), (dict(d=0), -1), (dict(d=32776), -1), (dict(rows=1 << 32), -1),
                                     (dict(d=252), -2), (dict(dtype=moe.MOE_F32, d=254), -2), (dict(dtype=moe.MOE_MXFP8), -6),
                                     (dict(dtype=9), -6), (dict(eps=-1e-9), -1), (dict(eps=NAN), -1), (dict(eps=INF), -1)])
def test_norm_limits(call, kw, code):
    assert call(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(y=None), -1), (dict(x=A + 8), -2), (dict(residual=C + 4), -2), (dict(gamma=C + 2), -2),
    (dict(h=C + 8), -2), (dict(y=B + 8), -2), (dict(h=B), -1), (dict(codes=C), -1), (dict(scales=C), -1),
    (dict(codes=C + 8, scales=D), -2), (dict(codes=C, scales=D + 2), -2), (dict(d=264, codes=C, scales=D), -2)])
def test_norm_pointers(kw, code):
    assert _norm(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), -1), (dict(h=None), -1), (dict(dx=None, dgamma=None), -1), (dict(ws=None), -1), (dict(ws=E + 64), -2),
    (dict(ws_bytes=64), -3), (dict(dy=A + 8), -2), (dict(h=B + 8), -2), (dict(dh=C + 8), -2), (dict(dx=C + 8), -2),
    (dict(dgamma=D + 2), -2), (dict(gamma=D + 2), -2)])
def test_norm_backward_pointers(kw, code):
    assert _norm_bwd(**kw) == code


def test_norm_of_no_rows():
    assert moe.moe_norm(moe.Norm(0, 256, moe.MOE_BF16, 0.0), None, None, None, None, None, stream=0) == 0
    assert moe.moe_norm_backward(moe.Norm(0, 256, moe.MOE_BF16, 0.0), None, None, None, None, None, None, stream=0) == 0
    assert moe.moe_norm_backward_workspace_bytes(moe.Norm(0, 256, moe.MOE_BF16, 0.0)) == 0
    assert moe.moe_norm_backward_workspace_bytes(moe.Norm(5, 256, moe.MOE_BF16, -1.0)) == 0
    assert moe.moe_norm_backward_workspace_bytes(moe.Norm(1 << 20, 7168, moe.MOE_BF16, 0.0)) >= 7168 * 4


def test_norm_without_its_descriptor():
    L = moe.lib()
    assert L.moe_norm(None, A, None, None, None, B, None, None, None) == -1
    assert L.moe_norm_backward(None, A, B, None, None, C, D, E, BIG, None) == -1
    assert L.moe_norm_backward_workspace_bytes(None) == 0
    assert L.moe_grouped_gemm(None, A, B, C, D, None, None) == -1
    assert L.moe_grouped_gemm_wgrad(None, A, B, C, D, 0, 0, None, 0, None, None) == -1
    assert L.moe_grouped_gemm_wgrad_workspace_bytes(None) == 0
    assert L.moe_adamw(None, None, 0, None) == -1


# ------------------------------------------------------------------------------------------------ dispatch of codes
def _codes(dtype=moe.MOE_MXFP8, El=8, **kw):
    a = dict(xq=[A, B], xq_scales=[A, B], pull_src=A, offsets=A, xe=C, xe_scales=D, ws=E, ws_bytes=BIG)
    shape = dict(R=2, T=64, d=1024, E=16, k=4, F=512)
    shape.update({n: kw.pop(n) for n in list(kw) if n in shape})
    a.update(kw)
    return moe.moe_dispatch_pull_codes(moe.Shape(*shape.values(), dtype), moe.Placement(A, El), *a.values(), stream=0, check=False)


@pytest.mark.parametrize("dtype", [moe.MOE_MXFP8, moe.MOE_MXFP4])
@pytest.mark.parametrize("kw,code", [
    (dict(xq=None), -1), (dict(xq=[A, None]), -1), (dict(xq=[A, B + 8]), -2), (dict(xq_scales=None), -1),
    (dict(xq_scales=[A, None]), -1), (dict(xq_scales=[A, B + 2]), -2), (dict(pull_src=None), -1), (dict(offsets=None), -1),
    (dict(xe=None), -1), (dict(xe=C + 8), -2), (dict(xe_scales=None), -1), (dict(xe_scales=D + 1), -2), (dict(ws=None), -1),
    (dict(ws=E + 64), -2), (dict(ws_bytes=64), -3), (dict(xe=B), -1), (dict(xe_scales=B), -1), (dict(k=0), -1), (dict(T=0), -1),
    (dict(R=65), -1), (dict(El=0), -1), (dict(d=1088), -2)])
def test_dispatch_of_codes(dtype, kw, code):
    assert _codes(dtype, **kw) == code


@pytest.mark.parametrize("dtype", [moe.MOE_F32, moe.MOE_BF16])
def test_dispatch_of_codes_takes_block_scaled_shapes_only(dtype):
    assert _codes(dtype) == -6


# ------------------------------------------------------------------------------------------------ products
GEMM = dict(rows=40, groups=4, K=64, N=72, dtype=moe.MOE_BF16, w_layout=0, ldx=0, ldy=0)


def _gemm(**kw):
    a = dict(x=A, w=B, offsets=C, y=D, status=None)
    g = dict(GEMM)
    g.update({n: kw.pop(n) for n in list(kw) if n in g})
    a.update(kw)
    return moe.moe_grouped_gemm(moe.Gemm(*g.values()), *a.values(), stream=0, check=False)


def _wgrad(**kw):
    a = dict(x=A, dy=B, offsets=C, dw=D, dw_dtype=moe.MOE_BF16, ws=E, ws_bytes=BIG, accumulate=False, status=None)
    g = dict(GEMM)
    g.update({n: kw.pop(n) for n in list(kw) if n in g})
    if g["dtype"] == moe.MOE_F32:
        a["dw_dtype"] = moe.MOE_F32
    a.update(kw)
    return moe.moe_grouped_gemm_wgrad(moe.Gemm(*g.values()), *a.values(), stream=0, check=False)


@pytest.mark.parametrize("call", [_gemm, _wgrad])
@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), -1), (dict(rows=1 << 31), -1), (dict(rows=(1 << 30) + 1), -1), (dict(groups=0), -1), (dict(groups=1025), -1), (dict(K=0), -1), (dict(N=0), -1),
    (dict(K=1 << 16, N=1 << 15), -1), (dict(K=(1 << 22) + 8, N=8), -1), (dict(w_layout=2), -1), (dict(w_layout=-1), -1),
    (dict(dtype=moe.MOE_MXFP8), -6), (dict(dtype=7), -6), (dict(K=60), -2), (dict(N=68), -2), (dict(dtype=moe.MOE_F32, K=62), -2),
    (dict(ldx=56), -1), (dict(ldy=64), -1), (dict(ldx=68), -2), (dict(ldy=76), -2), (dict(ldx=-8), -1), (dict(ldx=(1 << 22) + 8), -1),
    (dict(x=None), -1), (dict(x=A + 8), -2), (dict(offsets=None), -1), (dict(offsets=C + 2), -2), (dict(status=C + 2), -2)])
def test_product_limits(call, kw, code):
    assert call(**kw) == code


@pytest.mark.parametrize("kw,code", [(dict(w=None), -1), (dict(w=B + 8), -2), (dict(y=None), -1), (dict(y=D + 8), -2),
                                     (dict(y=A), -1), (dict(y=B), -1)])
def test_product_pointers(kw, code):
    assert _gemm(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), -1), (dict(dy=B + 8), -2), (dict(dw=None), -1), (dict(dw=D + 8), -2), (dict(dw=A), -1), (dict(dw=B), -1),
    (dict(dw_dtype=moe.MOE_MXFP8), -6), (dict(dtype=moe.MOE_F32, dw_dtype=moe.MOE_BF16), -6), (dict(accumulate=True), -1)])
def test_weight_gradient_pointers(kw, code):
    assert _wgrad(**kw) == code


# ------------------------------------------------------------------------------------------------ AdamW
STEP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1, state_dtype=moe.MOE_MXFP8, stochastic=1, seed=0, grad_scale=None,
            device_lr=None, device_step=None)
TENSOR = dict(param=A, grad=B, n=100, param_dtype=moe.MOE_BF16, grad_dtype=moe.MOE_BF16, m=C, v=D, m_scales=E, v_scales=E + 4096,
              master=None, weight_decay=0.1)


def _adamw(tensors=None, **kw):
    s, t = dict(STEP), dict(TENSOR)
    s.update({n: kw.pop(n) for n in list(kw) if n in s})
    t.update(kw)
    first = dict(TENSOR, n=0)                          # an empty tensor needs no pointers
    first.update(param=None, grad=None, m=None, v=None, m_scales=None, v_scales=None)
    return moe.moe_adamw(moe.AdamW(*s.values()), [moe.AdamWTensor(**first), moe.AdamWTensor(**t)], stream=0, check=False)


@pytest.mark.parametrize("kw,code", [
    (dict(lr=INF), -1), (dict(lr=NAN), -1), (dict(beta1=1.0), -1), (dict(beta1=-0.1), -1), (dict(beta2=1.0), -1), (dict(beta2=NAN), -1),
    (dict(eps=0.0), -1), (dict(eps=-1.0), -1), (dict(eps=1e-60), -1), (dict(eps=INF), -1), (dict(step=0), -1),
    (dict(state_dtype=moe.MOE_BF16), -6), (dict(grad_scale=A + 2), -2), (dict(device_lr=A + 2), -2), (dict(device_step=A + 4), -2),
    (dict(param=None), -1), (dict(param=A + 2), -2), (dict(grad=None), -1), (dict(grad=B + 8), -2), (dict(m=None), -1),
    (dict(m=C + 8), -2), (dict(v=None), -1), (dict(v=D + 8), -2), (dict(m_scales=None), -1), (dict(v_scales=E + 1), -2),
    (dict(master=A + 8), -2), (dict(master=A + 4096, param_dtype=moe.MOE_F32), -1), (dict(n=-1), -1), (dict(n=(1 << 40) + 1), -1),
    (dict(weight_decay=INF), -1), (dict(param_dtype=moe.MOE_MXFP8), -6), (dict(grad_dtype=5), -6),
    (dict(state_dtype=moe.MOE_F32, m=None), -1)])
def test_adamw_refusals(kw, code):
    assert _adamw(**kw) == code


@pytest.mark.parametrize("kw", [dict(grad=A), dict(m=A), dict(m=B), dict(v=C), dict(v=B), dict(master=A), dict(master=D), dict(m_scales=C),
                                dict(v_scales=E), dict(state_dtype=moe.MOE_F32, v=C)])
def test_adamw_refuses_a_buffer_in_two_places(kw):
    assert _adamw(**kw) == -1


def test_adamw_of_nothing():
    step = moe.AdamW(*STEP.values())
    assert moe.moe_adamw(step, [], stream=0) == 0
    empty = dict(TENSOR, n=0, param=None, grad=None, m=None, v=None, m_scales=None, v_scales=None)
    assert moe.moe_adamw(step, (moe.AdamWTensor(**empty) for _ in range(50)), stream=0) == 0
    assert moe.lib().moe_adamw(ctypes.byref(step), None, 1, None) == -1
    assert moe.lib().moe_adamw(ctypes.byref(step), None, -1, None) == -1


def test_wgrad_in_pieces_asks_for_its_workspace():
    """One matrix of 256 x 512 (2 tiles) with 100000 rows: pieces of 1024, 129 at most for any number of rows; groups that fill the card, or few
    rows: none."""
    g = moe.Gemm(100000, 1, 256, 512, moe.MOE_BF16, 0)
    need = moe.moe_grouped_gemm_wgrad_workspace_bytes(g)
    assert need == 768 + 130 * 256 * 512 * 4
    call = lambda **kw: moe.moe_grouped_gemm_wgrad(g, A, B, C, D, moe.MOE_BF16, stream=0, check=False, **kw)       # noqa: E731
    assert call() == -1 and call(ws=E + 64, ws_bytes=need) == -2 and call(ws=E, ws_bytes=98 * 256 * 512 * 4) == -3
    assert moe.moe_grouped_gemm_wgrad_workspace_bytes(moe.Gemm(100000, 64, 7168, 2048, moe.MOE_BF16, 0)) == 0
    assert moe.moe_grouped_gemm_wgrad_workspace_bytes(moe.Gemm(2047, 1, 256, 512, moe.MOE_BF16, 0)) == 0


@pytest.mark.parametrize("dtype", [moe.MOE_BF16, moe.MOE_F32])
@pytest.mark.parametrize("G,K,N", [(1, 256, 512), (1, 7168, 256), (12, 440, 368), (8, 1024, 1024), (1000, 64, 64), (1023, 8, 8), (3, 2048, 2048)])
def test_a_wgrad_workspace_for_more_rows_serves_fewer(dtype, G, K, N):
    size = lambda rows: moe.moe_grouped_gemm_wgrad_workspace_bytes(moe.Gemm(rows, G, K, N, dtype, 0))              # noqa: E731
    rows = sorted({int(1.03 ** i) + d for i in range(60, 700) for d in (-1, 0, 1) if 1.03 ** i < 1 << 29} | {1 << i for i in range(6, 30)})
    sizes = [size(r) for r in rows]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("eps,code", [(2.0 ** -126, 0), (1.1e-38, -1), (1e-39, -1), (1e-45, -1), (2.0 ** 126, 0), (1e38, -1), (1e39, -1), (1e300, -1)])
def test_adamw_takes_an_eps_whose_reciprocal_is_a_normal_float(eps, code):
    """The step multiplies by the reciprocal of root + eps: of a subnormal eps it would be infinite, and 0 times it a NaN; of a larger one zero."""
    assert moe.moe_adamw(moe.AdamW(*dict(STEP, eps=eps).values()), [], stream=0, check=False) == code


@pytest.mark.parametrize("lr,code", [(3e38, 0), (4e38, -1), (-4e38, -1), (1e300, -1)])
def test_adamw_takes_a_rate_that_fp32_holds(lr, code):
    assert moe.moe_adamw(moe.AdamW(*dict(STEP, lr=lr).values()), [], stream=0, check=False) == code


@pytest.mark.parametrize("dtype,rows,G,K,N", [(moe.MOE_BF16, 32768, 8, 7168, 2048), (moe.MOE_BF16, 32768, 1, 8192, 8192),
                                              (moe.MOE_BF16, 131072, 32, 7168, 2048), (moe.MOE_BF16, 16384, 8, 1024, 1024),
                                              (moe.MOE_BF16, 262144, 1, 4096, 4096), (moe.MOE_F32, 54882, 162, 2016, 7176),
                                              (moe.MOE_F32, 16563, 17, 7620, 2336), (moe.MOE_BF16, 1 << 30, 1024, 8, 8)])
def test_no_workspace_where_no_rows_use_one(dtype, rows, G, K, N):
    """Matrices of so many tiles, or with so large sums, that no number of rows up to these goes in pieces."""
    assert moe.moe_grouped_gemm_wgrad_workspace_bytes(moe.Gemm(rows, G, K, N, dtype, 0)) == 0


def test_a_kept_table_takes_new_gradients():
    table = moe.adamw_table([moe.AdamWTensor(**TENSOR), moe.AdamWTensor(**dict(TENSOR, n=0))])
    step = moe.AdamW(*STEP.values())
    table[0].grad = B + 8
    assert moe.moe_adamw(step, table, stream=0, check=False) == -2
    table[0].grad = A
    assert moe.moe_adamw(step, table, stream=0, check=False) == -1 and table[0].param == A and table[0].n == 100
