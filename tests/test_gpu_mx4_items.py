"""GPU parity of the MXFP4 expert products where a wave or a workgroup takes several items or tiles.

The streaming kernel gives an item (64 weight rows of an expert) to a wave where there are 4 of them for each
CU, else to a workgroup whose waves share its K; the tile kernel walks the tiles of 256 rows with one
workgroup a CU.  The sizes here make every one of them go from item to item with fills in flight, over
unequal row counts, half units of K, half stages and half columns, with rows out in bf16, in fp32 and through the
fused push.  Bars: the per-element allowance of _bound in 64 bits, as in test_gpu_mx4.
"""
import numpy as np
import pytest

from oracle import mx4_oracle as M4
from tests.mx4_packed import Packed
from tests.test_gpu_mx4 import _bound, _check_merged, _torch
from mixture_experts_layer_histogram_amd import moe

pytestmark = pytest.mark.gpu


def _choices(T, k, counts):
    """Choices [1][T][k] that give expert e counts[e] rows (at most T), no token an expert twice, -1 elsewhere."""
    idx = np.full((T, k), -1, dtype=np.int32)
    fill, at = np.zeros(T, dtype=int), 0
    for e, c in enumerate(counts):
        assert c <= T
        for i in range(c):
            t = (at + i) % T
            idx[t, fill[t]] = e
            fill[t] += 1
        at = (at + c) % T
    assert np.array_equal(np.bincount(idx[idx >= 0], minlength=len(counts)), counts)
    return idx[None]


def _references(P):
    """Rows in 64 bits and their allowance, from the codes that the gather left (checked against the oracle)."""
    off, src = P.offsets.cpu().numpy(), P.pull_src.cpu().numpy()
    N = int(off[-1])
    x = P.x[0].double().cpu().numpy()
    codes, sc, val = M4.quantize(x)
    assert np.array_equal(M4.unpack(P.xe[:N].cpu().numpy()), codes[src[:N, 1]])
    assert np.array_equal(P.xe_scales[:, :N].permute(1, 0, 2).reshape(N, -1).cpu().numpy(), sc[src[:N, 1]])
    ref, allow = np.zeros((N, P.d)), np.zeros((N, P.d))
    for e in range(P.E):
        a, b = int(off[e]), int(off[e + 1])
        if a < b:
            ref[a:b], allow[a:b] = _bound(val[src[a:b, 1]], *P.weights64(e))
    return ref, allow


def _every_form(P, counts, name):
    torch = _torch()
    idx = torch.from_numpy(_choices(P.T, P.k, counts)).cuda()
    w = torch.rand(1, P.T, P.k, device="cuda", generator=P.gen) - 0.5
    print(f"[mx4 items] {name}: T {P.T} d {P.d} F {P.F} E {P.E} k {P.k}, rows {sum(counts)}", flush=True)
    P.layout(idx)
    P.dispatch()
    P.ffn()                                    # bf16 rows
    assert P.status() == 0 and P.counts.tolist() == list(counts)
    ref, allow = _references(P)
    N = len(ref)
    got = P.ye[:N].double().cpu().numpy()
    lim = allow + (np.abs(ref) + allow) * 2.0 ** -8 + 1e-38
    err = np.abs(got - ref)
    assert (err <= lim).all(), (float((err / lim).max()), np.argwhere(err > lim)[:4].tolist())
    print(f"[mx4 items] {name}: relative error {np.linalg.norm(got - ref) / np.linalg.norm(ref):.2e}", flush=True)
    assert torch.isnan(P.ye[N:]).all()
    y = torch.full_like(P.y[0], float("nan"))
    moe.moe_combine_merge(P.shape, P.placement, P.ye, P.slot_of, w, [y])
    rows = P.ye.clone()
    for _ in range(2):                         # the same bits again, and through the fused push
        P.ye.fill_(float("nan"))
        P.ffn()
        assert torch.equal(P.ye[:N], rows[:N])
        assert torch.equal(P.push(w), y)
    assert P.nmax * P.d * 4 <= 16 << 20        # fp32 rows
    P.ye.fill_(float("nan"))
    P.forward_choices(idx, w)
    assert P.status() == 0 and torch.isnan(P.ye).all()
    _check_merged(P, ref, allow, w)
    first = P.y[0].clone()
    for _ in range(3):
        P.y[0].fill_(float("nan"))
        P.forward_choices(idx, w)
        assert torch.equal(P.y[0], first)
    need = P.ws.numel() - P.nmax * P.d * 4     # without room for them: bf16 rows in ye
    P.forward_choices(idx, w, ws_bytes=need)
    assert P.status() == 0 and torch.equal(P.y[0], y) and torch.equal(P.ye[:N], rows[:N])


UNEQUAL = [32, 0, 31, 1, 17, 32, 5, 0, 24, 2, 30, 16, 0, 0, 9, 32]


@pytest.mark.parametrize("T,d,F,E,k", [(120, 1152, 896, 64, 8),      # a wave an item, one or two of them
                                       (200, 2176, 896, 96, 8),      # a wave an item, two to four
                                       (64, 1152, 384, 32, 8),       # a workgroup an item, two or three; waves without units
                                       (33, 4224, 128, 16, 8)])      # 64 and 1056 items: a workgroup, then a wave
def test_streaming_from_item_to_item(T, d, F, E, k):
    counts = [UNEQUAL[(5 * e) % 16] if e % 3 else UNEQUAL[e % 16] for e in range(E)]
    P = Packed(T, d, F, E, k, seed=T)
    assert max(counts) == 32 and T * k <= 20 * E and sum(counts) <= T * k
    _every_form(P, counts, "streaming")


@pytest.mark.parametrize("T,d,F,E,k", [(200, 2176, 896, 96, 8), (120, 1152, 384, 64, 8)])
def test_streaming_beside_tiles(T, d, F, E, k):
    """Most experts have few rows, a handful 33 to T: both product kernels, each on its own experts."""
    counts = [UNEQUAL[(7 * e) % 16] // 2 for e in range(E)]
    for i, e in enumerate((0, 11, E // 2, E - 1)):
        counts[e] = (33, T, 64, 100)[i]
    assert T * k <= 20 * E and sum(counts) <= T * k
    _every_form(Packed(T, d, F, E, k, seed=T + 1), counts, "streaming and tiles")


@pytest.mark.parametrize("T,d,F,E,k", [(4096, 256, 128, 512, 4), (4096, 256, 384, 512, 4), (4096, 256, 896, 512, 4),
                                       (1600, 640, 256, 256, 4), (2048, 512, 1152, 400, 4), (4096, 256, 512, 1024, 4)])
def test_tiles_of_fp32_rows_from_tile_to_tile(T, d, F, E, k):
    """Two to four tiles a workgroup below 16 MiB of rows: experts of two whole tiles, spread over the list so that
    every XCD's range begins with some, then partial ones; one, two and more stages, half stages, half columns.
    The last case leaves experts of up to 32 rows to the streaming kernel and the tiles of some 250 others."""
    torch = _torch()
    few = T * k <= 20 * E
    heavy = min(512, T)
    counts = np.zeros(E, dtype=int)
    counts[:: E // 8] = heavy
    rest = counts == 0
    if few:
        counts[rest] = np.where(np.arange(rest.sum()) % 4 == 0, 40, 1 + np.arange(rest.sum()) % 3)
    else:
        counts[rest] = (T * k - counts.sum()) // rest.sum() - 1
        counts[np.flatnonzero(rest)[::2]] += 1
    assert counts.sum() <= T * k
    tiles = int(sum((c + 255) // 256 for c in counts if c > (32 if few else 0))) * ((d + 255) // 256)
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert tiles > cus
    _every_form(Packed(T, d, F, E, k, seed=F), [int(c) for c in counts], f"tiles ({tiles})")
