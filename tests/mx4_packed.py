"""A layer of given choices over MXFP4 experts whose weights are random codes (no host weights to quantise)."""
import numpy as np

from mixture_experts_layer_histogram_amd import moe


class Packed:
    """Device buffers; x: rows of one rank."""

    def __init__(self, T, d, F, E, k, seed=0, x=None):
        import torch
        self.torch = torch
        g = self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.d, self.F, self.E, self.k = T, d, F, E, k
        self.shape = moe.Shape(1, T, d, E, k, F, moe.MOE_MXFP4)
        self.e2l = torch.arange(E, dtype=torch.int32, device="cuda")
        self.placement = moe.Placement(self.e2l.data_ptr(), E)
        self.ex = None
        self.w, scales = [], []
        for rows, K in ((F, d), (F, d), (d, F)):
            codes = torch.randint(0, 256, (E, rows, K // 2), dtype=torch.uint8, device="cuda", generator=g)
            top = 126 - int(round(np.log2(K) / 2))          # values of some K ** -0.5
            sc = torch.randint(top - 3, top, (K // 128, E * rows, 4), dtype=torch.uint8, device="cuda", generator=g)
            self.w.append(codes)
            scales.append(sc)
        self.scale_codes = scales
        self.w_scales = moe.MXScales(*(t.data_ptr() for t in scales))
        self.x = [torch.randn(T, d, device="cuda", generator=g).to(torch.bfloat16) if x is None else x]
        n = self.nmax = moe.moe_max_pairs(self.shape, self.placement)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.counts, self.offsets = torch.empty(E, **i32), torch.empty(E + 1, **i32)
        self.pull_src, self.slot_of = torch.empty((n, 2), **i32), torch.empty((1, T, k), **i32)
        self.ws = torch.full((moe.moe_workspace_bytes(self.shape, self.placement),), 0x5A, dtype=torch.uint8, device="cuda")
        self.xe = torch.empty((n, d // 2), dtype=torch.uint8, device="cuda")
        self.xe_scales = torch.empty((d // 128, n, 4), dtype=torch.uint8, device="cuda")
        self.y = [torch.full((T, d), float("nan"), dtype=torch.bfloat16, device="cuda")]
        self.ye = None

    def rows(self):
        """ye, allocated on first use."""
        if self.ye is None:
            self.ye = self.torch.full((self.nmax, self.d), float("nan"), dtype=self.torch.bfloat16, device="cuda")
        return self.ye

    def status(self):
        return moe.moe_read_status(self.ws)

    def layout(self, idx):
        moe.moe_layout_choices(self.shape, self.placement, None, idx, self.counts, self.offsets, self.pull_src, self.slot_of,
                               self.ws)

    def dispatch(self):
        moe.moe_dispatch_pull(self.shape, self.placement, self.x, self.pull_src, self.offsets, self.xe, self.ws,
                              xe_scales=self.xe_scales)

    def ffn(self):
        moe.moe_expert_ffn(self.shape, self.placement, None, self.xe, self.offsets, *self.w, self.rows(), self.ws,
                           w_scales=self.w_scales, xe_scales=self.xe_scales)

    def push(self, w):
        """The merged rows of the product with the push fused into it."""
        recv = [self.torch.full((self.T, self.k, self.d), float("nan"), dtype=self.torch.bfloat16, device="cuda")]
        moe.moe_expert_ffn_push(self.shape, self.placement, None, self.xe, self.offsets, *self.w, self.pull_src, self.slot_of,
                                recv, self.ws, w_scales=self.w_scales, xe_scales=self.xe_scales)
        y = [self.torch.full_like(self.y[0], float("nan"))]
        moe.moe_weighted_merge(self.shape, self.placement, self.slot_of, w, recv, y)
        return y[0]

    def forward_choices(self, idx, w, ws_bytes=None):
        moe.moe_forward_choices(self.shape, self.placement, None, idx, w, self.x, *self.w, self.xe, self.rows(), self.y,
                                self.counts, self.offsets, self.pull_src, self.slot_of, self.ws, ws_bytes=ws_bytes,
                                w_scales=self.w_scales, xe_scales=self.xe_scales)

    def weights64(self, e):
        """Expert e's W1, W3, W2 in 64 bits."""
        torch, out = self.torch, []
        table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.double, device="cuda")
        for codes, sc in zip(self.w, self.scale_codes):
            rows, half = codes.shape[1:]
            v = table[torch.stack((codes[e] & 15, codes[e] >> 4), -1).long()].reshape(rows, 2 * half)
            unit = torch.exp2(sc[:, e * rows:(e + 1) * rows].permute(1, 0, 2).reshape(rows, -1).double() - 127)
            out.append((v * unit.repeat_interleave(32, 1)).cpu().numpy())
        return out
