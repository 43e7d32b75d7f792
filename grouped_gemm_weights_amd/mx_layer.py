"""Host orchestration of the MoE block in 8 bits on one GPU, through the C ABI.

``MxMoELayer`` owns the device buffers of one block whose expert weights and activations are 8-bit rows
with block scales (include/moe.h, "mx") and issues the library calls of one inference step on its
compute stream:

    norm:     moe_rms_norm         x + residual -> sum, xn (for the router), q and scales
    forward:  moe_route -> moe_permute (no row copy)
              -> moe_grouped_gemm_mx (gate and up, rows gathered) -> moe_mx_quantize (SwiGLU)
              -> moe_grouped_gemm_mx (down) -> moe_combine
              -> moe_dropout_add (p = 0: the sum and the block's output, rounded once)

An expert's block holds its gate and up rows as one matrix of 2 I rows, its down rows, and the scales of
both: a quarter of an f32 block and about half of a bf16 one.  The blocks are a merged buffer like the
bf16 layer's, so the pulls of ``moe_prefetch_layer`` and ``moe_prefetch_routed`` can fill it from pools of
such blocks too.
"""
from __future__ import annotations

import torch

from . import binding as B
from .synth import MoEConfig


class MxMoELayer:
    """Buffers of one 8-bit MoE block of shape ``cfg``, all experts resident on ``device``.

    Set ``x`` and ``residual`` ([T, H] in the layer's dtype), ``gamma`` (f32 [H]) and, after ``norm``,
    ``logits`` (f32 [T, E]); ``forward`` leaves the block's output in ``y`` (f32) and the new stream
    in ``out``.

    Experts are filled by ``load_expert``, by a pull into ``wbuf``, or by the caller in ``blocks``.  One
    that never was holds NaN, and so does the output of every token that is routed to it.
    """

    def __init__(self, cfg: MoEConfig, device="cuda", compute_stream=None, eps: float = 1e-6):
        T, E, k, H, I = cfg.T, cfg.E, cfg.k, cfg.H, cfg.I
        if H % 32 != 0 or I % 32 != 0:
            raise ValueError(f"8-bit rows are blocks of 32: H={H} and I={I} must be multiples of it")
        self.cfg, self.eps, self.dev = cfg, eps, torch.device(device)
        self.dt = B.MOE_F32 if cfg.dtype == "f32" else B.MOE_BF16
        self.R = R = T * k
        d = self.dev
        u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device=d)
        i32 = lambda *s: torch.empty(s, dtype=torch.int32, device=d)
        f32 = lambda *s: torch.empty(s, dtype=torch.float32, device=d)
        own = lambda *s: torch.empty(s, dtype=torch.float32 if cfg.dtype == "f32" else torch.bfloat16, device=d)
        self.x, self.residual, self.sum, self.xn, self.out = (own(T, H) for _ in range(5))
        self.gamma, self.rstd, self.logits = torch.ones(H, dtype=torch.float32, device=d), f32(T), f32(T, E)
        self.q, self.scales = u8(T, H), u8(T, B.moe_mx_scale_pitch(H))
        self.topk_idx, self.topk_w = i32(T, k), f32(T, k)
        self.counts, self.offsets, self.row_of, self.src_of = i32(E), i32(E + 1), i32(R), i32(R)
        self.gate_up = own(R, 2 * I)
        self.h, self.h_scales = u8(R, I), u8(R, B.moe_mx_scale_pitch(I))
        self.y_perm, self.y = f32(R, H), f32(T, H)
        self.status = torch.zeros(1, dtype=torch.int32, device=d)
        self.ws_bytes = B.moe_permute_workspace_size(T, E, k)
        self.ws = u8(max(1, self.ws_bytes))
        self._rng = torch.zeros(2, dtype=torch.int64, device=d)      # never drawn from: nothing is dropped
        # an expert's block: gate and up, down, their scales
        self.down_off = 2 * I * H
        self.up_scales_off = self.down_off + H * I
        self.down_scales_off = self.up_scales_off + 2 * I * B.moe_mx_scale_pitch(H)
        self.expert_bytes = self.down_scales_off + H * B.moe_mx_scale_pitch(I)
        # 0x7f is e4m3's NaN, with the scale 2^0: an expert that nobody filled does not pass for weights
        self.blocks = u8(E, self.expert_bytes).fill_(0x7F)
        self.slot_of = torch.arange(E, dtype=torch.int32, device=d)
        self.wbuf = B.wbuf(self.blocks, self.expert_bytes, E, E, self.slot_of)
        self.compute_stream = compute_stream or torch.cuda.Stream(device=d)
        torch.cuda.current_stream(d).synchronize()   # buffers initialised on torch's stream

    def load_expert(self, e: int, block: torch.Tensor) -> None:
        """Compute stream: expert e's weights to 8 bits, from its block [3 * H * I] (Wg | Wu | Wd) in the
        layer's dtype on the device, written on torch's current stream, which may write the next one to the
        same place after this call."""
        cfg, cs = self.cfg, self.compute_stream
        if not 0 <= e < cfg.E:
            raise ValueError(f"expert {e} outside [0, {cfg.E})")
        if block.numel() != 3 * cfg.H * cfg.I or block.dtype != self.x.dtype or not block.is_contiguous() or \
                block.device != self.x.device:
            raise ValueError(f"an expert's block is {3 * cfg.H * cfg.I} contiguous {self.x.dtype} values on "
                             f"{self.x.device}")
        current = torch.cuda.current_stream(self.dev)
        cs.wait_stream(current)
        block.record_stream(cs)
        at, src = self.blocks[e].data_ptr(), block.data_ptr()
        B.moe_mx_quantize(src, 2 * cfg.I, cfg.H, self.dt, 0, at, at + self.up_scales_off, cs)
        B.moe_mx_quantize(src + 2 * cfg.I * cfg.H * block.element_size(), cfg.H, cfg.I, self.dt, 0,
                          at + self.down_off, at + self.down_scales_off, cs)
        current.wait_stream(cs)

    def norm(self) -> None:
        """Compute stream: ``sum`` = x + residual, ``xn`` its norm, and the same in 8 bits."""
        cfg = self.cfg
        B.moe_rms_norm(self.x, self.residual, self.gamma, cfg.T, cfg.H, self.eps, self.dt, self.sum, self.xn,
                       self.q, self.scales, self.rstd, self.compute_stream)

    def forward(self) -> None:
        """Compute stream: from ``logits`` and the rows that ``norm`` left, ``y`` and ``out`` = sum + y."""
        cfg, cs = self.cfg, self.compute_stream
        T, E, k, H, I, R = cfg.T, cfg.E, cfg.k, cfg.H, cfg.I, self.R
        B.moe_route(self.logits, T, E, k, self.topk_idx, self.topk_w, self.status, cs)
        B.moe_permute(self.topk_idx, T, E, k, None, H, self.dt, self.counts, self.offsets, self.row_of,
                      self.src_of, None, self.ws, self.ws_bytes, self.status, cs)
        B.moe_grouped_gemm_mx(self.q, self.scales, self.src_of, k, self.offsets, R, E, H, 2 * I, self.wbuf, 0,
                              self.up_scales_off, self.dt, self.gate_up, self.status, cs)
        B.moe_mx_quantize(self.gate_up, R, I, self.dt, 1, self.h, self.h_scales, cs)
        B.moe_grouped_gemm_mx(self.h, self.h_scales, None, 0, self.offsets, R, E, I, H, self.wbuf,
                              self.down_off, self.down_scales_off, B.MOE_F32, self.y_perm, self.status, cs)
        B.moe_combine(self.y_perm, self.row_of, self.topk_w, T, k, H, self.y, cs)
        B.moe_dropout_add(self.y, B.MOE_F32, self.sum, T * H, 0.0, self._rng, self.dt, self.out, cs)

    def capture(self) -> torch.cuda.CUDAGraph:
        """``forward`` as one HIP graph (run it once before); ``norm`` and the router stay with the caller."""
        self.compute_stream.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=self.compute_stream):
            self.forward()
        return g

    def read_status(self) -> int:
        self.compute_stream.synchronize()
        return int(self.status.item())
