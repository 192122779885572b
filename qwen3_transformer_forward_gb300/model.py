"""Qwen3 forward pass on one GB300: sequences the libqw entry points.

This module does no arithmetic of the model.  It owns device buffers (via
PyTorch), builds the tensor-parallel weight layout at load time, and calls
one C-ABI entry point per step, in the order of Qwen3DecoderLayer.forward
and Qwen3ForCausalLM ([SK] §1, §8; [VH] §3-§5):

  embed (vocab-parallel) -> per layer:
     add+RMSNorm -> QKV GEMM (column) -> QK-norm + RoPE + KV store ->
     attention (prefill: varlen causal; decode: over the cache) ->
     o_proj GEMM (row, shard sum) -> add+RMSNorm ->
     gate_up GEMM (column) with fused SiluAndMul -> down GEMM (row, shard sum)
  -> final add+RMSNorm -> lm_head (last token per sequence in prefill) -> argmax

Sources: [VH] devpress "vocab 切 / head 切"; [TP] devpress tensor-parallel
maths; [SK] AIInfraGuide "3.3 模型骨架与核心算子".
"""
from __future__ import annotations

import contextlib
import dataclasses
from dataclasses import dataclass, field
from typing import Dict, List, Optional

import torch

from . import _lib as L


# ----------------------------------------------------------------------------
# load-time layout (the weight_loader of the parallel Linear family)
# ----------------------------------------------------------------------------

@dataclass(frozen=True)
class W4Config:
    """Linear weights in 4 bits (bf16 models): codes with a scale for each row and `group` columns.

    zeros: a zero point for each group too (asymmetric).  table: the tied embedding / lm_head table as well.
    """
    group: int = 128          # 32, 64 or 128; it divides the columns of every shard's rows
    zeros: bool = False
    table: bool = True


@dataclass
class W4Weight:
    """A weight of N stored rows of K columns in 4 bits (the format of qw_w4_quantize); a row split has tp * N rows."""
    codes: torch.Tensor              # uint8 [N, K/2]
    scales: torch.Tensor             # bf16 [N, K/group]
    zeros: Optional[torch.Tensor]    # uint8 [N, K/group]
    group: int


def w4_weight(w: torch.Tensor, c: W4Config) -> W4Weight:
    """Quantises a bf16 weight [..., K] on its device."""
    w = w.reshape(-1, w.shape[-1])
    N, K = w.shape
    new = lambda cols, dt: torch.empty(N, cols, dtype=dt, device=w.device)  # noqa: E731
    q = W4Weight(new(K // 2, torch.uint8), new(K // c.group, torch.bfloat16),
                 new(K // c.group, torch.uint8) if c.zeros else None, c.group)
    L.w4_quantize(w, c.group, q.codes, q.scales, q.zeros)
    return q


@dataclass
class LayerParams:
    # qkv, o, gate_up and down may be W4Weight: the same rows in 4 bits
    qkv: torch.Tensor        # [tp * (nh/tp + 2 nkv/tp) * hd, H]   shard r = [q_r; k_r; v_r]
    o: torch.Tensor          # [tp, H, nh/tp * hd]                 shard r = input columns of its heads
    gate_up: torch.Tensor    # [tp * 2 * I/tp, H]                  shard r = [gate_r; up_r]
    down: torch.Tensor       # [tp, H, I/tp]
    input_ln: torch.Tensor
    post_ln: torch.Tensor
    q_norm: torch.Tensor
    k_norm: torch.Tensor


@dataclass
class ModelParams:
    embed: torch.Tensor      # [V, H] (or W4Weight); tied with the lm_head ([SK] §8); shard r = row block r
    layers: List[LayerParams]
    final_norm: torch.Tensor


def shard_layer(shape, ck: Dict[str, torch.Tensor], layer: int, device) -> LayerParams:
    """Places one layer's checkpoint tensors into the per-shard stacked layout.

    QKVParallelLinear / MergedColumnParallelLinear narrow each checkpoint
    tensor along the output dim per shard; RowParallelLinear narrows along the
    input dim ([SK] §5, [TP] §3-§4).  Runs once at load time.
    """
    tp, hd = shape.tp, shape.head_dim
    nh_l, nkv_l, i_l = shape.n_heads // tp, shape.n_kv_heads // tp, shape.intermediate // tp
    p = f"layer{layer}."
    wq, wk, wv = ck[p + "q_proj"], ck[p + "k_proj"], ck[p + "v_proj"]
    wg, wu = ck[p + "gate_proj"], ck[p + "up_proj"]
    qkv = torch.cat([torch.cat([wq.narrow(0, r * nh_l * hd, nh_l * hd), wk.narrow(0, r * nkv_l * hd, nkv_l * hd),
                                wv.narrow(0, r * nkv_l * hd, nkv_l * hd)]) for r in range(tp)])
    gate_up = torch.cat([torch.cat([wg.narrow(0, r * i_l, i_l), wu.narrow(0, r * i_l, i_l)]) for r in range(tp)])
    wo, wd = ck[p + "o_proj"], ck[p + "down_proj"]
    o = torch.stack([wo.narrow(1, r * nh_l * hd, nh_l * hd) for r in range(tp)])
    down = torch.stack([wd.narrow(1, r * i_l, i_l) for r in range(tp)])

    def dev(t):
        return t.contiguous().to(device)
    return LayerParams(dev(qkv), dev(o), dev(gate_up), dev(down), dev(ck[p + "input_layernorm"]),
                       dev(ck[p + "post_attention_layernorm"]), dev(ck[p + "q_norm"]), dev(ck[p + "k_norm"]))


def w4_layer(p: LayerParams, c: W4Config) -> LayerParams:
    """The layer with its four linear weights in 4 bits."""
    return dataclasses.replace(p, **{n: w4_weight(getattr(p, n), c) for n in ("qkv", "o", "gate_up", "down")})


def w4_params(p: ModelParams, c: W4Config) -> ModelParams:
    """The parameters with their linear weights, and the tied table, in 4 bits."""
    return ModelParams(w4_weight(p.embed, c) if c.table else p.embed, [w4_layer(l, c) for l in p.layers], p.final_norm)


def load_params(shape, seed: int = 0, device="cuda", n_layers: Optional[int] = None, gen_device=None,
                w4: Optional[W4Config] = None) -> ModelParams:
    """Random-init parameters of the given shape from the seeded generator; w4: quantised layer by layer as they load."""
    import seeded_inputs as si
    gen_device = gen_device or device
    nl = shape.n_layers if n_layers is None else n_layers
    embed = si.checkpoint_tensor(shape, "embed_tokens", seed, gen_device).to(device)
    layers = []
    for l in range(nl):
        ck = {n: si.checkpoint_tensor(shape, n, seed, gen_device)
              for n in si.weight_names(l) + [f"layer{l}.{x}" for x in
                                             ("input_layernorm", "post_attention_layernorm", "q_norm", "k_norm")]}
        layer = shard_layer(shape, ck, l, device)
        layers.append(layer if w4 is None else w4_layer(layer, w4))
        del ck, layer
    final = si.checkpoint_tensor(shape, "norm", seed, gen_device).to(device)
    return ModelParams(w4_weight(embed, w4) if w4 is not None and w4.table else embed, layers, final)


# ----------------------------------------------------------------------------
# batch descriptions (the get_context() fields, [SK] §6-§7)
# ----------------------------------------------------------------------------

@dataclass(frozen=True)
class Kv8Config:
    """An 8-bit paged KV cache in place of the bf16 one (bf16 models with head_dim 128).

    The contexts of such a model carry a block_table (int32 [S, max_blocks]) and
    context_lens; slot_mapping and seq_base are not read.  window > 0: every layer
    sees the last `window` keys and the first n_sink.
    """
    kv_dtype: torch.dtype = torch.int8    # or torch.float8_e4m3fn
    block_size: int = 256
    scale_block: int = 64
    window: int = 0
    n_sink: int = 0


@dataclass
class PrefillContext:
    ids: torch.Tensor            # int64 [T]
    positions: torch.Tensor      # int64 [T]
    cu_seqlens: torch.Tensor     # int32 [S+1]
    slot_mapping: torch.Tensor   # int64 [T]
    seq_base: torch.Tensor       # int32 [S]
    last_idx: torch.Tensor       # int32 [S]
    max_seqlen: int
    block_table: Optional[torch.Tensor] = None    # int32 [S, max_blocks] (8-bit paged cache)
    context_lens: Optional[torch.Tensor] = None   # int32 [S]: cached keys, the new tokens included
    max_context: int = 0                          # >= every context_lens

    @property
    def n_tokens(self):
        return self.ids.shape[0]


@dataclass
class DecodeContext:
    ids: torch.Tensor            # int64 [B]
    positions: torch.Tensor      # int64 [B]
    context_lens: torch.Tensor   # int32 [B]
    slot_mapping: torch.Tensor   # int64 [B]
    seq_base: torch.Tensor       # int32 [B]
    max_context: int
    block_table: Optional[torch.Tensor] = None    # int32 [B, max_blocks] (8-bit paged cache)

    @property
    def n_tokens(self):
        return self.ids.shape[0]


def to_device_prefill(b, device="cuda", block_table=None, context_lens=None) -> PrefillContext:
    """block_table (8-bit paged cache): the prompts are whole, or context_lens counts the cached keys before them too."""
    ctx = PrefillContext(b.ids.to(device), b.positions.to(device), b.cu_seqlens.to(device),
                         b.slot_mapping.to(device), b.seq_base.to(device), b.last_idx.to(device), max(b.seq_lens))
    if block_table is not None:
        lens = torch.tensor(b.seq_lens, dtype=torch.int32) if context_lens is None else context_lens
        ctx.block_table, ctx.context_lens = block_table.to(device), lens.to(device)
        ctx.max_context = int(lens.max())
    return ctx


def to_device_decode(b, device="cuda", block_table=None) -> DecodeContext:
    """block_table: for the 8-bit paged cache."""
    return DecodeContext(b.ids.to(device), b.positions.to(device), b.context_lens.to(device),
                         b.slot_mapping.to(device), b.seq_base.to(device), int(b.context_lens.max()),
                         None if block_table is None else block_table.to(device))


# ----------------------------------------------------------------------------
# the forward pass
# ----------------------------------------------------------------------------

class Qwen3Forward:
    """Device buffers + the sequence of libqw calls for prefill and decode."""

    def __init__(self, shape, params: ModelParams, max_tokens: int, num_slots: int, max_seqs: int,
                 max_context: int, device="cuda", kv_caches=None, kv8: Optional[Kv8Config] = None):
        """kv_caches: (k, v), lists of one tensor per layer; with kv8 (k, v, k_scale, v_scale)."""
        self.m = shape
        self.p = params
        self.device = device
        dt = params.final_norm.dtype
        self.dtype = dt
        H, I, hd = shape.hidden, shape.intermediate, shape.head_dim
        tp = shape.tp
        self.qkv_width = tp * (shape.n_heads // tp + 2 * (shape.n_kv_heads // tp)) * hd
        T = max_tokens
        z = lambda *s: torch.empty(*s, dtype=dt, device=device)  # noqa: E731
        self.h = z(T, H)
        self.res = z(T, H)
        self.res2 = z(max(max_seqs, 1), H)   # decode: the residual alternates between res and res2
        self.y = z(T, H)
        self.qkv = z(T, self.qkv_width)
        self.q = z(T, shape.n_heads * hd)
        self.attn = z(T, shape.n_heads * hd)
        self.act = z(T, I)
        self.logits = z(max_seqs if max_seqs > 0 else T, shape.vocab)
        self.next_tokens = torch.empty(max(max_seqs, T), dtype=torch.int64, device=device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        nl = len(params.layers)
        self.kv8 = kv8
        self.k_scale, self.v_scale = [], []
        if kv8 is not None:
            if dt != torch.bfloat16 or hd != 128:
                raise ValueError("the 8-bit KV cache is for bf16 models with head_dim 128")
            if kv_caches is None:
                codes = lambda: [torch.zeros(num_slots, shape.n_kv_heads, hd, dtype=torch.int8,  # noqa: E731
                                             device=device).view(kv8.kv_dtype) for _ in range(nl)]
                scales = lambda: [torch.zeros(num_slots // kv8.scale_block, shape.n_kv_heads, dtype=torch.float32,  # noqa: E731
                                              device=device) for _ in range(nl)]
                kv_caches = codes(), codes(), scales(), scales()
            self.k_cache, self.v_cache, self.k_scale, self.v_scale = kv_caches
        elif kv_caches is None:
            self.k_cache = [torch.zeros(num_slots, shape.n_kv_heads, hd, dtype=dt, device=device) for _ in range(nl)]
            self.v_cache = [torch.zeros(num_slots, shape.n_kv_heads, hd, dtype=dt, device=device) for _ in range(nl)]
        else:
            self.k_cache, self.v_cache = kv_caches
        self.cos_sin = L.rope_cos_sin_table(shape.max_position, hd, shape.rope_theta).to(device)
        ws = 0
        for (M, N, K, mode, epi) in self._gemm_shapes(T) + self._gemm_shapes(max(max_seqs, 1)):
            ws = max(ws, L.gemm_workspace_size(M, N, K, tp, mode, epi, dt))
        ws = max(ws, L.attention_decode_workspace_size(max(max_seqs, 1), max_context, shape.n_heads, hd))
        if kv8 is not None:
            ws = max(ws, L.attention_decode_kv8_workspace_size(max(max_seqs, 1), max_context, shape.n_heads,
                                                               shape.n_kv_heads), L.ATTENTION_PREFILL_KV8_WORKSPACE_MAX)
        ws = max(ws, L.lm_head_workspace_size(max(max_seqs, 1), shape.vocab, H, tp, dt))
        if self.w4 or isinstance(params.embed, W4Weight):
            if dt != torch.bfloat16:
                raise ValueError("4-bit weights are for bf16 models")
            for (M, N, K, mode, epi) in self._gemm_shapes(T) + self._gemm_shapes(max(max_seqs, 1)):
                ws = max(ws, L.w4_gemm_workspace_size(M, N, K, tp, mode, epi))
            ws = max(ws, L.w4_lm_head_workspace_size(max(max_seqs, 1), shape.vocab, H, tp))
        # completion counters at its start must be zero before the first call
        self.workspace = torch.zeros(max(ws, 256), dtype=torch.uint8, device=device)
        self.scale = hd ** -0.5
        self.probe = None      # optional timing hook: probe(name, layer) -> context manager
        self.max_context = max_context
        self.max_seqs = max_seqs
        # decode batches of at most 16 tokens can run every layer in one
        # persistent kernel (qw_decode_layers); off by default: on GB300 it is
        # slower today than the per-operation kernels chained with programmatic
        # dependent launch (2.4 vs 1.4 ms per 28-layer step of 8 tokens)
        self.fused_decode = False
        # decode attention may stream cached history before the previous kernel ends
        # (valid while slot_mapping[b] == seq_base[b] + context_lens[b] - 1, which the
        # folded KV store requires anyway)
        self._history_ready = True
        self._fused = None     # (layer table, workspace), built on first use
        # prefill: QK-norm + RoPE + KV store in the QKV GEMM's epilogue (persistent
        # tensor-core kernel, the same results bit for bit); off by default: once
        # the plain QKV GEMM ran on 256-row tiles, it and the standalone kernel
        # took 19.4 ms per 8 x 2048-token prefill against 19.6 ms fused
        self.fused_qkv = False
        # prefill in five kernels per layer (QK-norm + RoPE + KV store in the QKV GEMM's
        # epilogue, residual add + RMSNorm in the o_proj and down GEMMs' epilogues);
        # off by default: on GB300 the longer epilogues, run after each tile's
        # mainloop with the tensor pipe idle, cost more than the kernels they
        # replace (8 x 2048-token prefill: 21.0 ms fused, 19.1 ms unfused)
        self.fused_prefill = False

    def _in_4_bits(self, *names) -> bool:
        """Some layer holds one of these weights in 4 bits; the others may be bf16."""
        return any(isinstance(getattr(p, n), W4Weight) for p in self.p.layers for n in names)

    @property
    def w4(self) -> bool:
        """Linear weights of the layers are in 4 bits, all or some."""
        return self._in_4_bits("qkv", "o", "gate_up", "down")

    def _linear(self, A, W, C, N, mode, epilogue, stream=None):
        """One linear layer, over bf16 / f32 or 4-bit weights."""
        if isinstance(W, W4Weight):
            L.w4_gemm(A, W.codes, W.scales, W.zeros, C, N, W.group, self.m.tp, mode, epilogue, self.workspace, stream,
                      weights_ready=True)   # loaded once, as every weight here
        else:
            L.gemm(A, W, C, N, self.m.tp, mode, epilogue, self.workspace, stream)

    def _embed(self, ids, out, stream=None):
        W = self.p.embed
        if isinstance(W, W4Weight):
            L.w4_embed_vocab(ids, W.codes, W.scales, W.zeros, W.group, self.m.tp, out, self.err, stream)
        else:
            L.embed_vocab(ids, W, self.m.tp, out, self.err, stream)

    def _around(self, name: str, layer: int):
        if self.probe is None:
            return contextlib.nullcontext()
        return self.probe(name, layer)

    def _gemm_shapes(self, M):
        m = self.m
        return [(M, self.qkv_width, m.hidden, L.QW_GEMM_COLUMN, L.QW_EPI_NONE),
                (M, m.hidden, m.n_heads * m.head_dim, L.QW_GEMM_ROW_REDUCE, L.QW_EPI_NONE),
                (M, 2 * m.intermediate, m.hidden, L.QW_GEMM_COLUMN, L.QW_EPI_SILU_MUL),
                (M, m.hidden, m.intermediate, L.QW_GEMM_ROW_REDUCE, L.QW_EPI_NONE)]

    def qkv_epilogue_ok(self) -> bool:
        """Prefill: QK-norm + RoPE + KV store as the QKV GEMM's epilogue (bf16,
        head_dim 128, two whole heads of one shard per 256-column tile)."""
        m = self.m
        return (self.fused_qkv and self.kv8 is None and self.dtype == torch.bfloat16 and m.head_dim == 128
                and ((m.n_heads + 2 * m.n_kv_heads) // m.tp) % 2 == 0 and m.hidden % 8 == 0
                and not self._in_4_bits("qkv"))

    def prefill_fusion_ok(self) -> bool:
        """Prefill through the fused epilogues: QK-norm + RoPE + KV store in the QKV
        GEMM (two whole heads of one shard per 256-column tile), residual add +
        RMSNorm in the o_proj and down GEMMs (a row's hidden columns in one
        cluster of 256-column tiles)."""
        m = self.m
        return (self.fused_prefill and self.kv8 is None and not self.w4 and self.dtype == torch.bfloat16 and m.head_dim == 128
                and ((m.n_heads + 2 * m.n_kv_heads) // m.tp) % 2 == 0 and m.hidden % 256 == 0
                and m.hidden <= 2048 and (m.n_heads * m.head_dim // m.tp) % 8 == 0
                and (m.intermediate // m.tp) % 8 == 0 and len(self.p.layers) > 0)

    def _prefill_layer(self, l: int, T: int, ctx, first: bool, next_gamma, stream=None):
        """One decoder layer of a prefill in five kernels ([SK] §1, §8).

        On entry y holds input_layernorm(residual) (for the first layer it is
        computed here from the embedding).  On exit the residual holds the
        stream after the layer and y = RMSNorm(residual) * next_gamma (the next
        layer's input_layernorm, or the final norm); with next_gamma None, h
        holds the MLP output and the residual the stream before it, as the
        unfused layer leaves them."""
        m, p = self.m, self.p.layers[l]
        tp = m.tp
        h, res, y = self.h[:T], self.res[:T], self.y[:T]
        q, attn, act = self.q[:T], self.attn[:T], self.act[:T]
        if first:
            with self._around("prefill.add_rmsnorm", l):
                L.add_rmsnorm(h, None, res, p.input_ln, m.eps, y, stream)
        with self._around("prefill.gemm_qkv_norm_rope_store_kv", l):
            L.qkv_gemm_norm_rope_store_kv(y, p.qkv, m.n_heads, m.n_kv_heads, m.head_dim, tp, ctx.positions,
                                          self.cos_sin, p.q_norm, p.k_norm, m.eps, ctx.slot_mapping, self.k_cache[l],
                                          self.v_cache[l], q, self.err, stream)
        with self._around("prefill.attention", l):
            L.attention_prefill(q, self.k_cache[l], self.v_cache[l], ctx.cu_seqlens, ctx.cu_seqlens, ctx.seq_base,
                                ctx.max_seqlen, m.n_heads, m.n_kv_heads, m.head_dim, self.scale, attn, stream)
        with self._around("prefill.gemm_o_add_rmsnorm", l):
            L.gemm_add_rmsnorm(attn, p.o, res, p.post_ln, m.eps, y, tp, stream)
        with self._around("prefill.gemm_gate_up_silu", l):
            L.gemm(y, p.gate_up, act, 2 * m.intermediate, tp, L.QW_GEMM_COLUMN, L.QW_EPI_SILU_MUL, self.workspace,
                   stream)
        if next_gamma is None:
            with self._around("prefill.gemm_down", l):
                L.gemm(act, p.down, h, m.hidden, tp, L.QW_GEMM_ROW_REDUCE, L.QW_EPI_NONE, self.workspace, stream)
        else:
            with self._around("prefill.gemm_down_add_rmsnorm", l):
                L.gemm_add_rmsnorm(act, p.down, res, next_gamma, m.eps, y, tp, stream)

    def norm_fusion_ok(self, T: int) -> bool:
        """Few bf16 tokens: each add+RMSNorm runs as the prologue of the GEMM it feeds, over bf16 weights in every layer."""
        return (self.dtype == torch.bfloat16 and T <= 16 and T <= self.res2.shape[0]
                and not self._in_4_bits("qkv", "gate_up"))

    def _res(self, c: int, T: int):
        """Residual after update c of a decode step (two per layer) when norms are fused."""
        return (self.res if c % 2 == 0 else self.res2)[:T]

    # -- one decoder layer ([SK] §1) ------------------------------------------
    def _layer(self, l: int, T: int, ctx, first: bool, decode: bool, fused: bool, stream=None):
        """fused: add+RMSNorm as the prologue of the GEMM that it feeds, in every layer or in none."""
        m, p = self.m, self.p.layers[l]
        tp = m.tp
        h, res, y = self.h[:T], self.res[:T], self.y[:T]
        ph = "decode" if decode else "prefill"
        qkv = self.qkv[:T]
        if fused:
            # residual update 2l here, 2l+1 before gate_up; the buffers alternate
            with self._around(f"{ph}.add_rmsnorm_gemm_qkv", l):
                L.add_rmsnorm_gemm(h, None if first else self._res(2 * l - 1, T), self._res(2 * l, T), p.input_ln,
                                   m.eps, p.qkv, qkv, self.qkv_width, tp, L.QW_EPI_NONE, stream)
        else:
            with self._around(f"{ph}.add_rmsnorm", l):
                L.add_rmsnorm(h, None if first else res, res, p.input_ln, m.eps, y, stream)
            if not decode and self.qkv_epilogue_ok():
                # QK-norm + RoPE + KV store as the QKV GEMM's epilogue: no QKV round trip
                with self._around(f"{ph}.gemm_qkv_norm_rope_store_kv", l):
                    L.qkv_gemm_norm_rope_store_kv(y, p.qkv, m.n_heads, m.n_kv_heads, m.head_dim, tp, ctx.positions,
                                                  self.cos_sin, p.q_norm, p.k_norm, m.eps, ctx.slot_mapping,
                                                  self.k_cache[l], self.v_cache[l], self.q[:T], self.err, stream)
            else:
                with self._around(f"{ph}.gemm_qkv", l):
                    self._linear(y, p.qkv, qkv, self.qkv_width, L.QW_GEMM_COLUMN, L.QW_EPI_NONE, stream)
        q = self.q[:T]
        attn = self.attn[:T]
        if not decode and self.qkv_epilogue_ok():
            with self._around(f"{ph}.attention", l):
                L.attention_prefill(q, self.k_cache[l], self.v_cache[l], ctx.cu_seqlens, ctx.cu_seqlens, ctx.seq_base,
                                    ctx.max_seqlen, m.n_heads, m.n_kv_heads, m.head_dim, self.scale, attn, stream)
        elif self.kv8 is not None:
            self._attention_kv8(l, qkv, q, attn, ctx, decode, ph, stream)
        elif decode and self.dtype == torch.bfloat16 and m.head_dim == 128:
            # QK-norm + RoPE + KV store folded into decode attention.  Sequence b's
            # cache is contiguous from seq_base[b] and this step's k/v go to its last
            # row, so the kernel before (the QKV GEMV) writes none of the cached
            # history: the history can stream in before that kernel finishes.
            with self._around(f"{ph}.attention", l):
                L.attention_decode_rope(qkv, m.n_heads, m.n_kv_heads, m.head_dim, tp, ctx.positions, self.cos_sin,
                                        p.q_norm, p.k_norm, m.eps, ctx.slot_mapping, self.k_cache[l],
                                        self.v_cache[l], self.err, ctx.context_lens, ctx.seq_base, ctx.max_context,
                                        self.scale, attn, self.workspace, stream,
                                        history_ready=self._history_ready)
        else:
            with self._around(f"{ph}.qkv_norm_rope_store_kv", l):
                L.qkv_norm_rope_store_kv(qkv, m.n_heads, m.n_kv_heads, m.head_dim, tp, ctx.positions, self.cos_sin,
                                         p.q_norm, p.k_norm, m.eps, ctx.slot_mapping, self.k_cache[l],
                                         self.v_cache[l], q, self.err, stream)
            with self._around(f"{ph}.attention", l):
                if decode:
                    L.attention_decode(q, self.k_cache[l], self.v_cache[l], ctx.context_lens, ctx.seq_base,
                                       ctx.max_context, m.n_heads, m.n_kv_heads, m.head_dim, self.scale, attn,
                                       self.workspace, stream)
                else:
                    L.attention_prefill(q, self.k_cache[l], self.v_cache[l], ctx.cu_seqlens, ctx.cu_seqlens,
                                        ctx.seq_base, ctx.max_seqlen, m.n_heads, m.n_kv_heads, m.head_dim,
                                        self.scale, attn, stream)
        with self._around(f"{ph}.gemm_o", l):
            self._linear(attn, p.o, h, m.hidden, L.QW_GEMM_ROW_REDUCE, L.QW_EPI_NONE, stream)
        act = self.act[:T]
        if fused:
            # residual update 2l + 1 as the prologue of gate_up + SiluAndMul
            with self._around(f"{ph}.add_rmsnorm_gemm_gate_up", l):
                L.add_rmsnorm_gemm(h, self._res(2 * l, T), self._res(2 * l + 1, T), p.post_ln, m.eps, p.gate_up, act,
                                   2 * m.intermediate, tp, L.QW_EPI_SILU_MUL, stream)
        else:
            with self._around(f"{ph}.add_rmsnorm", l):
                L.add_rmsnorm(h, res, res, p.post_ln, m.eps, y, stream)
            with self._around(f"{ph}.gemm_gate_up_silu", l):
                self._linear(y, p.gate_up, act, 2 * m.intermediate, L.QW_GEMM_COLUMN, L.QW_EPI_SILU_MUL, stream)
        with self._around(f"{ph}.gemm_down", l):
            self._linear(act, p.down, h, m.hidden, L.QW_GEMM_ROW_REDUCE, L.QW_EPI_NONE, stream)

    def _check_kv8(self, ctx, decode: bool):
        """Refuses a context without the fields that the 8-bit paged cache is addressed by."""
        if ctx.block_table is None or ctx.context_lens is None:
            raise ValueError("the 8-bit KV cache needs a context with block_table and context_lens")
        if not decode and ctx.n_tokens > 0 and ctx.max_context <= 0:   # no key would be read
            raise ValueError(f"the 8-bit KV cache needs a context with max_context >= every context_lens, not {ctx.max_context}")

    def _attention_kv8(self, l: int, qkv, q, attn, ctx, decode: bool, ph: str, stream=None):
        """QK-norm + RoPE + quantised append, then attention over the 8-bit paged cache."""
        m, p, c = self.m, self.p.layers[l], self.kv8
        cache = (self.k_cache[l], self.v_cache[l], self.k_scale[l], self.v_scale[l], c.scale_block)
        cu = None if decode else ctx.cu_seqlens
        with self._around(f"{ph}.kv8_append", l):
            L.kv8_append(qkv, m.n_heads, m.n_kv_heads, m.head_dim, m.tp, ctx.positions, self.cos_sin, p.q_norm, p.k_norm,
                         m.eps, cu, ctx.context_lens, ctx.block_table, c.block_size, *cache, q, self.err, stream)
        with self._around(f"{ph}.attention", l):
            if decode:
                L.attention_decode_kv8(q, *cache, ctx.context_lens, ctx.block_table, c.block_size, ctx.max_context,
                                       m.n_heads, m.n_kv_heads, m.head_dim, self.scale, attn, self.workspace, c.window,
                                       c.n_sink, stream)
            else:
                L.attention_prefill_kv8(q, *cache, cu, ctx.context_lens, ctx.block_table, c.block_size, ctx.max_seqlen,
                                        ctx.max_context, m.n_heads, m.n_kv_heads, m.head_dim, self.scale, attn,
                                        self.workspace, c.window, c.n_sink, stream)

    def fused_decode_ok(self, B: int) -> bool:
        m = self.m
        if not self.fused_decode or self.kv8 is not None or self.w4 or self.dtype != torch.bfloat16 or len(self.p.layers) == 0 or B > self.max_seqs:
            return False
        return L.decode_layers_workspace_size(len(self.p.layers), B, m.hidden, m.n_heads, m.n_kv_heads, m.head_dim,
                                              m.intermediate, m.tp, self.max_context) > 0

    def _fused_state(self):
        if self._fused is None:
            m = self.m
            rows = [dict(input_layernorm=p.input_ln, qkv=p.qkv, q_norm=p.q_norm, k_norm=p.k_norm, o_proj=p.o,
                         post_attention_layernorm=p.post_ln, gate_up=p.gate_up, down=p.down,
                         k_cache=self.k_cache[l], v_cache=self.v_cache[l]) for l, p in enumerate(self.p.layers)]
            table = L.decode_layer_table(rows)
            ws = max(L.decode_layers_workspace_size(len(rows), b, m.hidden, m.n_heads, m.n_kv_heads, m.head_dim,
                                                    m.intermediate, m.tp, self.max_context)
                     for b in range(1, min(self.max_seqs, 16) + 1))
            # its counters must be zero before the first call; every call leaves them so
            self._fused = (table, torch.zeros(ws, dtype=torch.uint8, device=self.device))
        return self._fused

    def _decode_fused(self, ctx, stream=None):
        """embedding -> all layers + final add+RMSNorm in one persistent kernel (qw_decode_layers)."""
        m = self.m
        B = ctx.n_tokens
        table, ws = self._fused_state()
        with self._around("decode.embed_vocab", -1):
            self._embed(ctx.ids, self.h[:B], stream)
        with self._around("decode.layers", -1):
            L.decode_layers(table, len(self.p.layers), self.h[:B], ctx.positions, ctx.slot_mapping, ctx.context_lens,
                            ctx.seq_base, ctx.max_context, m.n_heads, m.n_kv_heads, m.head_dim, m.intermediate, m.tp,
                            self.cos_sin, self.k_cache[0].shape[0], m.eps, self.scale, self.p.final_norm, self.y[:B],
                            ws, self.err, stream)
        return self.y[:B]

    def run_layers(self, ctx, decode: bool, hidden_in: Optional[torch.Tensor] = None, final_norm: bool = True,
                   stream=None):
        """embedding (or hidden_in) -> layers -> optional final add+RMSNorm; returns the hidden buffer view."""
        m = self.m
        T = ctx.n_tokens
        if self.kv8 is not None:
            self._check_kv8(ctx, decode)
        if decode and hidden_in is None and final_norm and self.fused_decode_ok(T):
            return self._decode_fused(ctx, stream)
        if hidden_in is None:
            with self._around(f"{'decode' if decode else 'prefill'}.embed_vocab", -1):
                self._embed(ctx.ids, self.h[:T], stream)
        else:
            self.h[:T].copy_(hidden_in)
        nl = len(self.p.layers)
        if not decode and self.prefill_fusion_ok():
            for l in range(nl):
                nxt = self.p.layers[l + 1].input_ln if l + 1 < nl else (self.p.final_norm if final_norm else None)
                self._prefill_layer(l, T, ctx, l == 0, nxt, stream)
            if final_norm:
                return self.y[:T]   # the last down GEMM applied the final norm
            return self.h[:T], self.res[:T]
        fused = decode and self.norm_fusion_ok(T)
        for l in range(nl):
            self._layer(l, T, ctx, l == 0, decode, fused, stream)
        res = self._res(2 * nl - 1, T) if fused and nl > 0 else self.res[:T]
        if not final_norm:
            return self.h[:T], res
        with self._around("final_norm", -1):
            L.add_rmsnorm(self.h[:T], None if nl == 0 else res, None, self.p.final_norm, m.eps, self.y[:T], stream)
        return self.y[:T]

    def compute_logits(self, hidden: torch.Tensor, last_idx: Optional[torch.Tensor], n_out: int, stream=None):
        """ParallelLMHead ([SK] §6): last token of each sequence in prefill, then greedy argmax."""
        logits = self.logits[:n_out]
        nt = self.next_tokens[:n_out]
        with self._around("lm_head", -1):
            W = self.p.embed
            if isinstance(W, W4Weight):
                L.w4_lm_head(hidden, last_idx, n_out, W.codes, W.scales, W.zeros, W.group, self.m.tp, logits, nt,
                             self.workspace, stream, weights_ready=True)
            else:
                L.lm_head(hidden, last_idx, n_out, W, self.m.tp, logits, nt, self.workspace, stream)
        return logits, nt

    def prefill(self, ctx: PrefillContext, stream=None):
        hidden = self.run_layers(ctx, decode=False, stream=stream)
        return self.compute_logits(hidden, ctx.last_idx, ctx.last_idx.shape[0], stream)

    def decode(self, ctx: DecodeContext, stream=None):
        hidden = self.run_layers(ctx, decode=True, stream=stream)
        return self.compute_logits(hidden, None, ctx.n_tokens, stream)
