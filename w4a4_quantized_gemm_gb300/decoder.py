"""A decoder layer served one token per sequence: the quantised linears with the paged cache, its
attention and the fused block norms between them ("W4A4 CUDA Kernel for Voice Clone", 3.4 and 4: the
kernels of a layer, captured in one CUDA graph).

    r, x -> qkv linear -> w4a4_kv_append (per-head q/k norm, rotation, cache) -> w4a4_paged_attention
         -> o linear -> w4a4_block_norm (residual add, norm before the MLP)
         -> gate|up linear with SiLU(gate) * up -> down linear
         -> w4a4_block_norm (residual add, norm before the next layer)

The module only allocates device buffers and issues the C-ABI calls.

    python -m w4a4_quantized_gemm_gb300.decoder [sequences] [tokens in the cache] [layers]

builds a stack of 1024-wide layers (16 query and 8 key-value heads of 128) with random weights and
prints the time of a decode step, captured as one CUDA graph.
"""
from __future__ import annotations

import sys

import torch

import w4a4_quantized_gemm_gb300 as w4


class _Packed:
    """Packed weights of one linear (fp32 W [N, K], LoRA factors, affine)."""

    def __init__(self, W, L_down, L_up, colscale, bias, gate_up=False):
        self.N, self.K = W.shape
        self.r = 0 if L_down is None else L_down.shape[1]
        self.packed = torch.empty(w4.packed_weights_bytes(self.N, self.K, self.r), dtype=torch.uint8, device=W.device)
        pack = w4.w4a4_pack_weights_gate_up if gate_up else w4.w4a4_pack_weights
        pack(W.contiguous(), L_down, L_up, self.packed, self.r)
        self.colscale, self.bias = colscale.contiguous(), None if bias is None else bias.contiguous()


class W4A4DecoderLayer:
    """One layer's weights and the buffers of a decode step of `seqs` sequences.

    Each of qkv, o, gate_up, down is (W fp32 [out, in], L_down, L_up, colscale, bias) as W4A4Linear
    takes them; gate_up has the gate rows first.  q_gain, k_gain: the per-head norms' gains [head_dim]
    (None: no such norm); mlp_gain [hidden]: the norm between attention and MLP.  The norm before
    attention belongs to the layer before (its gain is step's next_gain), so that it is fused with
    that layer's residual addition.
    """

    def __init__(self, qkv, o, gate_up, down, q_heads: int, kv_heads: int, head_dim: int, seqs: int, mlp_gain,
                 q_gain=None, k_gain=None, eps: float = 1e-6):
        self.qkv, self.o, self.down = _Packed(*qkv), _Packed(*o), _Packed(*down)
        self.gate_up = _Packed(*gate_up, gate_up=True)
        self.q_heads, self.kv_heads, self.dim, self.seqs, self.eps = q_heads, kv_heads, head_dim, seqs, eps
        self.mlp_gain, self.q_gain, self.k_gain = mlp_gain, q_gain, k_gain
        dev = self.qkv.packed.device

        def buf(*shape):
            return torch.empty(shape, dtype=torch.float16, device=dev)

        hidden = self.o.N
        self.qkv_out, self.q, self.attn = buf(seqs, self.qkv.N), buf(seqs, q_heads, head_dim), buf(seqs, q_heads, head_dim)
        self.o_out, self.x_mlp, self.down_out = buf(seqs, hidden), buf(seqs, hidden), buf(seqs, hidden)
        self.h = buf(seqs, self.gate_up.N // 2)
        need = max(w4.act_workspace_bytes(seqs, p.K, p.r) for p in (self.qkv, self.o, self.gate_up, self.down))
        self.ws = torch.empty(need, dtype=torch.uint8, device=dev)
        qkv_rows = self.qkv_out.unflatten(1, (q_heads + 2 * kv_heads, head_dim))
        self.split = qkv_rows.split((q_heads, kv_heads, kv_heads), dim=1)

    def _linear(self, p, X, Y, stream):
        w4.w4a4_forward(X, p.packed, p.colscale, p.bias, Y, p.r, self.ws, stream=stream)

    def step(self, x, r, positions, lengths, cache, rope, next_gain, x_next, stream=None):
        """One token of each sequence: x [seqs, hidden] its normalised input, r the residual stream
        (fp16 or fp32, updated in place), positions = lengths - 1 the token's place, lengths the
        cache's with it.  x_next receives the next layer's input under next_gain."""
        q, k, v = self.split
        self._linear(self.qkv, x, self.qkv_out, stream)
        w4.w4a4_kv_append(q, k, v, positions, cache, self.q, rope=rope, q_gain=self.q_gain, k_gain=self.k_gain,
                          eps=self.eps, stream=stream)
        w4.w4a4_paged_attention(self.q, cache, lengths, self.attn, stream=stream)
        self._linear(self.o, self.attn.view(self.seqs, -1), self.o_out, stream)
        w4.w4a4_block_norm(self.o_out, r, self.x_mlp, r, post=w4.NORM_NONE, pre_gain=self.mlp_gain, eps=self.eps,
                           stream=stream)
        g = self.gate_up
        w4.w4a4_quantize_act(self.x_mlp, g.packed, self.ws, g.r, stream)
        w4.w4a4_linear_silu_mul(self.ws, g.packed, g.colscale, g.bias, self.h, g.K, g.r, stream)
        self._linear(self.down, self.h, self.down_out, stream)
        w4.w4a4_block_norm(self.down_out, r, x_next, r, post=w4.NORM_NONE, pre_gain=next_gain, eps=self.eps,
                           stream=stream)


def random_layer(hidden: int, inner: int, q_heads: int, kv_heads: int, dim: int, seqs: int, rank: int = 32,
                 seed: int = 0):
    """A layer with N(0, 0.02) weights (LoRA factors included) and unit gains with some spread."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape, std=0.02, dtype=torch.float16):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    def linear(out, k):
        return n(out, k, dtype=torch.float32), n(k, rank), n(rank, out), 1 + n(out, std=0.1), n(out)

    return W4A4DecoderLayer(linear((q_heads + 2 * kv_heads) * dim, hidden), linear(hidden, q_heads * dim),
                            linear(2 * inner, hidden), linear(hidden, inner), q_heads, kv_heads, dim, seqs,
                            1 + n(hidden, std=0.1), 1 + n(dim, std=0.1), 1 + n(dim, std=0.1))


def paged_cache(seqs: int, tokens: int, kv_heads: int, dim: int, page_size: int = 16, dtype=torch.float16):
    """Zeroed pools and a page table with room for `tokens` tokens of every sequence."""
    per = -(-tokens // page_size)
    pools = [torch.zeros((seqs * per, page_size, kv_heads, dim), dtype=torch.float16, device="cuda").to(dtype)
             for _ in range(2)]
    table = torch.randperm(seqs * per, device="cuda").to(torch.int32).view(seqs, per)
    return w4.PagedKVCache(*pools, table)


def check_status(where: str):
    """Raises what a kernel has left in the device status; reading it clears it."""
    status = w4.w4a4_device_status()
    if status != w4.W4A4_OK:
        raise w4.W4A4Error(status, where)


def main(seqs: int = 32, tokens: int = 2048, layers: int = 28):
    hidden, inner, q_heads, kv_heads, dim = 1024, 3072, 16, 8, 128
    stack = [random_layer(hidden, inner, q_heads, kv_heads, dim, seqs, seed=i) for i in range(layers)]
    caches = [paged_cache(seqs, tokens, kv_heads, dim) for _ in range(layers)]
    rope = w4.w4a4_rope_table(tokens, dim, 1e6)
    lengths = torch.full((seqs,), tokens, dtype=torch.int32, device="cuda")
    positions = lengths - 1
    gain = torch.ones(hidden, dtype=torch.float16, device="cuda")
    r = torch.randn(seqs, hidden, device="cuda")
    x = [torch.empty(seqs, hidden, dtype=torch.float16, device="cuda") for _ in range(2)]

    def forward():
        w4.w4a4_block_norm(torch.zeros_like(x[0]), r, x[0], r, post=w4.NORM_NONE, pre_gain=gain)
        for i, (layer, cache) in enumerate(zip(stack, caches)):
            layer.step(x[i % 2], r, positions, lengths, cache, rope, gain, x[(i + 1) % 2])

    forward()  # warm-up: workspaces exist before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forward()
    for _ in range(3):
        graph.replay()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    check_status("decoder step")
    ms = start.elapsed_time(end) / 20
    print(f"{layers} layers, {seqs} sequences of {tokens} tokens: {ms * 1e3:.0f} us a step, {seqs / ms * 1e3:.0f} tokens/s")


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:4]))
