"""A decoder layer served one token per sequence, a chunk of new tokens of every sequence, or whole
prompts at once: the quantised linears with the paged cache, its attention and the fused block norms
between them ("W4A4 CUDA Kernel for Voice Clone", 3.4 and 4: the
kernels of a layer, captured in one CUDA graph).

    r, x -> qkv linear -> w4a4_kv_append (per-head q/k norm, rotation, cache) -> w4a4_paged_attention
         -> o linear -> w4a4_block_norm (residual add, norm before the MLP)
         -> gate|up linear with SiLU(gate) * up -> down linear
         -> w4a4_block_norm (residual add, norm before the next layer)

A chunk's attention is w4a4_chunk_attention (`W4A4DecoderLayer.chunk`); prompts that are attended to
once and need no cache take w4a4_qk_rope and w4a4_prompt_attention (`W4A4DecoderLayer.prompt`).

The module only allocates device buffers and issues the C-ABI calls.

    python -m w4a4_quantized_gemm_gb300.decoder [sequences] [tokens in the cache] [layers]

builds a stack of 1024-wide layers (16 query and 8 key-value heads of 128) with random weights and
prints the time of a prompt of so many tokens and of a decode step, captured as one CUDA graph.
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


class _Rows:
    """The buffers of a layer's pass over so many rows (tokens).  They belong to the stream that they are made for; the
    allocator learns of others that torch owns."""

    def __init__(self, layer, rows: int):
        dev, hq, hkv, dim = layer.qkv.packed.device, layer.q_heads, layer.kv_heads, layer.dim

        def buf(*shape):
            return torch.empty(shape, dtype=torch.float16, device=dev)

        hidden = layer.o.N
        self.qkv_out, self.q, self.attn = buf(rows, layer.qkv.N), buf(rows, hq, dim), buf(rows, hq, dim)
        self.o_out, self.x_mlp, self.down_out = buf(rows, hidden), buf(rows, hidden), buf(rows, hidden)
        self.h = buf(rows, layer.gate_up.N // 2)
        need = max(w4.act_workspace_bytes(rows, p.K, p.r) for p in (layer.qkv, layer.o, layer.gate_up, layer.down))
        self.ws = torch.empty(need, dtype=torch.uint8, device=dev)
        self.split = self.qkv_out.unflatten(1, (hq + 2 * hkv, dim)).split((hq, hkv, hkv), dim=1)
        self._streams = set()

    def used_on(self, stream):
        """Keeps the memory from being handed out again, once these are dropped, before `stream` is done with them."""
        if stream is None:
            stream = torch.cuda.current_stream(self.ws.device)
        handle, number = (getattr(stream, name, None) for name in ("cuda_stream", "stream_id"))
        if handle is None or handle in self._streams or (handle != 0 and number == handle):
            return  # a handle or an external stream, which may be gone by then, or one that is known
        self._streams.add(handle)
        for t in (self.qkv_out, self.q, self.attn, self.o_out, self.x_mlp, self.down_out, self.h, self.ws):
            t.record_stream(stream)


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
        self._rows = {}
        one = self.rows(seqs)
        self.qkv_out, self.q, self.attn, self.split = one.qkv_out, one.q, one.attn, one.split
        self.o_out, self.x_mlp, self.down_out, self.h, self.ws = one.o_out, one.x_mlp, one.down_out, one.h, one.ws

    def rows(self, n: int, stream=None) -> _Rows:
        """The buffers for n rows, made at their first use on `stream` (before a graph capture, if it is to use them)
        and kept as long as the layer: a captured graph may hold them.  Passes over as many rows use the same ones:
        those on different streams have to be ordered."""
        if n not in self._rows:
            with w4.on_stream(stream):
                self._rows[n] = _Rows(self, n)
        self._rows[n].used_on(stream)
        return self._rows[n]

    def _linear(self, p, X, Y, ws, stream):
        w4.w4a4_forward(X, p.packed, p.colscale, p.bias, Y, p.r, ws, stream=stream)

    def _after_attention(self, b, r, next_gain, x_next, stream):
        self._linear(self.o, b.attn.flatten(1), b.o_out, b.ws, stream)
        w4.w4a4_block_norm(b.o_out, r, b.x_mlp, r, post=w4.NORM_NONE, pre_gain=self.mlp_gain, eps=self.eps,
                           stream=stream)
        g = self.gate_up
        w4.w4a4_quantize_act(b.x_mlp, g.packed, b.ws, g.r, stream)
        w4.w4a4_linear_silu_mul(b.ws, g.packed, g.colscale, g.bias, b.h, g.K, g.r, stream)
        self._linear(self.down, b.h, b.down_out, b.ws, stream)
        w4.w4a4_block_norm(b.down_out, r, x_next, r, post=w4.NORM_NONE, pre_gain=next_gain, eps=self.eps,
                           stream=stream)

    def step(self, x, r, positions, lengths, cache, rope, next_gain, x_next, stream=None):
        """One token of each sequence: x [seqs, hidden] its normalised input, r the residual stream
        (fp16 or fp32, updated in place), positions = lengths - 1 the token's place, lengths the
        cache's with it.  x_next receives the next layer's input under next_gain."""
        b = self.rows(self.seqs, stream)
        q, k, v = b.split
        self._linear(self.qkv, x, b.qkv_out, b.ws, stream)
        w4.w4a4_kv_append(q, k, v, positions, cache, b.q, rope=rope, q_gain=self.q_gain, k_gain=self.k_gain,
                          eps=self.eps, stream=stream)
        w4.w4a4_paged_attention(b.q, cache, lengths, b.attn, stream=stream)
        self._after_attention(b, r, next_gain, x_next, stream)

    def chunk(self, x, r, positions, owners, starts, lengths, cache, rope, next_gain, x_next, stream=None):
        """A chunk of new tokens of every sequence, rows starts[b] .. starts[b + 1] - 1 of x [tokens, hidden]
        and r; row t is token positions[t] of sequence owners[t].  They go into the cache, which holds
        lengths[b] tokens of each with them, and are attended to over all of it.  The rest as for step."""
        b = self.rows(x.shape[0], stream)
        q, k, v = b.split
        self._linear(self.qkv, x, b.qkv_out, b.ws, stream)
        w4.w4a4_kv_append(q, k, v, positions, cache, b.q, seqs=owners, rope=rope, q_gain=self.q_gain,
                          k_gain=self.k_gain, eps=self.eps, stream=stream)
        w4.w4a4_chunk_attention(b.q, cache, starts, lengths, b.attn, stream=stream)
        self._after_attention(b, r, next_gain, x_next, stream)

    def prompt(self, x, r, positions, starts, rope, next_gain, x_next, causal=True, stream=None):
        """Whole prompts, packed one behind the other (rows starts[b] .. starts[b + 1] - 1), without a cache.
        Rows of x outside all of them are padding: positions[t] < 0, and their results are not defined."""
        b = self.rows(x.shape[0], stream)
        q, k, v = b.split
        self._linear(self.qkv, x, b.qkv_out, b.ws, stream)
        w4.w4a4_qk_rope(q, k, positions, q, k, rope=rope, q_gain=self.q_gain, k_gain=self.k_gain, eps=self.eps,
                        stream=stream)
        w4.w4a4_prompt_attention(q, k, v, starts, b.attn, causal=causal, stream=stream)
        self._after_attention(b, r, next_gain, x_next, stream)


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

    # the first sequence's prompt, into the caches, with no rows of the others
    starts = torch.full((seqs + 1,), tokens, dtype=torch.int32, device="cuda")
    starts[0] = 0
    owners = torch.zeros(tokens, dtype=torch.int32, device="cuda")
    places = torch.arange(tokens, dtype=torch.int32, device="cuda")
    stream = torch.randn(tokens, hidden, device="cuda")
    rows = [torch.randn(tokens, hidden, device="cuda").half() for _ in range(2)]

    def prefill():
        for i, (layer, cache) in enumerate(zip(stack, caches)):
            layer.chunk(rows[i % 2], stream, places, owners, starts, lengths, cache, rope, gain, rows[(i + 1) % 2])

    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for _ in range(2):  # the first pass makes buffers and workspaces
        start.record()
        prefill()
        end.record()
    torch.cuda.synchronize()
    check_status("prompt")
    ms = start.elapsed_time(end)
    print(f"{layers} layers, a prompt of {tokens} tokens: {ms:.2f} ms, {tokens / ms * 1e3:.0f} tokens/s")

    forward()  # warm-up: workspaces exist before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forward()
    for _ in range(3):
        graph.replay()
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
