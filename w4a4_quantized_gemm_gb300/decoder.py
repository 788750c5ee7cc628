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
    """The first n rows of a set of buffers: what a layer's pass over n rows (tokens) writes."""

    def __init__(self, layer, whole, n: int):
        for name in _ROWS:
            setattr(self, name, getattr(whole, name)[:n])
        self.ws = whole.ws[:_workspace_bytes(layer, n)]
        heads = layer.q_heads, layer.kv_heads, layer.kv_heads
        self.split = self.qkv_out.unflatten(1, (sum(heads), layer.dim)).split(heads, dim=1)


_ROWS = ("qkv_out", "q", "attn", "o_out", "x_mlp", "down_out", "h")


def _workspace_bytes(layer, rows: int) -> int:
    return max(w4.act_workspace_bytes(rows, p.K, p.r) for p in (layer.qkv, layer.o, layer.gate_up, layer.down))


class _Set:
    """Buffers for up to `rows` rows.  They belong to the stream that they are made for; the allocator learns of others
    that torch owns."""

    def __init__(self, layer, rows: int):
        dev, heads, hidden = layer.qkv.packed.device, (layer.q_heads, layer.dim), layer.o.N
        shapes = (layer.qkv.N,), heads, heads, (hidden,), (hidden,), (hidden,), (layer.gate_up.N // 2,)
        for name, shape in zip(_ROWS, shapes):
            setattr(self, name, torch.empty((rows, *shape), dtype=torch.float16, device=dev))
        self.ws = torch.empty(_workspace_bytes(layer, rows), dtype=torch.uint8, device=dev)
        self.rows, self._views, self._streams = rows, {}, set()

    def first(self, layer, n: int) -> _Rows:
        views = self._views
        if n not in views:
            if len(views) >= 64:  # views are small, but lengths are many
                views.clear()
            views[n] = _Rows(layer, self, n)
        return views[n]

    def used_on(self, stream):
        """Keeps the memory from being handed out again, once these are dropped, before `stream` is done with them."""
        if not self.ws.is_cuda:
            return
        if stream is None:
            stream = torch.cuda.current_stream(self.ws.device)
        handle, number = (getattr(stream, name, None) for name in ("cuda_stream", "stream_id"))
        if handle is None or handle in self._streams or (handle != 0 and number == handle):
            return  # a handle or an external stream, which may be gone by then, or one that is known
        self._streams.add(handle)
        for name in (*_ROWS, "ws"):
            getattr(self, name).record_stream(stream)


class Buffers:
    """Room for passes over any number of rows.  A pass takes the first rows of the largest set of buffers so far; where
    they do not suffice there is a new set, at least twice as large, and the others stay, since a captured graph may hold
    them: room for at most four times the rows of the largest pass, and a workspace a set.  Layers of the same
    shapes may share one, as a stack's do, whose passes follow one another.  Passes that may overlap on the GPU need
    one each."""

    def __init__(self):
        self._sets = {}

    def rows(self, layer, n: int, stream=None) -> _Rows:
        """The buffers that a pass of `layer` over n rows uses, made on `stream` if need be (before a graph capture, if it
        is to use them)."""
        sets = self._sets.setdefault(layer.shape, [])
        if not sets or sets[-1].rows < n:
            with w4.on_stream(stream):
                sets.append(_Set(layer, max(n, 2 * sets[-1].rows if sets else 0)))
        sets[-1].used_on(stream)
        return sets[-1].first(layer, n)


class W4A4DecoderLayer:
    """One layer's weights and the buffers of a decode step of `seqs` sequences.

    Each of qkv, o, gate_up, down is (W fp32 [out, in], L_down, L_up, colscale, bias) as W4A4Linear
    takes them; gate_up has the gate rows first.  q_gain, k_gain: the per-head norms' gains [head_dim]
    (None: no such norm); mlp_gain [hidden]: the norm between attention and MLP.  The norm before
    attention belongs to the layer before (its gain is step's next_gain), so that it is fused with
    that layer's residual addition.  buffers: what chunk and prompt write on their way (a Buffers of its
    own by default).
    """

    def __init__(self, qkv, o, gate_up, down, q_heads: int, kv_heads: int, head_dim: int, seqs: int, mlp_gain,
                 q_gain=None, k_gain=None, eps: float = 1e-6, buffers=None):
        self.qkv, self.o, self.down = _Packed(*qkv), _Packed(*o), _Packed(*down)
        self.gate_up = _Packed(*gate_up, gate_up=True)
        self.q_heads, self.kv_heads, self.dim, self.seqs, self.eps = q_heads, kv_heads, head_dim, seqs, eps
        self.mlp_gain, self.q_gain, self.k_gain = mlp_gain, q_gain, k_gain
        packed = self.qkv, self.o, self.gate_up, self.down
        self.shape = (*((p.N, p.K, p.r) for p in packed), q_heads, kv_heads, head_dim, self.qkv.packed.device)
        self.buffers = Buffers() if buffers is None else buffers
        self._step = _Set(self, seqs)
        one = self._step.first(self, seqs)
        self.qkv_out, self.q, self.attn, self.split = one.qkv_out, one.q, one.attn, one.split
        self.o_out, self.x_mlp, self.down_out, self.h, self.ws = one.o_out, one.x_mlp, one.down_out, one.h, one.ws

    def rows(self, n: int, stream=None, buffers=None) -> _Rows:
        """The buffers that chunk and prompt use for n rows."""
        return (self.buffers if buffers is None else buffers).rows(self, n, stream)

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
        self._step.used_on(stream)
        b = self._step.first(self, self.seqs)
        q, k, v = b.split
        self._linear(self.qkv, x, b.qkv_out, b.ws, stream)
        w4.w4a4_kv_append(q, k, v, positions, cache, b.q, rope=rope, q_gain=self.q_gain, k_gain=self.k_gain,
                          eps=self.eps, stream=stream)
        w4.w4a4_paged_attention(b.q, cache, lengths, b.attn, stream=stream)
        self._after_attention(b, r, next_gain, x_next, stream)

    def chunk(self, x, r, positions, owners, starts, lengths, cache, rope, next_gain, x_next, stream=None,
              buffers=None):
        """A chunk of new tokens of every sequence, rows starts[b] .. starts[b + 1] - 1 of x [tokens, hidden]
        and r; row t is token positions[t] of sequence owners[t].  They go into the cache, which holds
        lengths[b] tokens of each with them, and are attended to over all of it.  buffers: instead of the
        layer's.  The rest as for step."""
        b = self.rows(x.shape[0], stream, buffers)
        q, k, v = b.split
        self._linear(self.qkv, x, b.qkv_out, b.ws, stream)
        w4.w4a4_kv_append(q, k, v, positions, cache, b.q, seqs=owners, rope=rope, q_gain=self.q_gain,
                          k_gain=self.k_gain, eps=self.eps, stream=stream)
        w4.w4a4_chunk_attention(b.q, cache, starts, lengths, b.attn, stream=stream)
        self._after_attention(b, r, next_gain, x_next, stream)

    def prompt(self, x, r, positions, starts, rope, next_gain, x_next, causal=True, stream=None,
               buffers=None):
        """Whole prompts, packed one behind the other (rows starts[b] .. starts[b + 1] - 1), without a cache.
        Rows of x outside all of them are padding: positions[t] < 0, and their results are not defined."""
        b = self.rows(x.shape[0], stream, buffers)
        q, k, v = b.split
        self._linear(self.qkv, x, b.qkv_out, b.ws, stream)
        w4.w4a4_qk_rope(q, k, positions, q, k, rope=rope, q_gain=self.q_gain, k_gain=self.k_gain, eps=self.eps,
                        stream=stream)
        w4.w4a4_prompt_attention(q, k, v, starts, b.attn, causal=causal, stream=stream)
        self._after_attention(b, r, next_gain, x_next, stream)


def random_layer(hidden: int, inner: int, q_heads: int, kv_heads: int, dim: int, seqs: int, rank: int = 32,
                 seed: int = 0, buffers=None):
    """A layer with N(0, 0.02) weights (LoRA factors included) and unit gains with some spread."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape, std=0.02, dtype=torch.float16):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    def linear(out, k):
        return n(out, k, dtype=torch.float32), n(k, rank), n(rank, out), 1 + n(out, std=0.1), n(out)

    return W4A4DecoderLayer(linear((q_heads + 2 * kv_heads) * dim, hidden), linear(hidden, q_heads * dim),
                            linear(2 * inner, hidden), linear(hidden, inner), q_heads, kv_heads, dim, seqs,
                            1 + n(hidden, std=0.1), 1 + n(dim, std=0.1), 1 + n(dim, std=0.1), buffers=buffers)


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
    buffers = Buffers()
    stack = [random_layer(hidden, inner, q_heads, kv_heads, dim, seqs, seed=i, buffers=buffers) for i in range(layers)]
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
