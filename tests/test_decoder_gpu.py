"""The decoder layer's decode step: what lies between the quantised linears, from the linears'
own outputs, against definitions in 64 bits; and the same step from a CUDA graph."""
import pytest
import torch

import w4a4_quantized_gemm_gb300 as w4
from w4a4_quantized_gemm_gb300 import decoder

pytestmark = pytest.mark.gpu
F64 = torch.float64
U16 = 2.0 ** -11


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from w4a4_quantized_gemm_gb300 import build
    build.build()
    w4.lib()
    w4.w4a4_device_status()


def rms(x, gain, eps=1e-6):
    return x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * gain.to(F64)


def turn(x, rope, pos):
    c, s = rope[pos.long(), 0].to(F64)[:, None], rope[pos.long(), 1].to(F64)[:, None]
    a, b = x.chunk(2, dim=-1)
    return torch.cat((a * c - b * s, b * c + a * s), dim=-1)


def close(got, ref, tol, what):
    err = (got.to(F64) - ref).abs()
    assert torch.all(err <= tol * (1 + ref.abs())), f"{what}: {float((err / (1 + ref.abs())).max()):.2e} > {tol:.1e}"


@pytest.mark.parametrize("stream_dtype", [torch.float16, torch.float32])
def test_decode_steps(stream_dtype):
    seqs, hidden, hq, hkv, dim, room = 3, 512, 8, 2, 128, 50
    layer = decoder.random_layer(hidden, 640, hq, hkv, dim, seqs)
    cache = decoder.paged_cache(seqs, room, hkv, dim, page_size=8)
    k_pool, v_pool, table = cache._keep[:3]
    rope = w4.w4a4_rope_table(room, dim, 1e6)
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")
    gain = (1 + 0.1 * rand(hidden)).half()
    starts = torch.tensor([0, 17, 40], device="cuda", dtype=torch.int32)
    history = [[[], []] for _ in range(seqs)]
    for b, n in enumerate(starts.tolist()):  # what the cache already holds
        k, v = rand(n, hkv, dim).half(), rand(n, hkv, dim).half()
        tok = torch.arange(n, device="cuda")
        for pool, x, i in ((k_pool, k, 0), (v_pool, v, 1)):
            pool[table[b, tok // 8].long(), tok % 8] = x
            history[b][i] = list(x.to(F64))
    for step in range(4):
        pos = starts + step
        x, r = rand(seqs, hidden).half(), (3 * rand(seqs, hidden)).to(stream_dtype)
        before, x_next = r.clone().to(F64), torch.empty_like(x)
        layer.step(x, r, pos, pos + 1, cache, rope, gain, x_next)
        torch.cuda.synchronize()
        assert w4.w4a4_device_status() == 0
        qkv = layer.qkv_out.to(F64).unflatten(1, (hq + 2 * hkv, dim))
        q = turn(rms(qkv[:, :hq], layer.q_gain), rope, pos)
        k = turn(rms(qkv[:, hq:hq + hkv], layer.k_gain), rope, pos)
        close(layer.q, q, 2 * U16, "q")
        for b in range(seqs):
            history[b][0].append(k[b].half().to(F64))
            history[b][1].append(qkv[b, hq + hkv:])
            kk, vv = (torch.stack(h) for h in history[b])
            a = torch.einsum("hgd,nhd->hgn", layer.q[b].to(F64).view(hkv, -1, dim), kk) * dim ** -0.5
            # the probabilities' rounding, U16 of sum p |v|, and k's own rounding in the reference
            close(layer.attn[b], torch.einsum("hgn,nhd->hgd", a.softmax(-1), vv).reshape(hq, dim), 8 * U16, f"attn {b}")
        mid = before + layer.o_out.to(F64)
        close(layer.x_mlp, rms(mid, layer.mlp_gain), 2 * U16, "x_mlp")
        u = U16 if stream_dtype == torch.float16 else 2.0 ** -24
        after = mid + layer.down_out.to(F64)  # r was rounded once in between
        close(r, after, 3 * u + 2.0 ** -20, "r")
        close(x_next, rms(after, gain), 4 * U16, "x_next")


def test_step_from_a_graph_follows_the_lengths():
    seqs, hidden, hq, hkv, dim, room = 2, 256, 4, 4, 64, 40
    layer = decoder.random_layer(hidden, 256, hq, hkv, dim, seqs)
    caches = [decoder.paged_cache(seqs, room, hkv, dim) for _ in range(2)]
    caches[1]._keep[2].copy_(caches[0]._keep[2])
    rope = w4.w4a4_rope_table(room, dim, 1e4)
    gain = torch.ones(hidden, device="cuda", dtype=torch.float16)
    n = torch.ones(seqs, dtype=torch.int32, device="cuda")
    pos = n - 1
    x, x_next = (torch.zeros(seqs, hidden, device="cuda", dtype=torch.float16) for _ in range(2))
    r = torch.zeros(seqs, hidden, device="cuda")
    layer.step(x, r, pos, n, caches[0], rope, gain, x_next)  # workspaces exist before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step(x, r, pos, n, caches[0], rope, gain, x_next)
    g = torch.Generator(device="cuda").manual_seed(1)
    for step in range(5):
        x.copy_(torch.randn(seqs, hidden, generator=g, device="cuda"))
        r0 = torch.randn(seqs, hidden, generator=g, device="cuda")
        n.fill_(step + 1), pos.fill_(step)
        r.copy_(r0)
        graph.replay()
        torch.cuda.synchronize()
        want_x, want_r = x_next.clone(), r.clone()
        r.copy_(r0)
        layer.step(x, r, pos, n, caches[1], rope, gain, x_next)  # the same step, eagerly, on the other cache
        torch.cuda.synchronize()
        assert torch.equal(x_next, want_x) and torch.equal(r, want_r), step
    assert w4.w4a4_device_status() == 0
