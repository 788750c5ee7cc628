"""The decoder layer's passes on another stream than the current one: the memory of their buffers."""
import pytest
import torch

import w4a4_quantized_gemm_gb300 as w4
from tests.test_decoder_prompt_gpu import DIM, HKV, HQ, ints, layer_and_inputs
from w4a4_quantized_gemm_gb300 import decoder

pytestmark = pytest.mark.gpu
ROWS = 2000


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from w4a4_quantized_gemm_gb300 import build
    build.build()
    w4.lib()
    w4.w4a4_device_status()


def a_pass(kind, layer, x, r, gain):
    """A prompt, or the same tokens as a chunk into a cache, on a stream: returns a function of it and its results."""
    rope, at, starts = w4.w4a4_rope_table(ROWS, DIM, 1e6), ints(list(range(ROWS))), ints([0, ROWS])
    owners, lengths = ints([0] * ROWS), ints([ROWS])
    cache = decoder.paged_cache(1, ROWS, HKV, DIM)
    cache.workspace(HQ)

    def run(stream=None):
        stream_r, out = streams.pop(), outs.pop()
        if kind == "prompt":
            layer.prompt(x, stream_r, at, starts, rope, gain, out, stream=stream)
        else:
            layer.chunk(x, stream_r, at, owners, starts, lengths, cache, rope, gain, out, stream=stream)
        return stream_r, out

    streams, outs = [r.clone() for _ in range(4)], [torch.empty_like(x) for _ in range(4)]
    return run


@pytest.mark.parametrize("kind", ["prompt", "chunk"])
@pytest.mark.parametrize("handle", [False, True])
def test_buffers_made_for_a_side_stream(kind, handle):
    """No memory whose last use on the current stream is still to come."""
    layer, x, r, gain = layer_and_inputs(ROWS, 1, 4)
    run = a_pass(kind, layer, x, r, gain)
    side = torch.cuda.Stream()
    width = (HQ + 2 * HKV) * DIM  # what the fused q|k|v output takes
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [torch.full((ROWS, w), 7.0, dtype=torch.float16, device="cuda") for w in (width, HQ * DIM, HQ * DIM)]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # a tenth of a second
    copies = [h.clone() for h in held]
    del held
    got = run(side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert all(torch.all(c == 7) for c in copies)
    want = run()
    torch.cuda.synchronize()
    assert w4.w4a4_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("kind", ["prompt", "chunk"])
@pytest.mark.parametrize("first", ["side", "current"])
def test_buffers_outlive_the_layer(kind, first):
    """A layer dropped while a side stream still runs its pass, whose buffers were made for it or for the current one."""
    layer, x, r, gain = layer_and_inputs(ROWS, 1, 5)
    run = a_pass(kind, layer, x, r, gain)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    if first == "current":
        run()
        torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    run(side)
    b = layer.rows(ROWS, side)
    buffers = [(t.data_ptr(), t.numel() * t.element_size()) for t in (b.qkv_out, b.attn, b.o_out, b.h, b.ws)]
    weights = layer.qkv, layer.o, layer.gate_up, layer.down, layer.q_gain, layer.k_gain, layer.mlp_gain
    del layer, run, b
    again = [torch.empty(size, dtype=torch.uint8, device="cuda") for _, size in buffers]
    busy = not side.query()
    torch.cuda.synchronize()
    spans = [(p, p + n) for p, n in buffers]
    assert busy and not any(lo < t.data_ptr() + t.numel() and t.data_ptr() < hi for t in again for lo, hi in spans)
    assert len(weights) == 7  # they are the caller's to keep, as tensors are
