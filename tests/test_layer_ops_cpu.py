"""The decoder-layer operators (cache append, paged attention, block norm) refuse bad
calls on the host, before any launch; the binding's argument structs have the header's
layout."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import w4a4_quantized_gemm_gb300 as w4
from tests.layer_structs import FORMATS, fields, pack
from w4a4_quantized_gemm_gb300 import build as wbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000  # never dereferenced: every call below fails on the host
GOOD = 7 if not torch.cuda.is_available() else None  # every check passed, only the device is missing


@pytest.fixture(scope="module")
def L():
    wbuild.build()
    return w4.lib()


def cache(**over):
    d, size = over.get("head_dim", 128), 1 if over.get("dtype") == 3 else 2
    v = dict(k=A, v=A, page_table=A, k_page_stride=16 * 8 * d, k_token_stride=8 * d,
             k_head_stride=d, v_page_stride=16 * 8 * d, v_token_stride=8 * d, v_head_stride=d, table_stride=10,
             seqs=4, max_pages=10, pages=40, page_size=16, kv_heads=8, head_dim=d, dtype=0)
    assert d * size % 16 == 0 or "k_head_stride" in over
    return pack("w4a4_kv_cache", **{**v, **over})


def append(**over):
    v = dict(q=A, k=A, v=A, q_out=A + 64, positions=A, rope=A, q_token_stride=4096,
             q_head_stride=128, k_token_stride=4096, k_head_stride=128, v_token_stride=4096, v_head_stride=128,
             out_token_stride=2048, out_head_stride=128, tokens=4, q_heads=16, dtype=0, rope_rows=100, rot_dim=128,
             eps=1e-6)
    return pack("w4a4_kv_append_args", **{**v, **over})


def attention(**over):
    v = dict(q=A, out=A, lengths=A, workspace=A, workspace_bytes=1 << 40,
             q_token_stride=2048, q_head_stride=128, out_token_stride=2048, out_head_stride=128, scale=0.1,
             q_heads=16, dtype=0)
    return pack("w4a4_paged_attention_args", **{**v, **over})


def norm(**over):
    v = dict(y=A, r=A, r_out=A, x=A, y_stride=1024, r_stride=1024, r_out_stride=1024,
             x_stride=1024, rows=4, width=1024, dtype=0, res_dtype=0, post=1, pre=1, scale=1.0, eps=1e-6)
    return pack("w4a4_block_norm_args", **{**v, **over})


def test_struct_layouts_match_the_header(tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\ntypedef void* cudaStream_t;\n' + re.sub(
        r"#include <cuda_runtime_api.h>", "", open(os.path.join(ROOT, "include", "w4a4.h")).read()) +
        "int main(void) {\n" + "".join(
            'printf("%s.%s %%zu\\n", offsetof(%s, %s));\n' % (n, f, n, f) for n in
            FORMATS
            for f in fields(n)) + "return 0; }\n")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-o", str(exe), str(src)], check=True)
    want = dict(l.split() for l in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    for name, fmt in FORMATS.items():
        codes = [c for n, c in re.findall(r"(\d*)([Qqif])", fmt.format) for _ in range(int(n or 1))]
        names = fields(name)
        assert len(codes) == len(names), name
        at = 0
        for c, f in zip(codes, names):
            assert int(want[f"{name}.{f}"]) == at, f"{name}.{f}"
            at += 8 if c in "Qq" else 4
        assert at == fmt.size
    assert w4._CACHE.format == FORMATS["w4a4_kv_cache"].format


@pytest.mark.parametrize("over, status", [
    (dict(bytes=8), 1), (dict(seqs=-1), 1), (dict(page_size=0), 1), (dict(kv_heads=0), 1), (dict(dtype=2), 1),
    (dict(dtype=4), 1), (dict(head_dim=112), 2), (dict(head_dim=32), 2), (dict(k=0), 1), (dict(page_table=0), 1),
    (dict(k=A + 8), 3), (dict(v=A + 2), 3), (dict(page_table=A + 2), 3), (dict(k_scale=A + 1), 3),
    (dict(k_token_stride=1028), 3), (dict(v_head_stride=-128), 3), (dict(k_page_stride=1 << 40), 3),
    (dict(dtype=3, k_token_stride=1032), 3), (dict(table_stride=9), 1), (dict(max_pages=1 << 28, table_stride=1 << 28), 2),
    (dict(max_pages=(1 << 26) + 1, table_stride=1 << 27), 2), (dict(table_stride=0), 1),
    (dict(pages=-1), 1),
])
def test_cache_refusals(L, over, status):
    c = cache(**over)
    assert L.w4a4_kv_append(c, append(), None) == status
    assert L.w4a4_paged_attention(c, attention(), None) == status


@pytest.mark.parametrize("over, status", [
    (dict(bytes=0), 1), (dict(tokens=-1), 1), (dict(q_heads=-1), 1), (dict(dtype=2), 1), (dict(dtype=1), 1),
    (dict(dtype=3), 1), (dict(rot_dim=0), 1), (dict(rope_rows=0), 1), (dict(rot_dim=24), 2), (dict(rot_dim=144), 2),
    (dict(k=0), 1), (dict(v=0), 1), (dict(positions=0), 1), (dict(q=0), 1), (dict(q_out=0), 1),
    (dict(q=A + 2), 3), (dict(q_gain=A + 8), 3), (dict(rope=A + 4), 3), (dict(positions=A + 2), 3), (dict(seqs=A + 1), 3),
    (dict(q_token_stride=4100), 3), (dict(out_head_stride=-8), 3),
    (dict(q_out=A), 1),  # in place with other strides
    (dict(tokens=0), 0), (dict(tokens=0, q=0), 0),
])
def test_append_refusals(L, over, status):
    assert L.w4a4_kv_append(cache(), append(**over), None) == status
    assert L.w4a4_kv_append(None, append(), None) == 1
    assert L.w4a4_kv_append(cache(), None, None) == 1


@pytest.mark.parametrize("over, status", [
    (dict(bytes=1), 1), (dict(window=-1), 1), (dict(dtype=1), 1), (dict(dtype=2), 1), (dict(q_heads=0), 1),
    (dict(q_heads=12), 2), (dict(q_heads=1 << 20), 2), (dict(q=0), 1), (dict(out=0), 1), (dict(lengths=0), 1),
    (dict(workspace=0), 1), (dict(out=A + 4), 3), (dict(workspace=A + 8), 3), (dict(lse=A + 2), 3),
    (dict(lengths=A + 1), 3), (dict(q_head_stride=4), 3), (dict(workspace_bytes=1000), 4),
])
def test_attention_refusals(L, over, status):
    assert L.w4a4_paged_attention(cache(), attention(**over), None) == status
    assert L.w4a4_paged_attention(cache(seqs=0), attention(), None) == 0
    assert L.w4a4_paged_attention(cache(seqs=1 << 24), attention(), None) == 2
    assert L.w4a4_paged_attention(None, attention(), None) == 1


def test_attention_workspace_size(L):
    size = L.w4a4_paged_attention_workspace_bytes
    assert size(4, 16, 8, 128) > 0
    assert size(4, 16, 8, 128) < size(4000, 16, 8, 128)
    assert size(0, 16, 8, 128) > 0
    for bad in ((-1, 16, 8, 128), (4, 12, 8, 128), (4, 4, 8, 128), (4, 16, 0, 128), (4, 16, 8, 100)):
        assert size(*bad) == 0
    need = size(4, 16, 8, 128)
    assert L.w4a4_paged_attention(cache(), attention(workspace_bytes=need - 1), None) == 4


@pytest.mark.parametrize("over, status", [
    (dict(bytes=3), 1), (dict(rows=-1), 1), (dict(rows_per_gate=-1), 1), (dict(dtype=2), 1), (dict(dtype=3), 1),
    (dict(res_dtype=1), 1), (dict(post=3), 1), (dict(pre=-1), 1), (dict(width=1004), 2), (dict(width=0), 2),
    (dict(width=16392), 2), (dict(y=0), 1), (dict(r=0), 1), (dict(r_out=0), 1), (dict(y=A + 8), 3), (dict(gate=A + 2), 3),
    (dict(pre_bias=A + 4), 3), (dict(y_stride=1020), 3), (dict(r_stride=1016), 1), (dict(x_stride=512), 1),
    (dict(gate=A, gate_stride=512, rows_per_gate=1), 1), (dict(rows=0), 0),
])
def test_norm_refusals(L, over, status):
    assert L.w4a4_block_norm(norm(**over), None) == status
    assert L.w4a4_block_norm(None, None) == 1


@pytest.mark.skipif(torch.cuda.is_available(), reason="good calls would launch on a machine with a GPU")
def test_good_calls_reach_the_device_check(L):
    for kind in (0, 1, 3):
        act = 1 if kind == 1 else 0
        assert L.w4a4_kv_append(cache(dtype=kind), append(dtype=act), None) == GOOD
        assert L.w4a4_paged_attention(cache(dtype=kind), attention(dtype=act), None) == GOOD
    assert L.w4a4_kv_append(cache(), append(q=A, q_out=A, out_token_stride=4096), None) == GOOD  # in place
    assert L.w4a4_kv_append(cache(), append(rope=0, rot_dim=0, rope_rows=0), None) == GOOD
    assert L.w4a4_kv_append(cache(), append(q_heads=0, q=0, q_out=0), None) == GOOD
    assert L.w4a4_block_norm(norm(), None) == GOOD
    assert L.w4a4_block_norm(norm(x=0, x_stride=0, res_dtype=2), None) == GOOD
    assert L.w4a4_rope_table(ctypes.c_void_p(A), 10, 128, 1e6, None) == GOOD


def test_rope_table_refusals(L):
    p = ctypes.c_void_p(A)
    assert L.w4a4_rope_table(p, -1, 128, 1e6, None) == 1
    assert L.w4a4_rope_table(p, 10, 128, 0.0, None) == 1
    assert L.w4a4_rope_table(p, 10, 24, 1e6, None) == 2
    assert L.w4a4_rope_table(p, 10, 272, 1e6, None) == 2
    assert L.w4a4_rope_table(None, 10, 128, 1e6, None) == 1
    assert L.w4a4_rope_table(ctypes.c_void_p(A + 4), 10, 128, 1e6, None) == 3
    assert L.w4a4_rope_table(None, 0, 128, 1e6, None) == 0


def test_binding_refuses_tensors_it_cannot_describe(L):
    """On the host, from shapes and types alone: no device is touched."""
    k = torch.zeros(2, 16, 8, 128, dtype=torch.float16)
    table = torch.zeros(1, 2, dtype=torch.int32)
    for args in ((k, k[:, :8], table), (k, k.float(), table), (k.float(), k.float(), table), (k, k, table.long()),
                 (k, k, table), (k[0], k[0], table), (k, k, table[0])):  # (k, k, table): not on a GPU
        with pytest.raises(w4.W4A4Error):
            w4.PagedKVCache(*args)
    y = torch.zeros(3, 64, dtype=torch.float16)
    for args in ((y, y, y, y), (y, y[:2], y, y), (y, y, y[:, ::2], y), (None, y, y, y), (y, "r", y, y), (y.to_sparse(), y, y, y)):
        with pytest.raises(w4.W4A4Error):
            w4.w4a4_block_norm(*args)
    for args, named in (((y,), {}), ((y, y, y, y), dict(y=y)), ((y, y, y, y), dict(gain=y)), ((y,) * 16, {})):
        with pytest.raises(TypeError):
            w4.w4a4_block_norm(*args, **named)
    for args, named in (((y, y, y, y), dict(eps="a")), ((y, y, y, y), dict(rows_per_gate=1.5)), ((y, y, y, y), dict(stream="s"))):
        with pytest.raises(w4.W4A4Error):
            w4.w4a4_block_norm(*args, **named)
    for cache in (None, object(), 3):
        with pytest.raises(w4.W4A4Error):
            w4.w4a4_paged_attention(y, cache, y, y)
        with pytest.raises(w4.W4A4Error):
            w4.w4a4_kv_append(y, y, y, y, cache, y)
    with pytest.raises(AttributeError):
        w4.w4a4_no_such_function
    assert "rows_per_gate" in w4.w4a4_block_norm.__doc__


def test_status_string_of_the_index_status(L):
    assert b"outside its table" in L.w4a4_status_string(w4.W4A4_ERR_INDEX)
