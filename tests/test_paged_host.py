"""The paged-cache entry points' checks that need no GPU: every call below is
rejected before a launch (its pointers are never dereferenced), and the
reference of the tests against worked values."""
import ctypes
import math
import os
import re
import shutil
import subprocess

import pytest
import torch

import shared_kv_cache_gb300 as gqa
from shared_kv_cache_gb300 import build

from paged_cases import Case, ref_attention, ref_kept, ref_weights

INV, OVF, UNS = gqa.GQA_ERR_INVALID_ARGUMENT, gqa.GQA_ERR_KV_OVERFLOW, gqa.GQA_ERR_UNSUPPORTED
P = {n: 0x10000 * (i + 1) for i, n in enumerate(
    ["q", "k", "v", "qw", "kw", "cos", "sin", "pos", "kp", "vp", "tab", "cu", "seq", "qo", "out", "lse", "w", "win",
     "kept", "nsl", "ws", "dst"])}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    gqa.load_library()


def dims(**over):
    d = dict(batch=2, total_tokens=4, max_new_tokens=2, num_heads=8, kv_num_heads=2, head_size=64, page_size=16,
             num_pages=32, max_pages=8, dtype="fp16", rotary_interleaved=0, cos_cache_rows=128)
    d.update(over)
    return gqa.make_paged_dims(**d)


def append(d, **over):
    a = dict(query=P["q"], key=P["k"], value=P["v"], q_norm_weight=P["qw"], k_norm_weight=P["kw"], norm_eps=1e-6,
             cos_cache=P["cos"], sin_cache=P["sin"], positions=None, k_pages=P["kp"], v_pages=P["vp"],
             block_table=P["tab"], cu_seqlens=P["cu"], seqlens_k=P["seq"], total_sequence_length=64,
             query_out=P["qo"])
    a.update(over)
    return gqa.gqa_paged_append(d, **a)


def attend(d, **over):
    a = dict(query=P["q"], k_pages=P["kp"], v_pages=P["vp"], block_table=P["tab"], cu_seqlens=P["cu"],
             seqlens_k=P["seq"], total_sequence_length=64, scale=0.0, local_window_size=0, output=P["out"], lse=None,
             workspace=P["ws"], workspace_bytes=1 << 40)
    a.update(over)
    return gqa.gqa_paged_attention(d, **a)


def weigh(d, **over):
    a = dict(query=P["q"], lse=P["lse"], k_pages=P["kp"], block_table=P["tab"], cu_seqlens=P["cu"],
             seqlens_k=P["seq"], total_sequence_length=64, scale=0.0, local_window_size=0, weights_in=P["win"],
             weights=P["w"], workspace=P["ws"], workspace_bytes=1 << 40)
    a.update(over)
    return gqa.gqa_paged_key_weights(d, **a)


def evict(d, **over):
    a = dict(k_pages=P["kp"], v_pages=P["vp"], weights=P["w"], block_table=P["tab"], dst_block_table=P["dst"],
             dst_max_pages=4, seqlens_k=P["seq"], total_sequence_length=64, budget=32, recent=8, kept=P["kept"],
             new_seqlens=P["nsl"], workspace=None, workspace_bytes=0)
    a.update(over)
    return gqa.gqa_paged_evict(d, **a)


def header():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    return re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "gqa_paged.h")).read(), flags=re.S)


def test_binding_matches_header():
    """The ctypes mirror of gqa_paged_dims_t has the header's fields in order,
    and every function takes as many arguments as its prototype."""
    text = header()
    body = re.search(r"typedef struct \{(.*?)\}\s*gqa_paged_dims_t;", text, flags=re.S).group(1)
    assert [f for f, _ in gqa.gqa_paged_dims_t._fields_] == re.findall(r"int32_t\s+(\w+)\s*;", body)
    assert all(t is ctypes.c_int32 for _, t in gqa.gqa_paged_dims_t._fields_)
    assert set(gqa.EXPORTED_PAGED) == set(re.findall(r"\b(gqa_paged_[a-z_]+)\s*\(", text))
    for name in gqa.EXPORTED_PAGED:
        proto = re.search(r"\b" + name + r"\s*\((.*?)\)\s*;", text, flags=re.S).group(1)
        assert len(getattr(gqa.load_library(), name).argtypes) == proto.count(",") + 1, name


def test_header_is_c99(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "use.c"
    src.write_text('#include "gqa_paged.h"\nint main(void) { gqa_paged_dims_t d = {0}; '
                   'return gqa_paged_workspace_size(&d, 1, 0) != 0; }\n')
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(root, "include"), "-c",
                    str(src), "-o", str(tmp_path / "use.o")], check=True, capture_output=True, text=True)


CALLS = [append, attend, weigh, evict]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("bad", [dict(batch=0), dict(kv_num_heads=0), dict(head_size=12), dict(head_size=264),
                                 dict(page_size=4), dict(page_size=24), dict(page_size=2048), dict(num_pages=0),
                                 dict(max_pages=0), dict(dtype=7)])
def test_bad_dims(call, bad):
    assert call(dims(**bad)) == INV


@pytest.mark.parametrize("call", CALLS[:3])
@pytest.mark.parametrize("bad", [dict(total_tokens=0), dict(num_heads=7), dict(num_heads=0)])
def test_bad_token_dims(call, bad):
    assert call(dims(**bad)) == INV


@pytest.mark.parametrize("call", CALLS)
def test_lengths(call):
    assert call(dims(), total_sequence_length=129) == OVF     # 8 pages of 16
    assert call(dims(), total_sequence_length=0) == INV
    assert call(dims(num_pages=1 << 30), total_sequence_length=64) == UNS
    assert call(dims(batch=65536)) == UNS


@pytest.mark.parametrize("call,names", [
    (append, ["query", "key", "value", "k_pages", "v_pages", "block_table", "cu_seqlens", "seqlens_k", "query_out"]),
    (attend, ["query", "k_pages", "v_pages", "block_table", "cu_seqlens", "seqlens_k", "output"]),
    (weigh, ["query", "lse", "k_pages", "block_table", "cu_seqlens", "seqlens_k", "weights_in", "weights"]),
    (evict, ["k_pages", "v_pages", "weights", "block_table", "seqlens_k", "kept"]),
])
def test_pointers(call, names):
    small = {"block_table", "cu_seqlens", "seqlens_k", "lse", "weights", "weights_in", "kept"}
    for n in names:
        assert call(dims(), **{n: None}) == INV, n
        assert call(dims(), **{n: 0x777000 + (2 if n in small else 8)}) == INV, n


def test_other_checks():
    assert append(dims(), sin_cache=None) == INV
    assert append(dims(cos_cache_rows=63)) == INV
    assert append(dims(cos_cache_rows=0), positions=P["pos"]) == INV
    assert append(dims(), norm_eps=-1.0) == INV and append(dims(), norm_eps=math.nan) == INV
    assert append(dims(), key=None, value=None, query_out=P["q"]) == INV     # packed rows cannot be overwritten
    assert append(dims(), v_pages=P["kp"]) == INV
    assert append(dims(rotary_interleaved=2)) == INV
    assert attend(dims(), output=P["q"]) == INV
    assert attend(dims(), scale=math.inf) == INV
    assert attend(dims(max_new_tokens=0)) == INV
    assert weigh(dims(), scale=math.nan) == INV
    assert evict(dims(), budget=0) == INV
    assert evict(dims(), recent=33) == INV and evict(dims(), recent=-1) == INV
    assert evict(dims(), dst_max_pages=0) == INV
    assert evict(dims(), new_seqlens=P["seq"]) == INV


def test_workspace_checks():
    d = dims(head_size=128, num_heads=32, kv_num_heads=8, dtype="bf16")
    need = gqa.gqa_paged_workspace_size(d, 128)
    if need:
        assert attend(d, total_sequence_length=128, workspace_bytes=need - 1) == INV
        assert attend(d, total_sequence_length=128, workspace=None) == INV
        assert attend(d, total_sequence_length=128, workspace=P["ws"] + 8) == INV
    assert gqa.gqa_paged_workspace_size(dims(batch=0), 64) == 0


def test_python_layer_refuses_wrong_tensors():
    c = Case()
    d = {n: getattr(c, n) for n in Case.NAMES}
    with pytest.raises(ValueError, match="k_pages"):
        gqa.paged_attention(d["query"], d["k_pages"], d["v_pages"], d["table"], d["cu"], d["seqlens"], 1, 64)
    with pytest.raises(ValueError, match="k_pages"):
        gqa.paged_append(d["query"], d["key"], d["value"], d["k_pages"].float(), d["v_pages"], d["table"], d["cu"],
                         d["seqlens"], 64)


# ---------------------------------------------------------------------------
# the tests' reference
# ---------------------------------------------------------------------------
def test_reference_of_one_key_is_its_value():
    c = Case(past=(0,), new=(1,))
    out, lse, _, _ = ref_attention(c)
    v = c.gather(c.v_pages, 0, 1).double()
    assert torch.equal(out[0].view(c.Hkv, -1, c.D), v.expand(c.Hkv, c.H // c.Hkv, c.D).double())
    w, _, written = ref_weights(c, lse)
    assert torch.allclose(w[written], torch.full((c.Hkv,), c.H / c.Hkv, dtype=torch.float64))


def test_reference_weights_sum_to_the_rows():
    """Each (token, head) hands out a weight of one."""
    c = Case(past=(20, 0, 7), new=(3, 5, 0), window=9)
    _, lse, _, _ = ref_attention(c)
    zero = torch.zeros_like(c.weights)
    w, _, written = ref_weights(c, lse, weights_in=zero)
    assert math.isclose(w[written].sum().item(), 8 * c.H, rel_tol=1e-12)


def test_reference_kept():
    assert ref_kept([1.0, 5.0, 5.0, 2.0, 5.0, 0.0], 1, 3) == [1, 2, 5]
    assert ref_kept([math.nan, -math.inf, 1.0, 3.0], 1, 2) == [2, 3]
    assert ref_kept([math.nan, -math.inf, 1.0, 3.0], 1, 3) == [1, 2, 3]
    assert ref_kept([1.0, 2.0], 0, 5) == [0, 1]
