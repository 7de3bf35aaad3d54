"""CPU tests of the 4-bit KV cache: struct layouts, the exported symbols, the refusals of the C
entry points (before anything is launched) and the plain reference the GPU tests rely on."""
from __future__ import annotations

import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import kv4_reference as ref
import lossless_bf16_kv_amd as sz
from lossless_bf16_kv_amd import kv4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20          # stands for a device pointer; no call below reaches the GPU with it


def cache(**kw):
    c = kv4.splitzip_kv4_cache(P, P, P, P, P, P, 10, 64, 8, 128, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def batch(**kw):
    b = kv4.splitzip_kv4_batch(P, P, None, 5, 3, 5, 3, 1, 320)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def queries(**kw):
    q = kv4.splitzip_kv4_queries(P, 2048, 128, 16, 0, 0, 0, 0.1)
    for k, v in kw.items():
        setattr(q, k, v)
    return q


def call(name, c=None, b=None, q=None, **kw):
    L = kv4._lib()
    c, b, q = c or cache(), b or batch(), q or queries()
    refs = [ctypes.byref(x) for x in (c, b, q)]
    if name == "append":
        a = {"k": P, "ks": (1024, 128), "v": P, "vs": (1024, 128), "dtype": 0, **kw}
        return L.splitzip_kv4_append(refs[0], refs[1], a["k"], *a["ks"], a["v"], *a["vs"], a["dtype"], None)
    if name == "read":
        a = {"k": P, "v": P, "dtype": 0, **kw}
        return L.splitzip_kv4_read(refs[0], refs[1], a["k"], a["v"], a["dtype"], None)
    if name == "attend":
        a = {"out": P, "lse": P, "ws": None, "bytes": 0, **kw}
        return L.splitzip_kv4_attend(*refs, a["out"], a["lse"], a["ws"], a["bytes"], None)
    if name == "weigh":
        return L.splitzip_kv4_weigh(*refs, kw.get("lse", P), None)
    a = {"table": P, "stride": 5, "width": 5, "budget": 100, "sinks": 4, "recent": 8, "lens": P, "kept": P, **kw}
    return L.splitzip_kv4_evict(refs[0], refs[1], a["table"], a["stride"], a["width"], a["budget"], a["sinks"],
                                a["recent"], a["lens"], a["kept"], None)


def refused(name, word, **kw):
    assert call(name, **kw) == sz.E_INVALID
    text = sz.lib().splitzip_last_error().decode()
    assert word in text, text


def test_symbols_and_structs():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "splitzip_kv4.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(splitzip_kv4_\w+)\s*\(", text))
    assert names == {f"splitzip_kv4_{n}" for n in ("append", "read", "attend", "attend_workspace", "weigh", "evict")}
    for n in names:
        assert hasattr(sz.lib(), n)
    assert [ctypes.sizeof(x) for x in (kv4.splitzip_kv4_cache, kv4.splitzip_kv4_batch, kv4.splitzip_kv4_queries)] == [72, 56, 48]


@pytest.mark.parametrize("op", ["append", "read", "attend", "weigh", "evict"])
@pytest.mark.parametrize("field,value,word", [
    ("head_dim", 96, "head_dim"), ("head_dim", 0, "head_dim"), ("page_size", 24, "page_size"), ("page_size", 8, "page_size"),
    ("page_size", 2048, "page_size"), ("num_pages", 0, "num_pages"), ("kv_heads", 0, "kv_heads"), ("k_codes", None, "null"),
    ("status", None, "null"), ("v_codes", P + 4, "aligned"), ("weights", P + 4, "aligned")])
def test_cache_refusals(op, field, value, word):
    refused(op, word, c=cache(**{field: value}))


@pytest.mark.parametrize("op", ["append", "read", "attend", "weigh", "evict"])
@pytest.mark.parametrize("fields,word", [
    ({"lens": None}, "null"), ({"table": None}, "null"), ({"table_stride": 4}, "table_stride"), ({"n_seqs": -1}, "negative"),
    ({"total": -1}, "negative"), ({"table_width": -1}, "table_width"), ({"table_width": 1 << 25, "table_stride": 1 << 25}, "table_width"),
    ({"max_len": -1}, "max_len")])
def test_batch_refusals(op, fields, word):
    refused(op, word, b=batch(**fields))


@pytest.mark.parametrize("op", ["append", "read", "attend", "weigh"])
def test_rows_need_their_sequences(op):
    refused(op, "one row a sequence", b=batch(total=4))
    refused(op, "rows without a sequence", b=batch(n_seqs=0, cu_seqlens=P))


@pytest.mark.parametrize("op", ["attend", "weigh"])
@pytest.mark.parametrize("fields,word", [
    ({"dtype": 2}, "bf16 or fp16"), ({"q_heads": 12}, "multiple"), ({"q_heads": 0}, "multiple"), ({"window": -1}, "window"),
    ({"sinks": -1}, "sinks"), ({"scale": math.nan}, "finite"), ({"scale": math.inf}, "finite"), ({"q": None}, "null"),
    ({"q": P + 1}, "aligned")])
def test_query_refusals(op, fields, word):
    refused(op, word, q=queries(**fields))


def test_other_refusals():
    refused("append", "k and v", dtype=3)
    refused("append", "null", k=None)
    refused("append", "aligned", v=P + 1)
    refused("append", "aligned", k=P + 2, dtype=2)
    refused("read", "null", v=None)
    refused("read", "aligned", k=P + 8)
    refused("attend", "out", out=None)
    refused("attend", "out", out=P + 8)
    refused("weigh", "lse", lse=None)
    for kw in ({"budget": 0}, {"sinks": -1}, {"recent": -1}, {"sinks": 60, "recent": 41}):
        refused("evict", "budget", **kw)
    refused("evict", "null", kept=None)
    refused("evict", "out_table_stride", stride=3)
    # a call that wants a workspace and gets none
    b, need = batch(table_width=1000, table_stride=1000, max_len=64000), ctypes.c_uint64()
    c, q = cache(), queries()
    assert kv4._lib().splitzip_kv4_attend_workspace(ctypes.byref(c), ctypes.byref(b), ctypes.byref(q), ctypes.byref(need)) == 0
    assert need.value > 0
    refused("attend", "workspace", b=b)
    refused("attend", "workspace", b=b, ws=P, bytes=need.value - 1)
    L = kv4._lib()
    assert L.splitzip_kv4_attend(None, ctypes.byref(b), ctypes.byref(q), P, P, None, 0, None) == sz.E_INVALID
    assert L.splitzip_kv4_attend(ctypes.byref(c), None, ctypes.byref(q), P, P, None, 0, None) == sz.E_INVALID
    assert L.splitzip_kv4_attend(ctypes.byref(c), ctypes.byref(b), None, P, P, None, 0, None) == sz.E_INVALID


def test_nothing_to_do():
    none = batch(n_seqs=0, total=0, lens=None, table=None)
    for op in ("append", "read", "attend", "weigh", "evict"):
        assert call(op, b=none) == sz.OK


def test_python_refusals():
    for kw in ({"head_dim": 80}, {"page_size": 48}, {"num_pages": 0}, {"kv_heads": 0}):
        with pytest.raises(ValueError):
            kv4.KV4Cache(**{"num_pages": 4, **kw})
    u8 = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        kv4.KV4Cache.from_tensors(u8, u8, u8, u8, u8)
    if not torch.cuda.is_available():
        with pytest.raises(sz.SplitZipError):
            kv4.KV4Cache(4)


# ---- the reference itself ----------------------------------------------------------------------

def test_reference_quantizer():
    x = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4, np.float64)
    codes, scales = ref.quantize(x)
    assert scales.tolist() == [127] and codes[:8].tolist() == [0, 2, 2, 4, 4, 6, 6, 7]
    codes, scales = ref.quantize(np.full(32, 7.0))
    assert scales.tolist() == [128] and (codes == 6).all()          # 3.5 rounds to 4
    codes, scales = ref.quantize(-np.full(32, 6.999))
    assert scales.tolist() == [127] and (codes == 15).all()
    # the grid itself survives, and every value goes to the nearest of its block's grid
    g = np.random.default_rng(0)
    y = g.standard_normal((50, 64)) * np.exp(g.standard_normal((50, 1)) * 5)
    codes, scales = ref.quantize(y)
    z = ref.dequantize(codes, scales)
    assert np.array_equal(ref.dequantize(*ref.quantize(z)), z)
    step = 2.0 ** (scales.astype(float).repeat(32, 1) - 127)
    nearest = np.abs(np.abs(y)[..., None] - ref.GRID * step[..., None]).min(-1)
    assert np.array_equal(np.abs(z - y), nearest) and (np.sign(z) * np.sign(y) >= 0).all()
    top = np.abs(y / step).reshape(50, 2, 32).max(-1)
    assert ((3.5 <= top) & (top < 7)).all()


def test_reference_masks_and_choice():
    assert ref.sees(2, 5, None, 0).int().tolist() == [[1, 1, 1, 1, 0], [1, 1, 1, 1, 1]]
    assert ref.sees(2, 5, 2, 1).int().tolist() == [[1, 0, 1, 1, 0], [1, 0, 0, 1, 1]]
    assert ref.sees(3, 2, None, 0).int().tolist() == [[0, 0], [1, 0], [1, 1]]
    assert ref.choose([5.0, 1, 2, 2, 0, 2, 9], 7, 4, 1, 1) == [0, 2, 3, 6]
    assert ref.choose([math.nan, 0.0, -math.inf, math.nan], 4, 2, 0, 0) == [1, 2]
    assert ref.choose([1.0, 2.0], 2, 2, 0, 0) == [0, 1]
