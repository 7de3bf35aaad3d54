"""CPU tests: an eviction's new lengths must not lie over the old ones, which its kernels still read; and a
table's tokens leave room for the kernels' 32-bit token numbers, which run past a sequence's end."""
from __future__ import annotations

import ctypes

import pytest

import lossless_bf16_kv_amd as sz
from lossless_bf16_kv_amd import kv4

P = 1 << 20          # stands for a device pointer; no call below reaches the GPU with it


def evict(lens, out_lens, seqs=3):
    c = kv4.splitzip_kv4_cache(P, P, P, P, P, P, 10, 64, 8, 128, 0)
    b = kv4.splitzip_kv4_batch(P, lens, None, 5, seqs, 5, seqs, 1, 320)
    # too many tokens to keep: a call whose lengths are apart is refused for that, and nothing is launched
    status = kv4._lib().splitzip_kv4_evict(ctypes.byref(c), ctypes.byref(b), P, 5, 5, (1 << 31) - 1, 0, 0, out_lens, P, None)
    assert status == sz.E_INVALID
    return sz.lib().splitzip_last_error().decode()


@pytest.mark.parametrize("apart", [0, 4, 8, -4, -8])
def test_evict_lengths_over_each_other(apart):
    assert "overlap" in evict(P + 64, P + 64 + apart)


@pytest.mark.parametrize("apart", [12, -12, 4096])
def test_evict_lengths_apart(apart):
    assert "too many" in evict(P + 64, P + 64 + apart)


@pytest.mark.parametrize("op", ["append", "attend", "weigh", "evict"])
@pytest.mark.parametrize("tokens,fits", [((1 << 31) - (1 << 16) - 1024, True), ((1 << 31) - (1 << 16), False),
                                         ((1 << 31) - 1024 * 40, False)])
def test_table_of_nearly_2_31_tokens(op, tokens, fits):
    width = tokens // 1024
    c = kv4.splitzip_kv4_cache(P, P, P, P, P, P, 10, 1024, 8, 128, 0)
    b = kv4.splitzip_kv4_batch(P, P, None, width, 3, width, 3, 1, 320)
    q = kv4.splitzip_kv4_queries(P, 2048, 128, 16, 0, 0, 0, 0.1)
    L, refs = kv4._lib(), [ctypes.byref(x) for x in (c, b, q)]
    # each call lacks something that is looked at behind the table
    status = {"append": lambda: L.splitzip_kv4_append(refs[0], refs[1], None, 1024, 128, P, 1024, 128, 0, None),
              "attend": lambda: L.splitzip_kv4_attend(*refs, None, P, None, 0, None),
              "weigh": lambda: L.splitzip_kv4_weigh(*refs, None, None),
              "evict": lambda: L.splitzip_kv4_evict(refs[0], refs[1], P, 5, 5, 0, 0, 0, P, P, None)}[op]()
    assert status == sz.E_INVALID
    assert ("table_width" in sz.lib().splitzip_last_error().decode()) == (not fits)
