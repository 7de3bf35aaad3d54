"""CPU tests of what the 4-bit KV cache's calls launch, and of what they refuse because no launch or 32-bit number
holds it.  No call here reaches the GPU."""
from __future__ import annotations

import ctypes
import types

import pytest
import torch

import lossless_bf16_kv_amd as sz
from lossless_bf16_kv_amd import kv4
from test_kv4_host import batch, cache, call, queries

MOST = (1 << 31) - 1


def refused(name, word, **kw):
    assert call(name, **kw) == sz.E_INVALID
    text = sz.lib().splitzip_last_error().decode()
    assert word in text, text


# The kernels count up to 1024 tokens past a budget in 32 bits.
@pytest.mark.parametrize("budget", [MOST, MOST - 127, MOST - 1023, MOST - 65535])
def test_evict_budget_of_nearly_2_31(budget):
    refused("evict", "too many tokens to keep", c=cache(kv_heads=1), b=batch(n_seqs=1, total=1), budget=budget, lens=1 << 21)


@pytest.mark.parametrize("budget", [MOST, 1 << 32, (1 << 32) + 5])
def test_evict_budget_past_32_bits_is_not_cut(budget):
    # before anything of the cache is looked at
    with pytest.raises(ValueError, match="budget"):
        kv4.KV4Cache.evict(None, None, None, None, budget)


def launches(op, c=None, b=None, q=None, budget=100):
    """(workgroups, threads) of each launch."""
    f = kv4._lib().splitzip_kv4_launches
    f.argtypes = [ctypes.c_int32, *(ctypes.POINTER(t) for t in (kv4.splitzip_kv4_cache, kv4.splitzip_kv4_batch,
                                                                kv4.splitzip_kv4_queries)), ctypes.c_int32,
                  ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(ctypes.c_uint32)]
    groups, threads = (ctypes.c_uint64 * 2)(), (ctypes.c_uint32 * 2)()
    status = f(op, *(ctypes.byref(x) for x in (c or cache(), b or batch(), q or queries())), budget, groups, threads)
    assert status == sz.OK, sz.lib().splitzip_last_error().decode()
    return [(g, t) for g, t in zip(groups, threads) if g]


EVICT = 2


# HIP launches fewer than 2^32 threads at a time.  A choose launch that fails leaves nothing for the move behind it.
@pytest.mark.parametrize("seqs,budget", [(1 << 19, 128), (1 << 20, 1), (1 << 21, 16)])
def test_evict_of_too_many_heads(seqs, budget):
    refused("evict", "too many sequences and heads", b=batch(n_seqs=seqs, total=seqs), budget=budget, sinks=0, recent=0, lens=1 << 30)


@pytest.mark.parametrize("seqs,budget", [(3, 100), ((1 << 19) - 1, 16), (512, 1 << 19), (1, 64 << 20)])
def test_evict_launches(seqs, budget):
    b = batch(n_seqs=seqs, total=seqs, max_len=MOST, table_width=1 << 20, table_stride=1 << 20)
    choose, move = launches(EVICT, b=b, budget=budget)
    assert choose == (seqs * 8, 1024) and move[1] == 256
    assert all(g * t < 1 << 32 for g, t in (choose, move))
    # every token has a workgroup where that fits, and some workgroup takes it in turn where not
    turns = -(-budget // 128)
    assert move[0] == seqs * 8 * (turns if seqs * 8 * turns * 256 < 1 << 32 else ((1 << 32) - 1) // 256 // (seqs * 8))


@pytest.mark.parametrize("max_len,turns", [(0, 1), (1, 1), (128, 1), (129, 2), (1000, 8), (4096, 8), (MOST, 8)])
def test_evict_launch_goes_by_the_longest_sequence(max_len, turns):
    # no sequence keeps more tokens than it has
    choose, move = launches(EVICT, b=batch(table_width=100, table_stride=100, max_len=max_len), budget=1000)
    assert choose == (24, 1024) and move == (24 * turns, 256)


def test_evict_launch_goes_by_the_table():
    _, move = launches(EVICT, b=batch(max_len=MOST), budget=1 << 20)          # 5 pages of 64 tokens
    assert move == (24 * 3, 256)


ATTEND, WEIGH = 0, 1


# seqs, rows a sequence, KV heads, group, D, tokens a table holds; max_q: all rows, as a caller without a better guess says
@pytest.mark.parametrize("op", [ATTEND, WEIGH])
@pytest.mark.parametrize("seqs,n,heads,group,d,tokens", [
    (1024, 32, 8, 8, 128, 8192), (512, 128, 8, 8, 128, 8192), (256, 64, 8, 8, 256, 1 << 20), (512, 100, 8, 8, 128, 1 << 20),
    (1 << 18, 1, 8, 8, 128, 1 << 20), (1 << 18, 3, 16, 4, 64, 1 << 20), (1, 1 << 20, 1, 64, 128, 1 << 20), (1, 1, 1, 1, 64, 16),
    (4, 1 << 22, 1, 16, 256, 1 << 24)])
def test_attend_and_weigh_launches(op, seqs, n, heads, group, d, tokens):
    width = tokens // 16
    b = batch(n_seqs=seqs, total=seqs * n, cu_seqlens=1 << 20, table_width=width, table_stride=width, max_q=seqs * n, max_len=tokens)
    got = launches(op, c=cache(page_size=16, kv_heads=heads, head_dim=d), b=b,
                   q=queries(q_heads=heads * group, token_stride=heads * group * d, head_stride=d))
    assert got and got[0][0] % (seqs * heads) == 0
    assert all(g * t < 1 << 32 for g, t in got), got


@pytest.mark.parametrize("op", ["attend", "weigh"])
@pytest.mark.parametrize("seqs", [1 << 22, 1 << 24])
def test_attend_and_weigh_of_too_many_heads(op, seqs):
    refused(op, "sequences and heads", b=batch(n_seqs=seqs, total=seqs, max_q=1))


@pytest.mark.parametrize("op", ["append", "read"])
@pytest.mark.parametrize("d,rows,heads", [(64, 1 << 26, 8), (128, 1 << 25, 8), (256, 1 << 24, 8), (256, (1 << 27) + 1, 1)])
def test_append_and_read_of_too_many_rows(op, d, rows, heads):
    b = batch(n_seqs=1, total=rows, cu_seqlens=1 << 20)
    refused(op, "more rows and heads than a launch holds", c=cache(head_dim=d, kv_heads=heads), b=b)


# The kernels count past a sequence's last row in 32 bits: by 256 in tiles, by 4097 tiles of 32 where rows go in turn.
@pytest.mark.parametrize("op", ["attend", "weigh"])
@pytest.mark.parametrize("total,heads", [(MOST - 1, 1), (MOST - 255, 1), (MOST - 65535, 1), (MOST - 4097 * 32, 1), ((1 << 30) - 1, 2),
                                         ((1 << 25) - 1, 64)])
def test_rows_of_nearly_2_31(op, total, heads):
    b = batch(n_seqs=1, total=total, cu_seqlens=1 << 20)
    refused(op, "total * q_heads must be below 2^31 - 2^18", c=cache(kv_heads=1), b=b, q=queries(q_heads=heads))


def workspace(seqs, n, tokens, heads=8, group=8, d=128, max_q=None, max_len=None):
    width, need = tokens // 16, ctypes.c_uint64()
    c = cache(page_size=16, kv_heads=heads, head_dim=d)
    b = batch(n_seqs=seqs, total=seqs * n, cu_seqlens=1 << 20, table_width=width, table_stride=width, max_q=max_q or n,
              max_len=max_len or tokens)
    q = queries(q_heads=heads * group, token_stride=heads * group * d, head_stride=d)
    refs = [ctypes.byref(x) for x in (c, b, q, need)]
    assert kv4._lib().splitzip_kv4_attend_workspace(*refs) == sz.OK
    got = launches(ATTEND, c, b, q)
    return need.value, got[0][0]


# Splits that are there for balance are few where there are many sequences, however long the table could make these.
@pytest.mark.parametrize("seqs,n,tokens,most", [(256, 1, 1 << 20, 80 << 20), (256, 1, 1 << 17, 80 << 20), (1024, 4, 1 << 17, 300 << 20),
                                                (4096, 1, 1 << 20, 0), (1, 1, 1 << 20, 80 << 20), (32, 1, 1 << 20, 80 << 20)])
def test_attend_workspace_of_wide_tables(seqs, n, tokens, most):
    got, groups = workspace(seqs, n, tokens)
    assert got <= most and groups <= max(seqs * 8, 16 * 1024)


def test_attend_workspace_has_an_end():
    # hints that say far too little: one query a sequence where there are thousands
    got, _ = workspace(1, 4096, 1 << 17, max_q=1)
    assert 0 < got <= 512 << 20


@pytest.mark.parametrize("seqs,n,tokens,splits", [(256, 1, 8192, 2), (32, 1, 32768, 8), (1, 1, 4096, 16), (64, 1, 1 << 17, 32)])
def test_attend_splits(seqs, n, tokens, splits):
    got, groups = workspace(seqs, n, tokens)
    assert groups == seqs * 8 * splits and got == splits * seqs * n * 64 * (128 + 2) * 4


# max_q 0: not known.  The rows of a tile go by the mean, and empty workgroups have an end.
@pytest.mark.parametrize("seqs,n,group,threads,least", [(64, 3, 4, 256, 1), (256, 1, 8, 256, 1), (64, 100, 4, 512, 2), (16, 2048, 4, 512, 32),
                                                        (1, 4096, 4, 512, 64), (1, 1, 8, 256, 1)])
def test_attend_launch_without_max_q(seqs, n, group, threads, least):
    b = batch(n_seqs=seqs, total=seqs * n, cu_seqlens=1 << 20, table_width=64, table_stride=64, max_q=0, max_len=256)     # no splits
    (groups, got), *_ = launches(ATTEND, b=b, q=queries(q_heads=8 * group, token_stride=1024 * group))
    tiles = groups // (seqs * 8)
    assert got == threads and tiles >= least
    if seqs > 1:
        assert groups <= max(16384 + seqs * 8, 3 * least * seqs * 8)


def test_weigh_launch_without_max_q():
    # up to 16 rows a sequence stay in registers; a second launch is there for sequences that have more
    b = batch(n_seqs=64, total=192, cu_seqlens=1 << 20, table_width=64, table_stride=64, max_len=4096)
    got = []
    for max_q in (0, 3, 192):
        b.max_q = max_q
        got.append(launches(WEIGH, b=b, q=queries(q_heads=32, token_stride=4096)))
    assert got[0][:1] == got[1] != got[2] and len(got[0]) == 2 and got[0][1][0] <= 8192 and len(got[2]) == 1


def test_python_says_that_it_does_not_know():
    t = torch.zeros(3, 4, dtype=torch.int32)
    me = types.SimpleNamespace(page_size=16, _int32=lambda t, name, shape=None: 0)
    assert kv4.KV4Cache._batch(me, t, t, t, 300, None, None).max_q == 0
    assert kv4.KV4Cache._batch(me, t, t, t, 300, 7, None).max_q == 7


@pytest.mark.parametrize("max_q", [MOST, MOST + 1, 1 << 32, (1 << 32) + 1])
def test_python_hint_past_32_bits_is_not_cut(max_q):
    t = torch.zeros(3, 4, dtype=torch.int32)
    me = types.SimpleNamespace(page_size=16, _int32=lambda t, name, shape=None: 0)
    assert kv4.KV4Cache._batch(me, t, t, t, 300, max_q, None).max_q == MOST
    assert kv4.KV4Cache._batch(me, t, t, t, 300, None, max_q).max_len == MOST


@pytest.mark.parametrize("op", ["attend", "weigh"])
@pytest.mark.parametrize("scale", [3e38, -3e38, 2.4e38])
def test_scale_that_is_infinite_in_base_2(op, scale):
    # scores are held as powers of two: scale * log2(e) must be a 32-bit number too
    refused(op, "scale is not finite", q=queries(scale=scale))
