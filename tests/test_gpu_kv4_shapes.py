"""GPU tests of the 4-bit KV cache where its kernels change their shape: every number of rows that
has a tile of its own, splits of ragged sequences, masks and scales in each, sequences longer than
the registers of an eviction hold, prompts' weights with odd groups, and the decode example."""
from __future__ import annotations

import math
import os
import sys

import pytest
import torch

import kv4_reference as ref
from test_gpu_kv4 import BF16, FP16, Setup, check_attend, check_evict

pytestmark = pytest.mark.gpu

# queries of the longest sequence: with a group of 4, 20, 52, 100 and 300 rows
COUNTS = [(5, 2, 1, 0), (13, 1, 5, 0), (25, 12, 5, 2), (75, 30, 3, 0)]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attend_row_tiles(d, dtype, counts):
    s = Setup([401, 130, 5, 17], counts, heads=2, d=d, page=32, seed=d + counts[0])
    check_attend(s, 8, dtype)
    check_attend(s, 8, dtype, window=50, sinks=7)
    check_attend(s, 8, dtype, scale=-0.3)
    check_attend(s, 8, dtype, window=33, sinks=1, scale=0.0)
    s.cache.check()


@pytest.mark.parametrize("counts", [(1, 1, 1, 1), *COUNTS])
@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, FP16), (256, BF16)])
def test_attend_row_tiles_with_nan(d, dtype, counts):
    s = Setup([401, 130, 5, 17], counts, heads=2, d=d, page=32, seed=counts[0])
    page = lambda q, j: (int(s.table_h[q, j // 32]), j % 32)
    for q, j, h in ((0, 398, 0), (0, 20, 1), (1, 129, 1), (1, 3, 0), (2, 0, 1), (3, 16, 0), (0, 352, 1)):
        p, o = page(q, j)
        s.cache.v_scales[p, h, j % (d // 32), o] = 255
    for q, j in ((0, 380), (1, 127), (3, 2)):
        p, o = page(q, j)
        s.cache.k_scales[p, 1, o, 0] = 255
    for window, sinks in ((None, 0), (40, 2), (4, 0)):
        q = s.queries(4, dtype)
        out, lse = s.cache.attend(q.cuda(), s.table, s.lens, s.cu, window=window, sinks=sinks)
        eo, to, el, tl = ref.attend(ref.Cache(s.cache), q.double(), s.rows(), s.lens_l, s.counts, d ** -0.5, window, sinks, dtype)
        out, lse = out.cpu().double(), lse.cpu().double()
        assert torch.equal(lse.isnan(), el.isnan())
        assert torch.equal(out.isnan(), eo.isnan())
        assert ((out - eo).abs() <= to)[~eo.isnan()].all()


@pytest.mark.parametrize("d,group", [(64, 2), (128, 5)])
@pytest.mark.parametrize("max_len", [None, 300])
def test_attend_splits_of_ragged_lengths(d, group, max_len):
    # more splits than a joined row has lanes, sequences of one split and of none; and a hint that says too little
    s = Setup([9001, 130, 256, 257, 0, 1], [1] * 6, heads=1, d=d, page=64, seed=d)
    check_attend(s, group, BF16, cu=None, max_len=max_len)
    check_attend(s, group, BF16, cu=None, max_len=max_len, window=4500, sinks=300)
    s.cache.check()


def test_attend_tokens_of_one_page_and_many():
    # groups of 16 tokens of one pair on different pages, and first tokens that end inside a page
    for page, sinks in ((16, 24), (128, 130)):
        s = Setup([700, 333], [1, 3], heads=1, d=128, page=page, seed=page)
        check_attend(s, 4, BF16, window=40, sinks=sinks)
        check_attend(s, 16, BF16, window=300, sinks=sinks)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("counts,group,window,sinks", [((150, 70, 3, 1), 3, None, 0), ((150, 70, 3, 1), 3, 40, 5),
                                                       ((33, 20, 3, 7), 7, 300, 0)])
def test_weigh_prompts(d, dtype, counts, group, window, sinks):
    s = Setup([600, 70, 64, 270], counts, heads=2, d=d, page=32, seed=d + group)
    q = s.queries(2 * group, dtype)
    mask = {"window": window, "sinks": sinks}
    _, lse = s.cache.attend(q.cuda(), s.table, s.lens, s.cu, **mask)
    lse[10:13, 1] = -math.inf                                   # add nothing
    r = ref.Cache(s.cache)
    s.cache.weigh(q.cuda(), lse, s.table, s.lens, s.cu, **mask)
    w, tol = ref.weigh(r, q.double(), lse.cpu().double(), s.rows(), s.lens_l, s.counts, d ** -0.5, window, sinks)
    got = s.cache.weights.cpu().double()
    assert torch.equal(got.isnan(), w.isnan())
    ok = ~w.isnan()
    assert ((got - w).abs()[ok] <= tol[ok]).all(), ((got - w).abs() / tol)[ok].max()
    s.cache.check()


def test_weigh_nan_keys_and_rows_that_add_nothing():
    # a NaN key at tokens that no row, or only rows of lse -inf, see: nothing is added there
    s = Setup([100], [40], heads=1, d=64, page=32)
    p, o = int(s.table_h[0, 99 // 32]), 99 % 32
    q = s.queries(2, BF16)
    _, lse = s.cache.attend(q.cuda(), s.table, s.lens, s.cu)
    lse[39] = -math.inf                                         # the one query that sees token 99
    s.cache.k_scales[p, 0, o, 1] = 255
    s.cache.weigh(q.cuda(), lse, s.table, s.lens, s.cu)
    assert s.cache.weights[p, 0, o] == 0
    total = torch.nan_to_num(s.cache.weights).sum().item()
    assert abs(total - 78) < 1e-3 * 78


@pytest.mark.parametrize("kind", ["distinct", "few", "equal"])
def test_evict_more_than_the_registers_hold(kind):
    s = Setup([70001, 40000], [1, 1], heads=1, d=64, page=1024, extra=60, seed=9)
    g = torch.Generator().manual_seed(5)

    def weights(q, n):
        if kind == "distinct":
            return torch.rand(1, n, generator=g) + 1e-3
        if kind == "few":
            return (torch.rand(1, n, generator=g) ** 8 * 8).round() / 4
        return torch.full((1, n), 0.25)
    check_evict(s, weights, 20001, 7, 100)


def test_evict_all_kept_or_none_competes():
    # the border of keys in every position: all equal, one above, budget of sinks and recent alone
    s = Setup([300, 65, 64], [1] * 3, heads=2, d=64, extra=60, seed=2)

    def weights(q, n):
        w = torch.full((2, n), 0.5)
        w[1, n // 2] = 2.0
        return w
    for budget, sinks, recent in ((64, 0, 0), (64, 32, 32), (64, 31, 32), (1, 1, 0), (1, 0, 1)):
        check_evict(s, weights, budget, sinks, recent)


def test_decode_example():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import kv4_decode
    rounding, _, lens, ratio = kv4_decode.run(requests=3, prompt=700, budget=256, steps=70)
    # probabilities and the output are rounded to bf16, half a step each; the rest is fp32 on both sides, over 350 tokens
    assert rounding <= ref.half_step(BF16) + 2e-4
    assert all(256 <= n < 256 + 64 for n in lens) and min(ratio) > 1.2
