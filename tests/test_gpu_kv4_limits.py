"""GPU tests of the 4-bit KV cache at the ends of its range, against the 64-bit implementations of
tests/kv4_reference.py: the largest values that the format holds,
hints that say too little, too much or nothing."""
from __future__ import annotations

import math

import pytest
import torch

import kv4_reference as ref
from test_gpu_kv4 import BF16, FP16, Setup, check_attend, check_evict

pytestmark = pytest.mark.gpu


# queries of the two sequences: with a group of 4, 4, 20, 52, 100 and 300 rows of the first
@pytest.mark.parametrize("count", [1, 5, 13, 25, 75])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attend_largest_values(d, count):
    # Base-2 scores: 0 for the first 32 tokens, 6 for one 128 tokens on (which the same wave meets later), -192 for
    # the others.  That one holds the format's largest values: times 2^6 they leave 32 bits, times their
    # share of the softmax, 2/3, they do not.
    s = Setup([300, 700], [count, 1], heads=1, d=d, page=32, seed=d)
    n = len(s.k)
    k, v = torch.full((n, 1, d), 0.0), s.v.float()
    for first, length in ((0, 300), (300, 700)):
        k[first:first + length, 0, 0] = -192.0
        k[first:first + 32, 0, 0] = 0.0
        k[first + 130, 0, 0] = 6.0
        v[first + 130, 0] = 6 * 2.0 ** 125 * torch.where(torch.arange(d) % 3 == 0, -1.0, 1.0)
    s.cache.append(k.cuda(), v.cuda(), s.table, s.lens, s.fill_cu)
    q = torch.zeros(s.total, 4, d, dtype=BF16)
    q[:, :, 0] = 1.0
    scale = math.log(2)
    out, lse = s.cache.attend(q.cuda(), s.table, s.lens, s.cu, max_q=count, scale=scale)
    eo, to, el, tl = ref.attend(ref.Cache(s.cache), q.double(), s.rows(), s.lens_l, s.counts, scale, None, 0, BF16)
    assert out.isfinite().all()
    assert ((out.cpu().double() - eo).abs() <= to).all()
    assert ((lse.cpu().double() - el).abs() <= tl).all()


@pytest.mark.parametrize("max_len", [1, 129, 300])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_evict_hint_that_says_too_little(d, max_len):
    # a move workgroup takes several turns, the last of them short
    s = Setup([0, 1, 700, 523, 900], [1] * 5, heads=2, d=d, page=32, extra=100, seed=d)
    check_evict(s, lambda q, n: torch.rand(2, n, generator=s.g), 523, 4, 100, max_len=max_len)


# queries of the longest sequence: with a group of 4, 4, 20, 52, 100 and 300 rows
COUNTS = [(1, 1, 1, 0), (5, 2, 1, 0), (13, 1, 5, 0), (25, 12, 5, 2), (75, 30, 3, 0)]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attend_row_tiles_by_hint(d, dtype, counts):
    # a tile is as long as the longest sequence's rows, or as the mean's where nobody says
    s = Setup([401, 130, 5, 17], counts, heads=2, d=d, page=32, seed=d + counts[0])
    for kw in ({"max_q": counts[0]}, {"max_q": 10 ** 6}, {}):
        check_attend(s, 8, dtype, window=50, sinks=7, **kw)
        check_attend(s, 8, dtype, **kw)
    s.cache.check()


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("d,dtype", [(64, FP16), (128, BF16), (256, FP16)])
def test_attend_nan_in_row_tiles_by_hint(d, dtype, counts):
    s = Setup([401, 130, 5, 17], counts, heads=2, d=d, page=32, seed=counts[0])
    for q, j, h in ((0, 398, 0), (0, 20, 1), (1, 129, 1), (1, 3, 0), (2, 0, 1), (0, 352, 1)):
        s.cache.v_scales[int(s.table_h[q, j // 32]), h, j % (d // 32), j % 32] = 255
    for q, j in ((0, 380), (1, 127)):
        s.cache.k_scales[int(s.table_h[q, j // 32]), 1, j % 32, 0] = 255
    for window, sinks in ((None, 0), (40, 2)):
        check_attend(s, 4, dtype, window=window, sinks=sinks, max_q=counts[0])


def test_attend_one_long_sequence_among_many():
    # rows past the launch's tiles are taken in turn: 63 single queries and one sequence of 500
    s = Setup([40] * 63 + [500], [1] * 63 + [500], heads=8, d=64, page=64)
    check_attend(s, 8, BF16)
    check_attend(s, 32, BF16, window=30, sinks=3)


def test_check_waits_for_other_streams():
    s = Setup([20, 20], [1, 1], heads=1, d=64)
    x = torch.zeros(2, 1, 64, device="cuda", dtype=BF16)
    bad = torch.full((2, 2), -1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)           # some milliseconds at least, of which check() knows nothing
        s.cache.append(x, x, bad, s.lens)
    with pytest.raises(ValueError, match="page"):
        s.cache.check()
    s.cache.check()                             # cleared


@pytest.mark.parametrize("rows,first", [(600, 0), (600, 300), (1, 0), (37, 36)])
@pytest.mark.parametrize("d,counts", [(64, (1, 1)), (128, (20, 3)), (256, (70, 2))])
def test_attend_padded_batch(d, counts, rows, first):
    # `first` rows before the sequences and rows - first behind them, as a graph's fixed number of rows has
    s = Setup([90, 400], counts, heads=2, d=d, page=32, seed=d)
    q = torch.randn(s.total + rows, 6, d, generator=s.g).to(BF16).cuda()
    mine = slice(first, first + s.total)
    want = s.cache.attend(q[mine], s.table, s.lens, s.cu, max_q=max(counts))
    torch.empty(q.shape, dtype=q.dtype, device="cuda").fill_(float("nan"))       # what the results' memory may have held
    out, lse = s.cache.attend(q, s.table, s.lens, s.cu + first, max_q=max(counts))
    assert torch.equal(out[mine], want[0]) and torch.equal(lse[mine], want[1])
    for part in (slice(0, first), slice(first + s.total, None)):
        assert (out[part] == 0).all() and (lse[part] == -math.inf).all()
    s.cache.check()


@pytest.mark.parametrize("counts,group", [((1,) * 12, 8), ((5,) * 12, 8), ((40,) * 12, 3)])
@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, FP16), (256, BF16)])
def test_weigh_shared_pages(d, dtype, counts, group):
    # twelve sequences of one prefix: what its pages get is the sum over all of them
    s = Setup([300, *range(200, 310, 10)], counts, heads=2, d=d, page=32, seed=d)
    for q in range(1, 12):
        s.table_h[q, :6] = s.table_h[0, :6]
    s.table = s.table_h.cuda()
    q = s.queries(2 * group, dtype)
    for mask in ({"window": None, "sinks": 0}, {"window": 150, "sinks": 40}):
        _, lse = s.cache.attend(q.cuda(), s.table, s.lens, s.cu, **mask)
        s.cache.weights.nan_to_num_(0.25)
        r = ref.Cache(s.cache)
        s.cache.weigh(q.cuda(), lse, s.table, s.lens, s.cu, max_q=max(counts), **mask)
        w, tol = ref.weigh(r, q.double(), lse.cpu().double(), s.rows(), s.lens_l, s.counts, d ** -0.5, mask["window"], mask["sinks"])
        assert ((s.cache.weights.cpu().double() - w).abs() <= tol + 12 * ref.U32 * w.abs()).all()


@pytest.mark.parametrize("counts", [(1, 1), (7, 3), (40, 90)])
@pytest.mark.parametrize("d,dtype", [(64, FP16), (128, BF16), (256, BF16)])
@pytest.mark.parametrize("scale", [0.1, -0.1])
def test_queries_that_are_not_finite(d, dtype, counts, scale):
    s = Setup([90, 130], counts, heads=2, d=d, page=32, seed=d)
    q = s.queries(4, dtype)
    q[0, 0, 3], q[1, 1, d - 1], q[-1, 2, 17], q[-1, 3, d // 2] = math.inf, -math.inf, math.nan, math.inf
    out, lse = s.cache.attend(q.cuda(), s.table, s.lens, s.cu, scale=scale)
    eo, to, el, tl = ref.attend(ref.Cache(s.cache), q.double(), s.rows(), s.lens_l, s.counts, scale, None, 0, dtype)
    out, lse = out.cpu().double(), lse.cpu().double()
    assert el.isnan().any() and torch.equal(lse.isnan(), el.isnan()) and torch.equal(out.isnan(), eo.isnan())
    assert ((out - eo).abs() <= to)[~eo.isnan()].all() and ((lse - el).abs() <= tl)[~el.isnan()].all()


@pytest.mark.parametrize("counts", [(1, 1), (40, 90)])
def test_scale_of_0_leaves_the_queries_out(counts):
    # every token that a query sees counts alike, whatever the query holds
    s = Setup([90, 130], counts, heads=2, d=64, page=32)
    q = s.queries(4, BF16)
    q[0, 0, 3], q[-1, 2, 17] = math.inf, math.nan
    out, lse = check_attend(s, 4, BF16, scale=0.0, q=q.nan_to_num(0.0, 1.0, 1.0))[1:]
    got = s.cache.attend(q.cuda(), s.table, s.lens, s.cu, scale=0.0)
    assert torch.equal(got[0].cpu().double(), out) and torch.equal(got[1].cpu().double(), lse)


def test_results_carry_no_gradient():
    s = Setup([20, 9], [1, 1], heads=1, d=64)
    q = s.queries(2, BF16).cuda().requires_grad_()
    k = torch.randn(2, 1, 64, generator=s.g).cuda().requires_grad_()
    s.cache.append(k, k, s.table, s.lens)
    out, lse = s.cache.attend(q, s.table, s.lens)
    assert not out.requires_grad and not lse.requires_grad
    want = s.cache.attend(q.detach(), s.table, s.lens)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, FP16), (256, BF16)])
def test_weigh_without_max_q(d, dtype):
    # sequences of 4, 8, 16, 20 and 160 rows: the mean is below 16, and two kernels share them
    counts = [1] * 30 + [2, 4, 5, 40, 0, 3]
    s = Setup([30] * 30 + [90, 64, 70, 300, 5, 2], counts, heads=2, d=d, page=32, seed=d)
    assert s.total * 4 <= 16 * len(counts)
    q = s.queries(8, dtype)
    for mask in ({"window": None, "sinks": 0}, {"window": 33, "sinks": 5}):
        _, lse = s.cache.attend(q.cuda(), s.table, s.lens, s.cu, **mask)
        r = ref.Cache(s.cache)
        s.cache.weigh(q.cuda(), lse, s.table, s.lens, s.cu, **mask)
        w, tol = ref.weigh(r, q.double(), lse.cpu().double(), s.rows(), s.lens_l, s.counts, d ** -0.5, mask["window"], mask["sinks"])
        got = s.cache.weights.cpu().double()
        assert torch.equal(got.isnan(), w.isnan())
        ok = ~w.isnan()
        assert ((got - w).abs()[ok] <= tol[ok]).all()
