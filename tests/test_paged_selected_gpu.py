"""Bounds of the cache's pages, the selection of pages and attention over them (fa_page_bounds,
fa_select_pages, fa_fwd_paged_selected) against the fp64 reference.

Bounds and selections are compared exactly: minima and maxima of bf16 are bf16, and the selection is
that of exact scores.  Attention has the tolerances of the paged attention (test_paged_gpu.py)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import exact_io_aware_fwd_gb300 as fa
from oracle.serving import page_bounds, page_scores, select_pages
from test_paged_gpu import Cache, _built, cumulative, f64, i32  # noqa: F401
from test_paged_tree_gpu import check

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16

HEADS = [(1, 1, 64, 16), (8, 2, 128, 64), (6, 2, 64, 32), (32, 1, 128, 128), (12, 4, 128, 16), (40, 2, 64, 16)]
by_heads = pytest.mark.parametrize("heads", HEADS, ids=lambda h: "H%dkv%dd%dpage%d" % h)


def bounds_of(cache, b):
    return page_bounds(cache.keys(b)[0], cache.page)


# ------------------------------------------------------------------------------------------ bounds
@by_heads
@pytest.mark.parametrize("nq,lens", [([1], [1]), ([1, 1, 1, 1], [16, 17, 128, 129]), ([5, 0, 33, 200], [5, 40, 300, 200]),
                                     ([2, 1], [0, 1]), ([70], [50]), ([130, 128], [129, 1000])], ids=str)
def test_bounds(nq, lens, heads):
    H, Hkv, d, page = heads
    cache = Cache(lens, Hkv, d, page, sum(lens) + d)
    kc, _, table, kv = cache.dev()
    old = torch.full((kc.shape[0], Hkv, 2, d), 9.0, dtype=BF16, device=DEV)
    for total in (None, sum(nq)):
        got = old.clone()
        assert fa.fa_page_bounds(kc, table, kv, got, cu_seqlens=i32(cumulative(nq)), total=total) is not None
        assert fa.fa_get_error() == fa.FA_OK
        ref = f64(old)
        for b, n in enumerate(lens):
            if n == 0 or nq[b] == 0:
                continue
            lo, hi = bounds_of(cache, b)
            for i in range(max(n - nq[b], 0) // page, -(-n // page)):
                ref[cache.table[b, i], :, 0], ref[cache.table[b, i], :, 1] = lo[:, i], hi[:, i]
        assert np.array_equal(f64(got), ref)


def test_bounds_of_single_tokens_without_offsets_and_odd_keys():
    cache = Cache([40, 7], 2, 64, 16, 1)
    cache.k[cache.table[1, 0], 0, 3, 5] = float("nan")
    cache.k[cache.table[1, 0], 0, 4, 6] = float("inf")
    cache.k[cache.table[1, 0], 1, 4, 6] = float("-inf")
    kc, _, table, kv = cache.dev()
    out = torch.zeros(kc.shape[0], 2, 2, 64, dtype=BF16, device=DEV)
    fa.fa_page_bounds(kc, table, kv, out)
    page = out[cache.table[1, 0].item()]
    assert torch.all(page[0, :, 5].isnan()) and page[0, 1, 6] == float("inf") and page[1, 0, 6] == float("-inf")
    assert page.isnan().sum() == 2
    assert torch.all(out[cache.table[0, 0].item()] == 0)  # no new token there
    assert torch.any(out[cache.table[0, 2].item()] != 0)
    assert fa.fa_get_error() == fa.FA_OK


def test_bounds_out_of_range():
    """Pages outside the pool are neither read nor written, and lengths past the table are clamped."""
    cache = Cache([40], 2, 64, 16, 2)
    kc, _, table, kv = cache.dev()
    out = torch.zeros(kc.shape[0], 2, 2, 64, dtype=BF16, device=DEV)
    for tab, n in ((torch.full_like(table, 99), kv), (torch.full_like(table, -5), kv), (table, i32([1000])),
                   (table, i32([-4]))):
        out.zero_()
        fa.fa_page_bounds(kc, tab, n, out, cu_seqlens=i32([0, 40]))
        assert fa.fa_get_error() == fa.FA_ERR_INDEX
        if tab is not table or n[0] < 0:
            assert torch.all(out == 0)
    # offsets that do not ascend stay inside the call's tensors
    two = torch.cat([table, table])
    for cu in ([0, 30, 5], [50, 2, 9], [-3, 7, 1 << 30]):
        fa.fa_page_bounds(kc, two, i32([40, 40]), out, cu_seqlens=i32(cu), total=40)
    fa.fa_get_error()


def test_bounds_of_fewer_tokens_than_there_are():
    """A total below the last offset leaves pages out, which is reported; where it leaves none out the
    bounds are right."""
    cache = Cache([40, 50], 2, 64, 16, 3)
    kc, _, table, kv = cache.dev()
    cu = i32([0, 30, 60])
    want = torch.zeros(kc.shape[0], 2, 2, 64, dtype=BF16, device=DEV)
    fa.fa_page_bounds(kc, table, kv, want, cu_seqlens=cu, total=60)
    assert fa.fa_get_error() == fa.FA_OK
    for total, left_out in ((59, False), (49, False), (48, True), (30, True), (20, True), (0, True)):
        got = torch.zeros_like(want)
        fa.fa_page_bounds(kc, table, kv, got, cu_seqlens=cu, total=total)
        assert fa.fa_get_error() == (fa.FA_ERR_INDEX if left_out else fa.FA_OK), total
        assert torch.equal(got, want) != left_out
    # without a count: what the block table has room for, here 128 tokens
    got = torch.zeros_like(want)
    fa.fa_page_bounds(kc, table, kv, got, cu_seqlens=i32([0, 500, 501]))
    assert fa.fa_get_error() == fa.FA_ERR_INDEX
    for odd in ([0, 30, 5], [50, 2, 9], [-3, 7, 9]):
        fa.fa_page_bounds(kc, table, kv, got, cu_seqlens=i32(odd), total=60)
        assert fa.fa_get_error() == fa.FA_ERR_INDEX, odd


# --------------------------------------------------------------------------------------- selection
class Selection:
    """Bounds of a shuffled pool, queries, and the reference's choice."""

    def __init__(self, nq, lens, heads, seed, sigma=1.0, spread=1.0):
        self.H, self.Hkv, self.d, self.page = heads
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // self.page) for n in lens]
        order = torch.randperm(sum(need) + 2, generator=g).tolist()
        self.bounds = torch.full((sum(need) + 2, self.Hkv, 2, self.d), float("nan"), dtype=BF16)
        self.table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            for i in range(n):
                p = order.pop()
                self.table[b, i] = p
                mid = spread * torch.randn(self.Hkv, 1, self.d, generator=g)
                off = torch.randn(self.Hkv, 2, self.d, generator=g).abs() * torch.tensor([[-1.0], [1.0]])
                self.bounds[p] = (sigma * (mid + off)).to(BF16)
        self.nq, self.lens, self.cu = nq, lens, cumulative(nq)
        self.q = torch.randn(self.cu[-1], self.H, self.d, generator=g).to(BF16)

    def reference(self, top, first, last):
        out = np.full((self.cu[-1], self.Hkv, top), -1)
        for b, n in enumerate(self.nq):
            P = -(-self.lens[b] // self.page)
            box = f64(self.bounds[self.table[b, :P].long()]).transpose(2, 1, 0, 3)  # [2, Hkv, P, d]
            for i in range(n):
                t, sees = self.cu[b] + i, max(0, self.lens[b] - n + i + 1)
                have = -(-sees // self.page)
                s = page_scores(f64(self.q[t]), box[0], box[1])
                for h in range(self.Hkv):
                    pick = select_pages(s[h], have, top, first, last)
                    out[t, h, :len(pick)] = pick
        return out

    def check(self, top, first, last, **kw):
        args = dict(cu_seqlens=i32(self.cu), max_kv=max(self.lens))
        args.update(kw)
        got = fa.fa_select_pages(self.q.to(DEV), self.bounds.to(DEV), self.table.to(DEV), i32(self.lens), self.page,
                                 top, first, last, **args)
        assert fa.fa_get_error() == fa.FA_OK
        ref = self.reference(top, first, last)
        assert np.array_equal(got.cpu().numpy(), ref), np.argwhere(got.cpu().numpy() != ref)[:5]
        return got


@by_heads
@pytest.mark.parametrize("nq,lens", [([1], [1]), ([1, 1, 1], [100, 1000, 5000]), ([3, 0, 1, 5], [3, 9, 700, 4000]),
                                     ([4, 2], [2, 0]), ([17], [9000])], ids=str)
def test_select(nq, lens, heads):
    s = Selection(nq, lens, heads, sum(lens) + heads[0])
    for top, first, last in ((1, 0, 0), (2, 1, 1), (7, 2, 3), (5, 5, 0), (64, 0, 1)):
        s.check(top, first, last)


def test_select_of_one_page_more_and_less():
    """The numbers of pages at which another kernel takes over."""
    for count in (33, 256, 511, 512, 513, 1024, 1025, 4100):
        s = Selection([1, 1], [16 * count, 16 * (count // 2) + 1], (4, 2, 64, 16), count)
        for top, first, last in ((1, 0, 0), (20, 1, 2), (count - 1, 0, 1)):
            s.check(top, first, last)


def test_select_of_many_pages():
    s = Selection([1, 1], [150000, 90001], (8, 2, 64, 16), 3)
    s.check(100, 1, 4)
    s.check(2000, 0, 0)
    s.check(9000, 3, 1)


def test_select_of_equal_and_nearly_equal_pages():
    """Ties go to the lowest page; pages that float32 cannot tell apart are told apart."""
    heads = (4, 2, 128, 16)
    s = Selection([1], [16 * 900], heads, 4)
    s.bounds[:] = s.bounds[s.table[0, 0].item()].clone()  # all pages alike
    s.check(40, 1, 2)
    rng = np.random.default_rng(5)
    # large terms that cancel, and the difference in the smallest: invisible in float32
    big = torch.full((s.bounds.shape[0], 2, 2, 128), 1.0, dtype=BF16)
    s.q[:] = 1.0
    big[:, :, :, 0::4], big[:, :, :, 1::4] = 2.0 ** 20, -(2.0 ** 20)
    s.q[:, :, 1::4] = 1.0
    tiny = torch.from_numpy(rng.integers(0, 40, big.shape[0])).to(BF16) * 2.0 ** -9
    big[:, :, :, 2] = tiny[:, None, None]
    s.bounds = big
    s.check(40, 1, 2)
    s.q[:] = 0.0  # all scores are 0
    s.check(40, 1, 2)
    few = Selection([1], [16 * 300], heads, 6)
    few.bounds, few.q = big[:few.bounds.shape[0]].clone(), s.q.clone()
    few.check(17, 0, 1)  # all next to the border, ranked in shared memory
    few.bounds[:] = few.bounds[few.table[0, 0].item()].clone()
    few.check(17, 0, 1)
    few.q[:] = 0.0
    few.check(17, 0, 1)


@pytest.mark.parametrize("count", [60, 700, 1500])
@pytest.mark.parametrize("bound,rest", [(2.0 ** -5, 2.0 ** -65), (2.0 ** -133, 2.0 ** -59), (2.0 ** -130, 2.0 ** -62),
                                        (2.0 ** 100, 2.0 ** -64)])
def test_select_of_scores_a_little_apart(count, bound, rest):
    """Two pages at the border whose scores are 0 and 127 products of `rest` and `bound`, more than 2^-59
    of the largest bound times sum |q|, which is 1 here; the higher one has the higher index."""
    s = Selection([1], [16 * count], (1, 1, 128, 16), count)
    s.q[:] = rest
    s.q[:, :, 0] = 1.0
    pages = s.table[0].long()
    s.bounds[:] = 0.0
    s.bounds[:, :, :, 0] = -bound
    s.bounds[pages[3:9], :, :, 0] = bound
    s.bounds[pages[20], :, :, 0] = s.bounds[pages[50], :, :, 0] = 0.0
    s.bounds[pages[50], :, :, 1:] = bound
    got = s.check(7, 0, 0)
    assert got.flatten().tolist() == [3, 4, 5, 6, 7, 8, 50]
    s.bounds[pages[50], :, :, 1:] = 0.0
    assert s.check(7, 0, 0).flatten().tolist() == [3, 4, 5, 6, 7, 8, 20]


@pytest.mark.parametrize("count", [100, 512, 513, 700, 1100])
def test_select_of_scores_that_are_not_finite(count):
    heads = (4, 2, 64, 16)
    s = Selection([1, 2], [16 * 50, 16 * (count - 1) + 3], heads, 7)
    pages = s.table[1].long()
    s.bounds[pages[10], 0, 1, 3] = float("inf")
    s.bounds[pages[20], 1, 0, 5] = float("nan")
    s.bounds[pages[30], 1] = float("nan")
    s.bounds[pages[40], :, 0] = float("-inf")
    s.bounds[pages[50]] = 3e38
    s.check(9, 1, 2)
    s.check(3, 0, 0)
    s.q[0, 0, 0] = float("inf")
    s.check(9, 1, 2)
    # a query that is not a number: every score counts as infinity
    s.q[1, 3, 5] = float("nan")
    got = fa.fa_select_pages(s.q.to(DEV), s.bounds.to(DEV), s.table.to(DEV), i32(s.lens), 16, 6, 1, 1,
                             cu_seqlens=i32(s.cu)).cpu()
    P = -(-(s.lens[1] - 1) // 16)
    assert got[1, 1].tolist() == [0, 1, 2, 3, 4, P - 1]


@pytest.mark.parametrize("count", [60, 900, 1500, 5000])
def test_select_of_scores_near_the_largest_number(count):
    """The k-th score plus twice its error bound is not finite: 4 + 2^-6 times the largest bf16 below
    2^126 is 2^128 (1 - 2^-16), and the bound is 2^-15 of it."""
    s = Selection([1], [16 * count], (2, 1, 64, 16), count)
    s.q[:] = 0.0
    s.q[0, :, 3], s.q[0, :, 40] = 4.0, 2.0 ** -6
    s.bounds[:] = 0.0
    s.bounds[:, :, :, 3] = s.bounds[:, :, :, 40] = 1.9921875 * 2.0 ** 125
    s.check(50, 1, 2)  # all equal
    s.bounds[s.table[0, 20:40].long()] = 0.0
    s.check(50, 1, 2)


@pytest.mark.parametrize("count", [60, 700, 1500])
def test_select_of_scores_below_the_smallest_normal_number(count):
    """Products of 2^-130 have few bits left in float32, and those of 2^-150 none."""
    s = Selection([1, 2], [16 * count, 16 * count - 5], (4, 2, 64, 16), count)
    q, bounds = s.q, s.bounds
    for at, by in ((-20, -110), (-10, -130), (20, -130), (-70, -60), (-100, -100)):
        s.q, s.bounds = q * 2.0 ** at, bounds * 2.0 ** by
        s.check(30, 1, 2)


def test_select_in_a_graph_and_on_another_stream():
    s = Selection([1, 3], [3000, 9000], (8, 2, 128, 16), 8)
    args = (s.q.to(DEV), s.bounds.to(DEV), s.table.to(DEV), i32(s.lens), 16, 20, 1, 2)
    want = s.check(20, 1, 2)
    cu = i32(s.cu)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = fa.fa_select_pages(*args, cu_seqlens=cu, max_kv=9000)
    got.zero_()
    g.replay()
    assert torch.equal(got, want)
    args[3].copy_(i32([100, 5000]))  # other lengths in the same graph
    g.replay()
    assert torch.equal(got, fa.fa_select_pages(*args, cu_seqlens=cu))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = fa.fa_select_pages(*args, cu_seqlens=cu, stream=side)
    side.synchronize()
    assert torch.equal(other, got) and fa.fa_get_error() == fa.FA_OK


def test_select_out_of_range():
    s = Selection([1, 1], [500, 900], (4, 2, 64, 16), 9)
    q, bounds, table = s.q.to(DEV), s.bounds.to(DEV), s.table.to(DEV)
    # pages outside the pool score 0, like bounds of zeros
    wild = table.clone()
    wild[1, 7], wild[1, 9] = 9999, -3
    got = fa.fa_select_pages(q, bounds, wild, i32(s.lens), 16, 12)
    assert fa.fa_get_error() == fa.FA_ERR_INDEX
    s.bounds[s.table[1, 7].item()] = 0
    s.bounds[s.table[1, 9].item()] = 0
    assert np.array_equal(got.cpu().numpy(), s.reference(12, 1, 1))
    fa.fa_select_pages(q, bounds, table, i32([500, 1 << 30]), 16, 12)
    assert fa.fa_get_error() == fa.FA_ERR_INDEX
    # tokens behind the last sequence keep what they have; offsets that do not ascend stay inside
    out = torch.full((2, 2, 12), 55, dtype=torch.int32, device=DEV)
    fa.fa_select_pages(q, bounds, table, i32(s.lens), 16, 12, cu_seqlens=i32([0, 1, 1]), out=out)
    assert torch.all(out[1] == 55) and torch.all(out[0, :, 0] == 0)
    for cu in ([2, 1, 0], [-4, 9, 1]):
        fa.fa_select_pages(q, bounds, table, i32(s.lens), 16, 12, cu_seqlens=i32(cu))
    fa.fa_get_error()


def test_refusals():
    s = Selection([1], [500], (4, 2, 64, 16), 10)
    q, bounds, table, lens = s.q.to(DEV), s.bounds.to(DEV), s.table.to(DEV), i32(s.lens)
    for bad in (dict(top=0), dict(top=2, first=2, last=1), dict(top=4, first=-1), dict(page_size=24),
                dict(q=q.float()), dict(q=q[:, :3].contiguous()), dict(bounds=bounds[:, :, :1].contiguous()),
                dict(lens=lens.long()), dict(out=torch.zeros(1, 2, 3, dtype=torch.int32, device=DEV)),
                dict(workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))):
        a = dict(q=q, bounds=bounds, table=table, lens=lens, page_size=16, top=4, first=1, last=1, out=None,
                 workspace=None)
        a.update(bad)
        with pytest.raises((ValueError, fa.FAError)):
            fa.fa_select_pages(a["q"], a["bounds"], a["table"], a["lens"], a["page_size"], a["top"], a["first"],
                               a["last"], out=a["out"], workspace=a["workspace"])


# --------------------------------------------------------------------------- attention over them
def run(nq, lens, heads, top, seed, shuffle=False, sigma=1.0, holes=0.0, **kw):
    H, Hkv, d, page = heads
    rng = np.random.default_rng(seed)
    cache = Cache(lens, Hkv, d, page, seed, sigma)
    cu = cumulative(nq)
    q = (sigma * torch.randn(cu[-1], H, d, generator=torch.Generator().manual_seed(seed + 1))).to(BF16)
    pages = np.full((cu[-1], Hkv, top), -1, dtype=np.int32)
    per = []
    for b, n in enumerate(nq):
        P = -(-lens[b] // page)
        seen = np.zeros((n, Hkv, lens[b]), dtype=bool)
        for i in range(n):
            for h in range(Hkv):
                pick = np.sort(rng.permutation(P)[:top])
                if shuffle:
                    rng.shuffle(pick)
                keep = rng.random(len(pick)) >= holes
                pages[cu[b] + i, h, :len(pick)] = np.where(keep, pick, -1 - rng.integers(0, 5))
                for p in pick[keep]:
                    seen[i, h, p * page:(p + 1) * page] = True
            seen[i, :, max(0, lens[b] - n + i + 1):] = False
        per.append((*cache.keys(b), seen))
    args = (q.to(DEV), *cache.dev(), torch.from_numpy(pages).to(DEV))
    out, lse = fa.fa_fwd_paged_selected(*args, cu_seqlens=i32(cu), **kw)
    assert fa.fa_get_error() == fa.FA_OK
    check(out, lse, q, cu, per, d ** -0.5)
    return args, cu, out, lse


@by_heads
@pytest.mark.parametrize("nq,lens,top", [([1], [1], 1), ([1, 1, 1], [100, 900, 2000], 5), ([3, 0, 1, 4], [3, 9, 700, 1500], 9),
                                         ([4, 2], [2, 0], 2), ([1] * 12, [600 + 37 * i for i in range(12)], 20),
                                         ([1], [3000], 130)], ids=str)
def test_selected(nq, lens, top, heads):
    run(nq, lens, heads, top, sum(lens) + top)


@pytest.mark.parametrize("heads", [(8, 2, 128, 64), (20, 1, 64, 16)], ids=lambda h: "H%dkv%dd%dpage%d" % h)
def test_selected_in_any_order_and_with_holes(heads):
    for seed, nq, lens in ((1, [2, 1], [1500, 800]), (2, [1] * 40, [300 + 11 * i for i in range(40)])):
        run(nq, lens, heads, 12, seed, shuffle=True, holes=0.3)
        run(nq, lens, heads, 12, seed, shuffle=True, holes=1.0)  # nothing is listed: no result
    run([1], [900], heads, 12, 3, sigma=6.0)


def test_a_page_listed_twice_counts_twice():
    args, cu, out, lse = run([1], [64], (4, 2, 64, 16), 2, 5)
    twice = args[5].repeat(1, 1, 2).contiguous()
    o2, l2 = fa.fa_fwd_paged_selected(*args[:5], twice, cu_seqlens=i32(cu))
    assert torch.allclose(l2, lse + float(np.log(2.0)), atol=2.0 ** -12)
    most = float(args[2].nan_to_num(0).abs().max())  # sum p|v| and |O| are at most this
    assert float((o2.float() - out.float()).abs().max()) <= 2 * (2.0 ** -7 + 2.0 ** -14) * most


def test_all_pages_are_plain_attention():
    lens, heads = [700, 1900, 40], (8, 2, 128, 64)
    P = -(-max(lens) // 64)
    cache = Cache(lens, 2, 128, 64, 6)
    q = torch.randn(3, 8, 128, generator=torch.Generator().manual_seed(7)).to(BF16).to(DEV)
    pages = torch.arange(P, dtype=torch.int32, device=DEV).expand(3, 2, P).contiguous()
    o, lse = fa.fa_fwd_paged_selected(q, *cache.dev(), pages)  # entries behind a sequence's end have no keys
    ref, ref_lse = fa.fa_fwd_paged(q, *cache.dev())
    assert torch.allclose(lse, ref_lse, atol=2.0 ** -11)
    most = float(cache.v.nan_to_num(0).abs().max())  # sum p|v| and |O| are at most this
    assert float((o.float() - ref.float()).abs().max()) <= 2 * (2.0 ** -7 + 2.0 ** -14) * most
    assert fa.fa_get_error() == fa.FA_OK


def test_selected_repeats_in_a_graph_and_on_another_stream():
    args, cu, out, lse = run([1, 2, 1, 1], [5000, 900, 3000, 10], (8, 2, 128, 16), 60, 8)
    g = torch.cuda.CUDAGraph()
    offsets = i32(cu)
    with torch.cuda.graph(g):
        o2, l2 = fa.fa_fwd_paged_selected(*args, cu_seqlens=offsets)
    o2.zero_()
    g.replay()
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o3, l3 = fa.fa_fwd_paged_selected(*args, cu_seqlens=offsets, stream=side)
    side.synchronize()
    assert torch.equal(o3, out) and torch.equal(l3, lse)


def test_selected_out_of_range():
    """Pages outside the pool read as zeros; entries behind the end have no keys; tokens behind the last
    sequence keep their rows."""
    cache = Cache([100, 60], 2, 64, 16, 9)
    q = torch.randn(2, 4, 64).to(BF16).to(DEV)
    kc, vc, table, lens = cache.dev()
    pages = torch.tensor([[0, 6, 7, 1 << 30], [3, 4, 100, -(1 << 31)]], dtype=torch.int32, device=DEV)
    pages = pages[:, None].repeat(1, 2, 1)
    o, lse = fa.fa_fwd_paged_selected(q, kc, vc, table, lens, pages)
    assert fa.fa_get_error() == fa.FA_OK and torch.all(lse.isfinite())
    wild = table.clone()
    wild[0, 0], wild[0, 6] = 1000, -9
    o, lse = fa.fa_fwd_paged_selected(q, kc, vc, wild, lens, pages)
    assert fa.fa_get_error() == fa.FA_ERR_INDEX
    assert torch.all(o[0] == 0) and torch.allclose(lse[:, 0], torch.full((4,), float(np.log(20.0)), device=DEV))
    for top in (4, 40):  # whole segments, and parts that are joined
        long = torch.cat([pages, torch.full((2, 2, 200), 2, dtype=torch.int32, device=DEV)], 2)[:, :, :top * 4].contiguous()
        o, lse = torch.full_like(q, 5), torch.full((4, 2), 5.0, device=DEV)
        fa.fa_fwd_paged_selected(q, kc, vc, table, lens, long, cu_seqlens=i32([0, 1, 1]), out=o, lse=lse)
        assert torch.all(o[1] == 5) and torch.all(lse[:, 1] == 5) and torch.all(o[0] != 5)
    fa.fa_fwd_paged_selected(q, kc, vc, table, i32([100, 5000]), pages)
    assert fa.fa_get_error() == fa.FA_ERR_INDEX
    for cu in ([2, 1, 0], [-4, 9, 1]):
        fa.fa_fwd_paged_selected(q, kc, vc, table, lens, pages, cu_seqlens=i32(cu))
    fa.fa_get_error()


# ------------------------------------------------------------------------------- as it is used
def test_decoding_steps_over_selected_pages():
    """Append, renew the bounds, select, attend, step after step; with as many pages as there are the
    result is plain attention's, with fewer that of the reference's choice."""
    H, Hkv, d, page, top = 8, 2, 64, 16, 5
    lens = [150, 31, 200]
    g = torch.Generator().manual_seed(11)
    cache = Cache([n + 40 for n in lens], Hkv, d, page, 12)
    kc, vc, table, _ = cache.dev()
    bounds = torch.zeros(kc.shape[0], Hkv, 2, d, dtype=BF16, device=DEV)
    fa.fa_page_bounds(kc, table, i32(lens), bounds, cu_seqlens=i32(cumulative(lens)))
    rope = fa.fa_rope_table(512, d, device=DEV)
    for step in range(20):
        lens = [n + 1 for n in lens]
        kv = i32(lens)
        x = torch.randn(3, H + 2 * Hkv, d, generator=g).to(BF16).to(DEV)
        q, k, v = x.split([H, Hkv, Hkv], dim=1)
        q = fa.fa_kv_append(q, k, v, kc, vc, table, kv, table=rope)
        fa.fa_page_bounds(kc, table, kv, bounds)
        pages = fa.fa_select_pages(q, bounds, table, kv, page, top, first=1, last=1, max_kv=max(lens))
        o, lse = fa.fa_fwd_paged_selected(q, kc, vc, table, kv, pages)
        assert fa.fa_get_error() == fa.FA_OK
        if step % 6:
            continue
        per = []
        for b, n in enumerate(lens):
            pool, vals = f64(kc), f64(vc)
            at = [(cache.table[b, j // page].item(), j % page) for j in range(n)]
            K = np.stack([pool[p, :, r] for p, r in at], 1)
            V = np.stack([vals[p, :, r] for p, r in at], 1)
            lo, hi = page_bounds(K, page)
            s = page_scores(f64(q[b]), lo, hi)
            seen = np.zeros((1, Hkv, n), bool)
            for h in range(Hkv):
                pick = select_pages(s[h], -(-n // page), top, 1, 1)
                assert pages[b, h].tolist() == pick.tolist() + [-1] * (top - len(pick))
                for p in pick:
                    seen[0, h, p * page:(p + 1) * page] = True
            per.append((K, V, seen))
        check(o, lse, q, [0, 1, 2, 3], per, d ** -0.5)
