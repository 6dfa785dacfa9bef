"""The paged cache (fa_kv_append), attention over it (fa_fwd_paged) and attention behind shared
prefixes (fa_fwd_shared_prefix) against the fp64 reference.

Tolerances.  P is rounded to bf16 (half a step, 2^-8 of each weight) before P V and O once more, so
|O - ref| <= 2^-8 (sum p|v|) + 2^-8 |ref|; float32 sums and exponentials (2^-22 each, relative to
score magnitudes of at most a few tens) stay inside 2^-14 sum p|v|.  LSE: the scores' float32
dot products are off by at most 2^-24 (d + 16) scale sum|q k|, the exponentials and the logarithm
by 2^-20."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import exact_io_aware_fwd_gb300 as fa
from oracle.serving import attend, norm_rope, paged_keys

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    fa.build()
    fa.load_library()


def f64(t):
    return t.detach().double().cpu().numpy()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def cumulative(n):
    return [0] + np.cumsum(n).tolist()


class Cache:
    """A shuffled pool whose unused rows, and rows past a length, hold NaN."""

    def __init__(self, lens, Hkv, d, page, seed, sigma=1.0, extra=3):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lens]
        order = torch.randperm(sum(need) + extra, generator=g).tolist()
        width = max(1, max(need, default=1))
        self.k, self.v = (torch.full((sum(need) + extra, Hkv, page, d), float("nan"), dtype=BF16)
                          for _ in range(2))
        self.table = torch.full((len(lens), width), -1, dtype=torch.int32)
        for b, n in enumerate(lens):
            for i in range(need[b]):
                p = order.pop()
                m = min(page, n - i * page)
                self.table[b, i] = p
                self.k[p, :, :m] = (sigma * torch.randn(Hkv, m, d, generator=g)).to(BF16)
                self.v[p, :, :m] = torch.randn(Hkv, m, d, generator=g).to(BF16)
        self.lens, self.page = list(lens), page
        self.np = (self.k.float().numpy(), self.v.float().numpy())

    def dev(self):
        return self.k.to(DEV), self.v.to(DEV), self.table.to(DEV), i32(self.lens)

    def keys(self, b):
        return [paged_keys(c, self.table[b].numpy(), self.lens[b]) for c in self.np]


def check(out, lse, q, cu, per_seq, scale, label=""):
    """per_seq: (K, V, limits) of each sequence."""
    out, lse, q = f64(out), f64(lse), f64(q)
    d = q.shape[-1]
    for b, (K, V, limits) in enumerate(per_seq):
        a, e = cu[b], cu[b + 1]
        O, L, A, size = attend(q[a:e], K, V, scale, limits)
        excess = np.abs(out[a:e] - O) - ((2.0 ** -8 + 2.0 ** -14) * A + 2.0 ** -8 * np.abs(O))
        assert np.all(excess <= 1e-30), (label, b, float(excess.max()))
        got = lse[:, a:e].T
        assert np.array_equal(np.isfinite(got), np.isfinite(L)), (label, b)
        fin = np.isfinite(L)
        assert np.all(got[~fin] == L[~fin])
        bound = 2.0 ** -24 * (d + 16) * size + 2.0 ** -20 * (1 + np.abs(np.where(fin, L, 0)))
        assert np.all(np.abs(got[fin] - L[fin]) <= bound[fin]), (label, b)


def limits_of(n, length, causal):
    return [length - n + i + 1 if causal else length for i in range(n)]


def run_paged(case_q, lens, H, Hkv, d, page, causal, seed, sigma=1.0, scale=None, **kw):
    cache = Cache(lens, Hkv, d, page, seed, sigma)
    cu = cumulative(case_q)
    g = torch.Generator().manual_seed(seed + 1)
    q = (sigma * torch.randn(cu[-1], H, d, generator=g)).to(BF16)
    args = dict(cu_seqlens=i32(cu), max_q=max(max(case_q), 1), max_kv=max(lens), causal=causal, scale=scale)
    args.update(kw)
    out, lse = fa.fa_fwd_paged(q.to(DEV), *cache.dev(), **args)
    assert fa.fa_get_error() == fa.FA_OK
    per = [(*cache.keys(b), limits_of(case_q[b], lens[b], causal)) for b in range(len(lens))]
    check(out, lse, q, cu, per, d ** -0.5 if scale is None else scale, str((case_q, lens, H, Hkv, d, page)))
    return cache, q, out, lse


LENGTHS = [
    ([1], [1]),
    ([1], [17]),
    ([1, 1, 1, 1, 1, 1, 1, 1], [0, 1, 15, 16, 63, 64, 65, 129]),
    ([1, 1, 1], [511, 512, 513]),
    ([1, 1, 1, 1], [5000, 3, 700, 1]),         # split over the keys, next to short ones
    ([3, 0, 1, 5, 2], [40, 9, 1, 5, 300]),     # several new tokens, none, as many as keys
    ([4, 2], [2, 0]),                          # more new tokens than keys: rows without a key
]


@pytest.mark.parametrize("heads", [(1, 1, 64, 16), (8, 2, 128, 64), (6, 2, 64, 32), (32, 1, 128, 128),
                                   (12, 12, 128, 16), (5, 1, 64, 128)],
                         ids=lambda h: "H%dkv%dd%dpage%d" % h)
@pytest.mark.parametrize("causal", [False, True], ids=["all", "causal"])
@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda x: "-".join(map(str, x[1])))
def test_paged(lengths, causal, heads):
    H, Hkv, d, page = heads
    run_paged(*lengths, H, Hkv, d, page, causal, seed=sum(lengths[1]) + H)


@pytest.mark.parametrize("nq,lens", [([40, 1, 130], [900, 31, 130]), ([257, 64], [1500, 64]), ([300], [300])])
@pytest.mark.parametrize("heads", [(8, 2, 128, 64), (3, 1, 64, 16), (4, 4, 128, 32)],
                         ids=lambda h: "H%dkv%dd%dpage%d" % h)
def test_paged_chunks(nq, lens, heads):
    """Chunks of prompts, many rows a head, with the causal mask ending inside tiles."""
    H, Hkv, d, page = heads
    for causal in (True, False):
        for max_kv in (max(lens), 2000):  # the second: not short enough for whole segments a CTA
            run_paged(nq, lens, H, Hkv, d, page, causal, seed=len(nq) + H, max_kv=max_kv)


@pytest.mark.parametrize("d", [64, 128])
def test_paged_batches_that_mix_single_tokens_and_a_chunk(d):
    rng = np.random.default_rng(1)
    for chunk in (512, 2048):
        nq, lens = [1] * 63, rng.integers(1, 1500, 64).tolist()
        nq.insert(20, chunk)
        lens[20] = chunk + 300
        run_paged(nq, lens, 8, 2, d, 64, True, seed=7)


@pytest.mark.parametrize("d", [64, 128])
def test_paged_long_chunks(d):
    run_paged([3000], [5000], 4, 2, d, 64, True, seed=5)
    run_paged([4096, 1], [4096, 3000], 2, 1, d, 16, True, seed=6)


@pytest.mark.parametrize("max_kv", [400, 2000], ids=["whole", "tiles"])
@pytest.mark.parametrize("heads", [(1, 1, 64, 16), (4, 1, 128, 64), (4, 2, 128, 32)],
                         ids=lambda h: "H%dkv%dd%dpage%d" % h)
def test_paged_chunks_longer_than_their_keys(heads, max_kv):
    """Hundreds of tokens that see no key: a first query tile without keys next to a second with some."""
    for causal in (True, False):
        run_paged([300, 5, 700], [50, 400, 300], *heads, causal, seed=3, max_kv=max_kv)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,n,max_kv", [(3, 900, 2000), (3, 900, 900), (3, 9000, 9000), (40, 900, 2000), (300, 3000, 3000)],
                         ids=["few rows", "whole", "long", "one tile", "many rows"])
def test_paged_hidden_key_that_is_not_finite(nq, n, max_kv, d):
    """The last key is hidden from all tokens but the last: whatever it holds, their bits stay."""
    cache = Cache([n], 1, d, 16, seed=4)
    k, v, table, lens = cache.dev()
    q = torch.randn(nq, 2, d, device=DEV).to(BF16)
    kw = dict(cu_seqlens=i32([0, nq]), max_q=nq, max_kv=max_kv, causal=True)
    want = fa.fa_fwd_paged(q, k, v, table, lens, **kw)
    page = int(cache.table[0, (n - 1) // 16])
    for value in (float("inf"), float("-inf"), float("nan")):
        k[page, :, (n - 1) % 16] = value
        got = fa.fa_fwd_paged(q, k, v, table, lens, **kw)
        assert torch.equal(got[0][:-1], want[0][:-1]) and torch.equal(got[1][:, :-1], want[1][:, :-1])
    assert torch.isnan(got[0][-1]).all()
    assert fa.fa_get_error() == fa.FA_OK


def test_paged_without_pages():
    """Block tables of no columns: no keys, zeros and -inf."""
    k = torch.zeros(2, 1, 16, 64, dtype=BF16, device=DEV)
    table, none = torch.empty(3, 0, dtype=torch.int32, device=DEV), i32([0, 0, 0])
    q = torch.randn(3, 4, 64, device=DEV).to(BF16)
    many = torch.randn(120, 4, 64, device=DEV).to(BF16)
    for out, lse in (fa.fa_fwd_paged(q, k, k, table, none),
                     fa.fa_fwd_shared_prefix(q, k, k, table, none, table[:1].contiguous(), none[:1].contiguous(), i32([0, 3])),
                     fa.fa_fwd_paged(many, k, k, table, none, cu_seqlens=i32([0, 40, 80, 120]), max_kv=3000)):
        assert not out.any() and torch.isneginf(lse).all()
    assert fa.fa_get_error() == fa.FA_OK


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True], ids=["all", "causal"])
def test_paged_one_query_tile(causal, d):
    """17 to 128 rows a key/value head (both tile slots on one query tile): no, one, two, three, many
    key tiles of a row, whole or split, and tokens without a key."""
    lens = [0, 1, 100, 128, 129, 256, 257, 384, 500, 640, 3000, 5]
    nq = [3, 1, 5, 32, 2, 9, 1, 32, 17, 30, 32, 20]
    run_paged(nq, lens, 8, 2, d, 16, causal, seed=31)
    run_paged([1] * 12, lens, 40, 2, d, 128, causal, seed=32)
    run_paged([32, 5], [9000, 40], 4, 1, d, 64, causal, seed=33)
    run_paged([120], [300], 1, 1, d, 32, causal, seed=34, max_kv=2000)
    run_paged([5] * 40, [700 + 13 * i for i in range(40)], 32, 8, d, 64, causal, seed=35)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda x: "-".join(map(str, x[1])))
def test_paged_loose_bounds(lengths, d):
    """Short lengths under a bound that allows long ones: the split is chosen on the device."""
    run_paged(*lengths, 6, 2, d, 16, True, seed=21, max_kv=max(2000, max(lengths[1])))


@pytest.mark.parametrize("d", [64, 128])
def test_paged_whole_segments_of_several_row_tiles(d):
    """More than 16 rows a key/value head where a CTA takes whole segments."""
    for causal in (True, False):
        run_paged([40, 1, 0, 17], [300, 1000, 5, 12], 4, 1, d, 16, causal, seed=51)
        run_paged([130], [130], 6, 2, d, 64, causal, seed=52)
        run_paged([5] * 19, list(range(1, 20)), 32, 8, d, 32, causal, seed=53)  # 304 row tiles, few keys


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,lens", [([1], [20000]), ([1, 1, 1, 1], [5000, 0, 1025, 16]), ([3, 0, 2], [9001, 7, 1]),
                                     ([1] * 8, [4100, 1024, 1030, 1, 0, 4000, 17, 2048]), ([16], [6000])],
                         ids=lambda x: "-".join(map(str, x)))
def test_paged_few_long_segments(nq, lens, d):
    """At most 8 segments: CTAs share their keys."""
    for H in (1, 4):
        _, q, out, lse = run_paged(nq, lens, H, 1, d, 64, True, seed=61)
        again = run_paged(nq, lens, H, 1, d, 64, True, seed=61)
        assert torch.equal(out, again[2]) and torch.equal(lse, again[3])


@pytest.mark.parametrize("B,most", [(19, 1024), (19, 1025), (20, 512), (20, 513), (20, 64), (38, 300), (39, 300)])
def test_paged_where_whole_segments_end(B, most):
    """152 and 304 segments, 512 and 1024 keys: on both sides of the sizes at which a CTA takes whole
    segments."""
    lens = [most] + [(53 * b) % (most + 1) for b in range(1, B)]
    run_paged([1 + b % 2 for b in range(B)], lens, 24, 8, 64, 64, True, seed=41)


def test_paged_many_ragged_sequences():
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 900, 150).tolist()
    run_paged([1] * 150, lens, 4, 2, 64, 16, True, seed=9)
    nq = rng.integers(0, 4, 150).tolist()
    run_paged(nq, lens, 4, 2, 64, 16, True, seed=10)


@pytest.mark.parametrize("most", [127, 128, 129, 255, 256, 257])
@pytest.mark.parametrize("B", [3, 80], ids=["few segments", "many segments"])
def test_paged_at_the_lengths_where_splitting_begins(B, most):
    lens = [most] + [1 + (37 * b) % most for b in range(1, B)]
    run_paged([1] * B, lens, 8, 4, 64, 32, True, seed=most)


def test_paged_more_sequences_than_threads():
    """The scan over the sequences takes several rounds (256 and 384 entries at a time)."""
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 60, 900).tolist()
    lens[700] = 3000
    run_paged([1] * 900, lens, 2, 1, 64, 16, True, seed=13)
    nq = rng.integers(0, 3, 900).tolist()
    nq[3] = 40
    run_paged(nq, lens, 2, 1, 128, 16, True, seed=14)


def test_paged_128_heads_of_one_key_head():
    run_paged([1, 3], [300, 900], 128, 1, 64, 32, True, seed=15)
    run_paged([1, 1], [30, 2000], 128, 1, 128, 16, False, seed=16)


@pytest.mark.parametrize("scale,sigma", [(0.0, 1.0), (1.5, 1.0), (None, 4.0)])
def test_paged_scales(scale, sigma):
    run_paged([1, 2], [700, 70], 4, 2, 64, 16, True, seed=4, scale=scale, sigma=sigma)


def test_paged_defaults_and_capacity():
    """One token per sequence without cu_seqlens, bounds from the block table: the same bits as
    with close bounds where the lengths are split the same way."""
    cache, q, out, lse = run_paged([1] * 5, [100, 2000, 1, 64, 900], 8, 2, 128, 16, True, seed=12)
    k, v, table, lens = cache.dev()
    wide = torch.full((5, 4 * table.shape[1]), -1, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    o2, l2 = fa.fa_fwd_paged(q.to(DEV), k, v, wide, lens)
    assert fa.fa_get_error() == fa.FA_OK
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_paged_is_bitwise_repeatable_and_leaves_other_rows():
    cache = Cache([3000, 10, 1200], 2, 128, 64, seed=21)
    q = torch.randn(9, 8, 128, device=DEV).to(BF16)
    cu = i32([0, 2, 2, 5])  # tokens 5..8 belong to no sequence
    out = torch.full_like(q, 7.0)
    lse = torch.full((8, 9), 7.0, device=DEV)
    first = None
    for _ in range(3):
        o, l = fa.fa_fwd_paged(q, *cache.dev(), cu_seqlens=cu, max_q=3, causal=True, out=out, lse=lse)
        assert torch.all(o[5:] == 7.0) and torch.all(l[:, 5:] == 7.0)
        assert not torch.any(o[:5] == 7.0)
        first = first or (o.clone(), l.clone())
        assert torch.equal(o, first[0]) and torch.equal(l, first[1])
    assert fa.fa_get_error() == fa.FA_OK


@pytest.mark.parametrize("nq,max_kv", [(1, 224), (1, 2000), (40, 224), (40, 2000)],
                         ids=["whole", "few rows", "whole, tiles", "many rows"])
def test_paged_bad_pages_read_as_zeros_and_are_reported(nq, max_kv):
    """Pages outside the pool are not read: their keys and values count as zeros, and the status
    says so."""
    lens, Hkv, d, page = [200, 90], 2, 64, 32
    cache = Cache(lens, Hkv, d, page, seed=31)
    k, v, table, ln = cache.dev()
    table[0, 1], table[0, 4], table[1, 0] = -5, k.shape[0], 1 << 30
    q = torch.randn(2 * nq, 4, d, device=DEV).to(BF16)
    out, lse = fa.fa_fwd_paged(q, k, v, table, ln, cu_seqlens=i32([0, nq, 2 * nq]), max_q=nq,
                               max_kv=max_kv)
    assert fa.fa_get_error() == fa.FA_ERR_INDEX and fa.fa_get_error() == fa.FA_OK
    per = []
    for b, gone in ((0, [1, 4]), (1, [0])):
        K, V = cache.keys(b)
        for g in gone:
            K[:, g * page:(g + 1) * page], V[:, g * page:(g + 1) * page] = 0, 0
        per.append((K, V, [lens[b]] * nq))
    check(out, lse, q, [0, nq, 2 * nq], per, d ** -0.5)


def test_paged_lengths_past_their_bounds():
    cache = Cache([100], 1, 64, 16, seed=5)
    k, v, table, _ = cache.dev()
    q = torch.randn(1, 1, 64, device=DEV).to(BF16)
    full, _ = fa.fa_fwd_paged(q, k, v, table[:, :6].contiguous(), i32([96]))
    assert fa.fa_get_error() == fa.FA_OK
    for lens, kw in ((500, {}), (100, dict(max_kv=96))):
        out, _ = fa.fa_fwd_paged(q, k, v, table[:, :6].contiguous(), i32([lens]), **kw)
        assert fa.fa_get_error() == fa.FA_ERR_INDEX
        assert torch.equal(out, full)
    out, lse = fa.fa_fwd_paged(q, k, v, table, i32([-3]))
    assert fa.fa_get_error() == fa.FA_ERR_INDEX
    assert not out.any() and torch.isinf(lse).all()
    # more new tokens than max_q: the first max_q of them are computed, the others left
    q5 = torch.randn(5, 1, 64, device=DEV).to(BF16)
    want, _ = fa.fa_fwd_paged(q5, k, v, table, i32([100]), cu_seqlens=i32([0, 5]), causal=True)
    out = torch.full_like(q5, 7.0)
    fa.fa_fwd_paged(q5, k, v, table, i32([100]), cu_seqlens=i32([0, 5]), max_q=2, causal=True, out=out)
    assert fa.fa_get_error() == fa.FA_ERR_INDEX
    assert torch.equal(out[:2], want[:2]) and torch.all(out[2:] == 7.0)


def test_paged_offsets_past_32_bits():
    """A pool of more than 2^31 elements (and 2^32 bytes): the last pages are read and written."""
    Hkv, page, d = 8, 128, 128
    pages = (1 << 31) // (Hkv * page * d) + 40
    k = torch.empty(pages, Hkv, page, d, dtype=BF16, device=DEV)
    v = torch.empty(pages, Hkv, page, d, dtype=BF16, device=DEV)
    lens = [300, 140]
    table = torch.tensor([[pages - 1, 3, pages - 7], [pages - 2, pages - 3, -1]], dtype=torch.int32)
    new = torch.randn(sum(lens), 2 * Hkv, d).to(BF16)
    nk, nv = new[:, :Hkv].to(DEV), new[:, Hkv:].to(DEV)
    fa.fa_kv_append(None, nk, nv, k, v, table.to(DEV), i32(lens), cu_seqlens=i32(cumulative(lens)))
    assert torch.equal(k[pages - 7, :, 43], nk[299]) and torch.equal(v[pages - 3, :, 11], nv[439])
    q = torch.randn(2, Hkv, d, device=DEV).to(BF16)
    out, lse = fa.fa_fwd_paged(q, k, v, table.to(DEV), i32(lens))
    assert fa.fa_get_error() == fa.FA_OK
    cut = cumulative(lens)
    per = [(f64(nk[cut[b]:cut[b + 1]]).transpose(1, 0, 2), f64(nv[cut[b]:cut[b + 1]]).transpose(1, 0, 2), [lens[b]])
           for b in range(2)]
    check(out, lse, q, [0, 1, 2], per, d ** -0.5)


def test_paged_streams_and_graphs():
    cache = Cache([2500, 30, 700], 2, 64, 16, seed=41)
    k, v, table, lens = cache.dev()
    q = torch.randn(3, 4, 64, device=DEV).to(BF16)
    want = fa.fa_fwd_paged(q, k, v, table, lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fa.fa_fwd_paged(q, k, v, table, lens, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # two graphs with a workspace each, replayed at once on two streams
    graphs, outs, qs, streams = [], [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(2):
        qs.append(q.clone())
        ws = torch.empty(fa.fa_fwd_paged_workspace_size(3, 3, 4, 2, 64), dtype=torch.uint8, device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((fa.fa_fwd_paged(qs[i], k, v, table, lens, workspace=ws), ws))
        graphs.append(g)
    qs[1].copy_(q.flip(0))
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs[0][0]))
    ref = fa.fa_fwd_paged(q.flip(0).contiguous(), k, v, table, lens)
    assert all(torch.equal(a, b) for a, b in zip(ref, outs[1][0]))
    # lengths that grow between replays of one graph
    lens.copy_(i32([2400, 29, 690]))
    graphs[0].replay()
    torch.cuda.synchronize()
    ref = fa.fa_fwd_paged(q, k, v, table, lens)
    assert all(torch.equal(a, b) for a, b in zip(ref, outs[0][0]))
    assert fa.fa_get_error() == fa.FA_OK


def test_calls_in_a_row_wait_for_each_other():
    """Launches overlap the end of the one before; every call still sees what was written ahead of
    it on the stream: lengths that a kernel in between advances, keys that the call before appended,
    a workspace and outputs that the call before used."""
    B, H, Hkv, d, page, steps = 6, 8, 2, 64, 16, 60
    k = torch.zeros(B * 40, Hkv, page, d, dtype=BF16, device=DEV)
    v = torch.zeros_like(k)
    table = torch.arange(B * 40, device=DEV).view(B, 40).to(torch.int32)
    new = torch.randn(steps, B, H + 2 * Hkv, d, device=DEV).to(BF16)
    lens = i32([0, 100, 200, 300, 400, 500])
    q = torch.empty(B, H, d, dtype=BF16, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(H, B, device=DEV)
    ws = torch.empty(fa.fa_fwd_paged_workspace_size(B, B, H, Hkv, d), dtype=torch.uint8, device=DEV)

    def run(wait):
        k.zero_(), v.zero_()
        ln, outs = lens.clone(), []
        for s in range(steps):
            ln += 1
            x = new[s].split([H, Hkv, Hkv], dim=1)
            fa.fa_kv_append(*x, k, v, table, ln, q_out=q)
            wait()
            fa.fa_fwd_paged(q, k, v, table, ln, out=out, lse=lse, workspace=ws)
            wait()
            outs.append((out.clone(), lse.clone()))
        return outs

    waited = run(torch.cuda.synchronize)
    for _ in range(3):
        for a, b in zip(waited, run(lambda: None)):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert fa.fa_get_error() == fa.FA_OK


@pytest.mark.parametrize("d", [64, 128])
def test_tensor_core_kernel_times_out_then_recovers(d, monkeypatch):
    """Waits of the pipeline that run out end the kernel, the call reports it, and the next call is
    right again (no fault, nothing left behind)."""
    args = ([200, 90], [1500, 700], 4, 2, d, 32, True)
    cache = Cache(args[1], 2, d, 32, seed=3)
    q = torch.randn(290, 4, d, device=DEV).to(BF16)
    monkeypatch.setenv("FA_WAIT_TIMEOUT_US", "1")
    fa.fa_fwd_paged(q, *cache.dev(), cu_seqlens=i32([0, 200, 290]), max_q=200, causal=True)
    status = fa.fa_get_error()
    monkeypatch.delenv("FA_WAIT_TIMEOUT_US")
    assert status == fa.FA_ERR_TIMEOUT, fa.fa_status_string(status)
    run_paged(*args, seed=17)


@pytest.mark.parametrize("d", [64, 128])
def test_join_reads_nothing_out_of_range_after_a_launch_that_gave_up(d, monkeypatch):
    """A launch that gives up leaves the workspace as it was: spans whose end wraps past 2^31 among
    what it may hold are skipped by the join."""
    cache = Cache([4000], 1, d, 64, seed=3)
    q = torch.randn(1, 64, d, device=DEV).to(BF16)
    size = fa.fa_fwd_paged_workspace_size(1, 1, 64, 1, d)
    want, _ = fa.fa_fwd_paged(q, *cache.dev(), max_kv=4000)
    for span in ([1, 0x7FFFFFFF], [0x7FFFFFFF, 2], [-5, 3], [0x7FFFFFFF, 0x7FFFFFFF]):
        ws = i32(span).repeat(size // 8).view(torch.uint8)
        monkeypatch.setenv("FA_WAIT_TIMEOUT_US", "1")
        fa.fa_fwd_paged(q, *cache.dev(), max_kv=4000, workspace=ws)
        fa.fa_get_error()
        monkeypatch.delenv("FA_WAIT_TIMEOUT_US")
        out, _ = fa.fa_fwd_paged(q, *cache.dev(), max_kv=4000, workspace=ws)
        assert fa.fa_get_error() == fa.FA_OK and torch.equal(out, want)


@pytest.mark.parametrize("d", [64, 128])
def test_join_skips_spans_that_a_launch_that_gave_up_did_not_write(d, monkeypatch):
    """Six or seven segments a CTA, whose pieces wait for one of four places from the fifth on: with a
    limit of 1 us the launch gives up before it has written every span, and the join finds what the
    workspace held there.  It skips such spans: their rows become those of a query without keys."""
    B, nq = 1000, 40
    cache = Cache([100] * B, 1, d, 64, seed=9)
    args, q = cache.dev(), torch.randn(B * nq, 1, d, device=DEV).to(BF16)
    kw = dict(cu_seqlens=i32(list(range(0, B * nq + 1, nq))), max_q=nq, max_kv=2000)
    want, want_lse = fa.fa_fwd_paged(q, *args, **kw)
    assert fa.fa_get_error() == fa.FA_OK and torch.isfinite(want_lse).all()
    size = fa.fa_fwd_paged_workspace_size(B, B * nq, 1, 1, d)
    for span in ([1, 0x7FFFFFFF], [0x7FFFFFFF, 2], [-5, 3], [0x7FFFFFFF, 0x7FFFFFFF], [151, 2]):
        ws = i32(span).repeat(size // 8).view(torch.uint8)
        out, lse = torch.full_like(want, 7.0), torch.full_like(want_lse, 7.0)
        monkeypatch.setenv("FA_WAIT_TIMEOUT_US", "1")
        fa.fa_fwd_paged(q, *args, **kw, workspace=ws, out=out, lse=lse)
        assert fa.fa_get_error() == fa.FA_ERR_TIMEOUT
        monkeypatch.delenv("FA_WAIT_TIMEOUT_US")
        skipped = torch.isneginf(lse[0])
        assert skipped.any() and not out[skipped].any()
        again = fa.fa_fwd_paged(q, *args, **kw, workspace=ws, out=out, lse=lse)
        assert fa.fa_get_error() == fa.FA_OK
        assert torch.equal(again[0], want) and torch.equal(again[1], want_lse)


@pytest.mark.parametrize("G", [1, 64], ids=["few rows", "many rows"])
def test_paged_length_at_the_end_of_its_type(G):
    """kv_lens of 2^31 - 1 over pages that are all the same one: clamped to 2^31 - 256 keys and
    reported.  Scores are 0 and V is 1, so weights are 1, a worker's sums are integers below 2^24
    (exact), and joining at most 1216 parts leaves 1216 x 2^-24 of relative error."""
    k = torch.zeros(1, 1, 128, 64, dtype=BF16, device=DEV)
    v = torch.ones_like(k)
    table = torch.zeros(1, 1 << 24, dtype=torch.int32, device=DEV)
    q = torch.ones(1, G, 64, dtype=BF16, device=DEV)
    out, lse = fa.fa_fwd_paged(q, k, v, table, i32([0x7FFFFFFF]))
    assert fa.fa_get_error() == fa.FA_ERR_INDEX
    bound = 1216 * 2.0 ** -24
    assert np.abs(f64(out) - 1).max() <= 2 * bound + 2.0 ** -8
    assert np.abs(f64(lse) - np.log(2.0 ** 31 - 256)).max() <= bound + 2.0 ** -20 * 22


@pytest.mark.parametrize("nq,max_kv", [(2, 700), (2, 2000), (40, 2000)], ids=["whole", "few rows", "many rows"])
def test_offsets_that_do_not_ascend_are_reported(nq, max_kv):
    cache = Cache([700, 20, 300], 2, 64, 16, seed=17)
    k, v, table, lens = cache.dev()
    q = torch.randn(3 * nq, 4, 64, device=DEV).to(BF16)
    n = 3 * nq
    for cu in ([0, n, 0, n], [-3, nq, 2 * nq, n], [0, nq, 2 * nq, n + 9], [n, 0, n, 0]):
        fa.fa_fwd_paged(q, k, v, table, lens, cu_seqlens=i32(cu), max_q=n, max_kv=max_kv)
        assert fa.fa_get_error() == fa.FA_ERR_INDEX
    groups = i32([0, 3, 1])
    fa.fa_fwd_shared_prefix(q, k, v, table, lens, table[:2].contiguous(), lens[:2].contiguous(), groups,
                            cu_seqlens=i32([0, nq, 2 * nq, n]), max_q=nq, max_kv=max_kv)
    assert fa.fa_get_error() == fa.FA_ERR_INDEX


@pytest.mark.parametrize("nq", [1, 40], ids=["few rows", "many rows"])
def test_stream_argument_writes_no_memory_that_the_current_stream_still_uses(nq):
    """Memory freed on the current stream while a kernel there has still to write it is not handed
    to a call on another stream."""
    cache = Cache([3000, 40], 2, 128, 64, seed=7)
    args = cache.dev()
    q = torch.randn(2 * nq, 8, 128, device=DEV).to(BF16)
    kw = dict(cu_seqlens=i32([0, nq, 2 * nq]), max_q=nq, max_kv=3000)
    want = fa.fa_fwd_paged(q, *args, **kw)
    ws = fa.fa_fwd_paged_workspace_size(2, 2 * nq, 8, 2, 128)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    old = [torch.empty_like(t) for t in want] + [torch.empty(ws, dtype=torch.uint8, device=DEV)]
    torch.cuda._sleep(20_000_000)
    for t in old:
        t.fill_(9)
    del old, t
    got = fa.fa_fwd_paged(q, *args, **kw, stream=side)
    torch.cuda.synchronize()
    assert fa.fa_get_error() == fa.FA_OK
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    with pytest.raises(ValueError):
        fa.fa_fwd_paged(None, *args, stream=side)


def test_paged_empty_and_refusals():
    cache = Cache([5, 6], 2, 64, 16, seed=1)
    k, v, table, lens = cache.dev()
    q = torch.empty(0, 4, 64, dtype=BF16, device=DEV)
    out, lse = fa.fa_fwd_paged(q, k, v, table, lens, cu_seqlens=i32([0, 0, 0]))
    assert out.numel() == 0 and lse.numel() == 0
    q = torch.zeros(2, 4, 64, dtype=BF16, device=DEV)
    for bad in (dict(q=q[:, :3]), dict(q=q.float()), dict(table=table.long()), dict(table=table[:1]),
                dict(lens=lens[:1]), dict(v=v[:, :1]), dict(v=v[:3]), dict(k=k.float()),
                dict(cu_seqlens=i32([0, 2])), dict(q=torch.zeros(3, 4, 64, dtype=BF16, device=DEV)),
                dict(out=torch.zeros(2, 4, 64, device=DEV)), dict(lse=torch.zeros(2, 4, device=DEV)),
                dict(table=table.cpu()), dict(k=k.transpose(1, 2), v=v.transpose(1, 2))):
        a = dict(q=q, k=k, v=v, table=table, lens=lens)
        a.update({n: t for n, t in bad.items() if n in a})
        kw = {n: t for n, t in bad.items() if n not in a}
        with pytest.raises(ValueError):
            fa.fa_fwd_paged(a["q"], a["k"], a["v"], a["table"], a["lens"], **kw)
    with pytest.raises(fa.binding.FAError):
        fa.fa_fwd_paged(q, k, v, table, lens, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    odd = torch.zeros(4, 2, 24, 64, dtype=BF16, device=DEV)
    with pytest.raises(fa.binding.FAError):
        fa.fa_fwd_paged(q, odd, odd, table, lens)


# ------------------------------------------------------------------------------------------ append
@pytest.mark.parametrize("heads", [(8, 2, 128, 64, 128, False, True), (3, 3, 64, 16, 32, True, False),
                                   (16, 1, 128, 128, 64, False, True), (4, 2, 64, 32, 0, False, False)],
                         ids=lambda h: "H%dkv%dd%dpage%dr%d%s%s" % (*h[:5], "i" if h[5] else "", "n" if h[6] else ""))
@pytest.mark.parametrize("lengths", [([1, 1, 1], [1, 64, 300]), ([130, 0, 1, 17], [130, 5, 33, 200]),
                                     ([3, 6], [1, 6])], ids=["decode", "prompts", "more than keys"])
def test_append(lengths, heads):
    H, Hkv, d, page, rot, inter, norm = heads
    nq, lens = lengths
    cache = Cache(lens, Hkv, d, page, seed=50 + H)
    k, v, table, ln = cache.dev()
    cu, T = cumulative(nq), sum(nq)
    qkv = torch.randn(T + 2, H + 2 * Hkv, d, device=DEV).to(BF16)  # two tokens behind the last sequence
    q, kn, vn = qkv.split([H, Hkv, Hkv], dim=1)
    w = [1 + 0.2 * torch.randn(d, device=DEV) if norm else None for _ in range(2)]
    inv = fa.rope_frequencies(rot)[0] if rot else None
    tab = fa.fa_rope_table(4096, rot, inv_freq=inv) if rot else None
    off = i32([7 * b for b in range(len(lens))])
    q_out = torch.full((T + 2, H, d), 7.0, dtype=BF16, device=DEV)
    k0, v0 = k.clone(), v.clone()
    got = fa.fa_kv_append(q, kn, vn, k, v, table, ln, cu_seqlens=i32(cu), pos_offset=off, table=tab,
                          interleaved=inter, q_weight=w[0], k_weight=w[1], q_out=q_out)
    assert fa.fa_get_error() == fa.FA_OK and got is q_out
    assert torch.all(q_out[T:] == 7.0)
    ref = dict(inv_freq=None if inv is None else inv.numpy(), interleaved=inter)
    written = torch.zeros(k.shape[0], page, dtype=torch.bool)
    for b in range(len(lens)):
        a, e = cu[b], cu[b + 1]
        key = np.arange(lens[b] - nq[b], lens[b])
        pos = np.where(key >= 0, key + 7 * b, 0)
        for x, wt, target in ((q, w[0], got[a:e]), (kn, w[1], None)):
            r = norm_rope(f64(x[a:e]), pos, None if wt is None else f64(wt), **ref)
            if target is None:
                for i in range(nq[b]):
                    if key[i] < 0:
                        continue
                    p, o = int(table[b, key[i] // page]), int(key[i] % page)
                    written[p, o] = True
                    err = np.abs(f64(k[p, :, o]) - r[i]) - (2.0 ** -8 * np.abs(r[i]) + 2.0 ** -18 * np.abs(r[i]).max())
                    assert err.max() <= 0
                    assert torch.equal(v[p, :, o], vn[a + i])
            elif r.size:
                err = np.abs(f64(target) - r) - (2.0 ** -8 * np.abs(r) + 2.0 ** -18 * np.abs(r).max(-1, keepdims=True))
                assert err.max() <= 0
    same = ~written.to(DEV)[:, None, :, None].expand_as(k)  # nothing else of the pool moved
    assert torch.equal(torch.nan_to_num(k)[same], torch.nan_to_num(k0)[same])
    assert torch.equal(torch.nan_to_num(v)[same], torch.nan_to_num(v0)[same])


def test_append_bad_pages_write_nothing():
    k = torch.full((4, 1, 16, 64), 5.0, dtype=BF16, device=DEV)
    v = k.clone()
    x = torch.ones(5, 1, 64, dtype=BF16, device=DEV)
    table = i32([[4], [-1], [2], [0], [1 << 30]])
    q = fa.fa_kv_append(x, x, x, k, v, table, i32([3, 3, 17, 2, 1]))
    assert fa.fa_get_error() == fa.FA_ERR_INDEX
    assert torch.equal(q, x)
    assert torch.equal(k[0, 0, 1], x[3, 0]) and k.sum() == v.sum() == 5.0 * k.numel() - 4 * 64
    for lens in (-2, -0x80000000):
        fa.fa_kv_append(None, x[:1], x[:1], k, v, i32([[1]]), i32([lens]))
        assert fa.fa_get_error() == fa.FA_ERR_INDEX
    # a position past 32 bits is past the table; the key is written all the same
    rope = fa.fa_rope_table(8, 64)
    far = fa.fa_kv_append(x[:1], x[:1], x[:1], k, v, i32([[0]]), i32([2]), table=rope, pos_offset=i32([0x7FFFFFFF]))
    assert fa.fa_get_error() == fa.FA_ERR_INDEX
    last = fa.fa_kv_append(x[:1], x[:1], x[:1], k, v, i32([[0]]), i32([2]), table=rope, pos_offset=i32([6]))
    assert fa.fa_get_error() == fa.FA_OK and torch.equal(far, last)
    fa.fa_kv_append(None, x[:1], x[:1], k, v, i32([[0]]), i32([2]))
    assert k.sum() == 5.0 * k.numel() - 4 * 64
    # offsets that do not ascend (reported or not): nothing written outside the sequences' pages
    fa.fa_kv_append(None, x[:3], x[:3], k, v, i32([[0], [0]]), i32([2, 2]), cu_seqlens=i32([2, 1, 3]))
    fa.fa_get_error()
    fa.fa_kv_append(None, x[:1], x[:1], k, v, i32([[0]]), i32([2]))
    assert k.sum() == 5.0 * k.numel() - 4 * 64


def test_append_refusals():
    k = torch.zeros(4, 2, 16, 64, dtype=BF16, device=DEV)
    x = torch.zeros(2, 2, 64, dtype=BF16, device=DEV)
    table, lens = i32([[0], [1]]), i32([1, 1])
    for bad in (dict(k=x[:, :1]), dict(v=x[:1]), dict(q=x[:1]), dict(k=x.float()),
                dict(pos_offset=i32([1])), dict(cu_seqlens=i32([0, 1])),
                dict(k=torch.zeros(3, 2, 64, dtype=BF16, device=DEV))):
        a = dict(q=x, k=x, v=x)
        a.update({n: t for n, t in bad.items() if n in a})
        with pytest.raises(ValueError):
            fa.fa_kv_append(a["q"], a["k"], a["v"], k, k.clone(), table, lens,
                            **{n: t for n, t in bad.items() if n not in a})
    assert fa.fa_kv_append(x[:0], x[:0], x[:0], k, k.clone(), table, lens, cu_seqlens=i32([0, 0, 0])).shape[0] == 0


# --------------------------------------------------------------------------------- shared prefixes
def run_prefix(groups, pre, nq, lens, H, Hkv, d, page, causal, seed, **kw):
    """groups: how many sequences behind each prefix."""
    cache = Cache(list(lens) + list(pre), Hkv, d, page, seed)
    k, v, table, ln = cache.dev()
    B, cu = len(lens), cumulative(nq)
    gcu = cumulative(groups)
    q = torch.randn(cu[-1], H, d, generator=torch.Generator().manual_seed(seed)).to(BF16)
    args = dict(cu_seqlens=i32(cu), max_q=max(nq), max_kv=max(lens), max_prefix=max(pre), causal=causal)
    args.update(kw)
    out, lse = fa.fa_fwd_shared_prefix(q.to(DEV), k, v, table[:B].contiguous(), ln[:B].contiguous(),
                                       table[B:].contiguous(), ln[B:].contiguous(), i32(gcu), **args)
    assert fa.fa_get_error() == fa.FA_OK
    per = []
    for b in range(B):
        g = int(np.searchsorted(gcu, b, side="right")) - 1
        both = [np.concatenate([p, s], 1) for p, s in zip(cache.keys(B + g), cache.keys(b))]
        per.append((*both, [pre[g] + max(0, x) for x in limits_of(nq[b], lens[b], causal)]))
    check(out, lse, q, cu, per, d ** -0.5, str((groups, pre, nq, lens)))
    return out, lse


@pytest.mark.parametrize("heads", [(4, 2, 128, 64), (1, 1, 64, 16), (24, 3, 64, 32), (32, 1, 128, 128)],
                         ids=lambda h: "H%dkv%dd%dpage%d" % h)
@pytest.mark.parametrize("batch", [
    ([1], [100], [1], [5]),
    ([3], [1000], [1, 1, 1], [0, 1, 200]),
    ([2, 0, 4], [70, 33, 2100], [1] * 6, [1, 0, 16, 100, 64, 3]),
    ([2, 3], [0, 17], [2, 1, 0, 3, 1], [2, 0, 9, 800, 1]),
    ([40], [600], [1] * 40, list(range(40))),
], ids=lambda b: "%s-%s" % (b[0], b[1]))
def test_shared_prefix(batch, heads):
    H, Hkv, d, page = heads
    for causal in (True, False):
        run_prefix(*batch, H, Hkv, d, page, causal, seed=60 + H)
        # under a bound that is too long for whole sequences a CTA
        run_prefix(*batch, H, Hkv, d, page, causal, seed=60 + H, max_prefix=5000)


def test_shared_prefix_large_groups():
    """Hundreds of query rows a key/value head behind one prefix, in two groups."""
    rng = np.random.default_rng(8)
    run_prefix([70, 9], [1500, 40], [2] * 79, rng.integers(2, 90, 79).tolist(), 8, 2, 128, 64, True, seed=71)
    run_prefix([150], [777], [1] * 150, rng.integers(0, 30, 150).tolist(), 6, 2, 64, 16, True, seed=72)


@pytest.mark.parametrize("d", [64, 128])
def test_shared_prefix_whole_sequences(d):
    """Sequences small enough for a CTA each, prefix and own keys: one, two and three turns, several
    row tiles, prefixes and sequences without keys, tokens without own keys."""
    rng = np.random.default_rng(28)
    run_prefix([1, 3, 15], [1000, 17, 0], [1] * 19, rng.integers(0, 150, 19).tolist(), 32, 8, d, 16, True, seed=81)
    run_prefix([20, 16], [500, 33], [1] * 36, rng.integers(0, 100, 36).tolist(), 8, 8, d, 64, True, seed=82)
    run_prefix([50], [256], [1] * 50, rng.integers(0, 256, 50).tolist(), 8, 8, d, 32, False, seed=83)
    run_prefix([2, 0, 2], [100, 5, 300], [40, 7, 0, 33], [40, 3, 2, 90], 8, 2, d, 128, True, seed=84)


def test_shared_prefix_of_the_sequences_own_table():
    """One table for both: every sequence's own keys are its prefix's pages again."""
    cache = Cache([100, 37], 2, 64, 32, seed=85)
    k, v, table, lens = cache.dev()
    q = torch.randn(2, 4, 64, device=DEV).to(BF16)
    own = i32([70, 20])
    for bounds in (dict(max_prefix=100, max_kv=70), dict(max_prefix=4000, max_kv=4000)):
        out, lse = fa.fa_fwd_shared_prefix(q, k, v, table, own, table, lens, i32([0, 1, 2]), **bounds)
        assert fa.fa_get_error() == fa.FA_OK
        per = []
        for b, n in enumerate((70, 20)):
            K, V = cache.keys(b)
            per.append((np.concatenate([K, K[:, :n]], 1), np.concatenate([V, V[:, :n]], 1), [cache.lens[b] + n]))
        check(out, lse, q, [0, 1, 2], per, 64 ** -0.5)


@pytest.mark.parametrize("bound", [300, 5000], ids=["whole", "two lists"])
def test_shared_prefix_reports_what_is_out_of_range(bound):
    cache = Cache([20, 30, 200], 1, 64, 16, seed=86)
    k, v, table, lens = cache.dev()
    q = torch.randn(2, 2, 64, device=DEV).to(BF16)
    args = [q, k, v, table[:2].contiguous(), lens[:2].contiguous(), table[2:].contiguous(), lens[2:].contiguous()]
    want = fa.fa_fwd_shared_prefix(*args, i32([0, 2]), max_prefix=bound, max_kv=30)[0]
    assert fa.fa_get_error() == fa.FA_OK
    long = args[:6] + [i32([5000 + bound])]
    got = fa.fa_fwd_shared_prefix(*long, i32([0, 2]), max_prefix=200, max_kv=30 if bound == 300 else 5000)[0]
    assert fa.fa_get_error() == fa.FA_ERR_INDEX
    assert torch.allclose(got.float(), want.float(), atol=2 ** -6)
    bad = args[5].clone()
    bad[0, 3] = -1
    fa.fa_fwd_shared_prefix(*args[:5], bad, args[6], i32([0, 2]), max_prefix=bound, max_kv=30)
    assert fa.fa_get_error() == fa.FA_ERR_INDEX
    fa.fa_fwd_shared_prefix(*args, i32([0, 9]), max_prefix=bound, max_kv=30)
    assert fa.fa_get_error() == fa.FA_ERR_INDEX


@pytest.mark.parametrize("d", [64, 128])
def test_shared_prefix_lists_of_both_kinds(d):
    """Each list on either kernel's tiles: long chunks behind few or many rows, groups without a
    sequence, prefixes alone, own keys alone."""
    rng = np.random.default_rng(18)
    run_prefix([1, 0, 0, 0, 0, 0, 0, 0], [500] + [20] * 7, [40], [900], 2, 1, d, 64, True, seed=73)
    run_prefix([2, 3], [3000, 40], [70, 1, 40, 100, 3], [70, 700, 60, 1200, 3], 8, 2, d, 32, True, seed=74)
    run_prefix([2, 1], [4000, 10], [30, 50, 2], [30, 50, 2], 8, 2, d, 16, False, seed=75)
    run_prefix([20, 30], [1700, 2400], [1] * 50, [0] * 50, 8, 1, d, 64, True, seed=76)
    run_prefix([20, 30], [0, 0], [1] * 50, rng.integers(0, 400, 50).tolist(), 8, 1, d, 64, True, seed=77)
    run_prefix([90], [0], [2] * 90, rng.integers(2, 300, 90).tolist(), 4, 1, d, 16, True, seed=78)


def test_shared_prefix_defaults_repeat_and_graph():
    cache = Cache([20, 300, 41, 900, 700], 2, 64, 16, seed=81)
    k, v, table, ln = cache.dev()
    q = torch.randn(3, 8, 64, device=DEV).to(BF16)
    args = (k, v, table[:3].contiguous(), ln[:3].contiguous(), table[3:].contiguous(), ln[3:].contiguous(),
            i32([0, 2, 3]))
    want = fa.fa_fwd_shared_prefix(q, *args)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(want, fa.fa_fwd_shared_prefix(q, *args)))
    g = torch.cuda.CUDAGraph()
    static = torch.zeros_like(q)
    with torch.cuda.graph(g):
        out = fa.fa_fwd_shared_prefix(static, *args)
    static.copy_(q)
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(want, out))
    # a prefix in the sequences' own block tables is the same attention
    cat = torch.full((3, 200), -1, dtype=torch.int32, device=DEV)
    lens = []
    for b, grp in enumerate((3, 3, 4)):
        own, shared = -(-cache.lens[b] // 16), cache.lens[grp] // 16
        cat[b, :shared], cat[b, shared:shared + own] = table[grp, :shared], table[b, :own]
        lens.append(shared * 16 + cache.lens[b])
    whole = i32([c // 16 * 16 for c in cache.lens[3:]])  # whole pages of the prefixes
    a = fa.fa_fwd_shared_prefix(q, *args[:5], whole, args[6])
    b = fa.fa_fwd_paged(q, k, v, cat, i32(lens))
    assert torch.allclose(a[0].float(), b[0].float(), atol=2.0 ** -6) and torch.allclose(a[1], b[1], atol=1e-5)
    assert fa.fa_get_error() == fa.FA_OK


def test_shared_prefix_refusals():
    cache = Cache([5, 6, 20], 2, 64, 16, seed=1)
    k, v, table, ln = cache.dev()
    q = torch.zeros(2, 4, 64, dtype=BF16, device=DEV)
    good = [q, k, v, table[:2].contiguous(), ln[:2].contiguous(), table[2:].contiguous(),
            ln[2:].contiguous(), i32([0, 2])]
    fa.fa_fwd_shared_prefix(*good)
    for at, bad in ((5, table[2]), (5, table[2:].long()), (6, ln), (7, i32([0, 1, 2])), (7, i32([0, 2]).cpu())):
        args = list(good)
        args[at] = bad
        with pytest.raises(ValueError):
            fa.fa_fwd_shared_prefix(*args)
    with pytest.raises(fa.binding.FAError):
        fa.fa_fwd_shared_prefix(*good, max_prefix=-1)


def test_a_batch_of_no_sequences():
    """No sequences and no tokens: every call of a step returns empty outputs, the given ones if any."""
    H, Hkv, d = 4, 2, 64
    k = torch.full((3, Hkv, 16, d), 5.0, dtype=BF16, device=DEV)
    v = k.clone()
    table, lens, zero = torch.empty(0, 4, dtype=torch.int32, device=DEV), i32([]), i32([0])
    x = torch.empty(0, H + 2 * Hkv, d, dtype=BF16, device=DEV)
    q_out, out, lse = torch.empty(0, H, d, dtype=BF16, device=DEV), torch.empty(0, H, d, dtype=BF16, device=DEV), \
        torch.empty(H, 0, device=DEV)
    for kw in ({}, dict(cu_seqlens=zero)):
        assert fa.fa_kv_append(*x.split([H, Hkv, Hkv], dim=1), k, v, table, lens, q_out=q_out, **kw) is q_out
        q = fa.fa_kv_append(*x.split([H, Hkv, Hkv], dim=1), k, v, table, lens, **kw)
        got = fa.fa_fwd_paged(q, k, v, table, lens, **kw)
        assert got[0].shape == (0, H, d) and got[1].shape == (H, 0)
        got = fa.fa_fwd_paged(q, k, v, table, lens, out=out, lse=lse, **kw)
        assert got[0] is out and got[1] is lse
        for pre in (dict(table=table, lens=lens, cu=zero), dict(table=i32([[0]]), lens=i32([9]), cu=i32([0, 0]))):
            got = fa.fa_fwd_shared_prefix(q, k, v, table, lens, pre["table"], pre["lens"], pre["cu"], **kw)
            assert got[0].shape == (0, H, d) and got[1].shape == (H, 0)
    assert torch.all(k == 5.0) and torch.all(v == 5.0)
    with pytest.raises(ValueError):
        fa.fa_kv_append(*x.split([H, Hkv, Hkv], dim=1), k, v, table, lens, q_out=q_out[:, :1])
    with pytest.raises(ValueError):
        fa.fa_fwd_paged(q, k, v, table, lens, out=lse)
    assert fa.fa_get_error() == fa.FA_OK


# -------------------------------------------------------------------------------------- as one run
def test_calls_under_inference_mode_and_with_leaves():
    """Outputs allocated by the binding are ordinary tensors (inference tensors in that mode)."""
    cache = Cache([200, 90], 2, 64, 16, seed=91)
    args = cache.dev()
    q = torch.randn(2, 4, 64, device=DEV).to(BF16)
    want = fa.fa_fwd_paged(q, *args)[0]
    with torch.inference_mode():
        got = fa.fa_fwd_paged(q, *args)[0]
        assert got.is_inference() and torch.equal(got + 0, want)
        w = torch.ones(64, device=DEV)
        grads = fa.fa_qk_norm_rope_bwd(q, q, q, q, q, q_weight=w, k_weight=w)
        assert all(torch.isfinite(g + 0).all() for g in grads)
    leaf = q.clone().requires_grad_()
    out = fa.fa_fwd_paged(leaf, *args)[0]
    assert not out.requires_grad and torch.equal(out, want)
    dq, dk, dv, dwq, dwk = fa.fa_qk_norm_rope_bwd(q, q, q, q, q, q_weight=w, k_weight=w)
    assert dq.stride() == (3 * 4 * 64, 64, 1) and dk.data_ptr() == dq.data_ptr() + 2 * 4 * 64
    dq.add_(1)
    assert dwk.data_ptr() == dwq.data_ptr() + 4 * 64 and dwq.shape == dwk.shape == (64,)


def test_generation_run():
    """A prompt in one packed pass, its keys into the cache, then tokens one by one, against one
    causal pass over everything; then the same continuation for four sequences behind the prompt
    as a shared prefix."""
    H, Hkv, d, page, prompt, steps = 8, 2, 128, 32, 150, 9
    total = prompt + steps
    g = torch.Generator().manual_seed(91)
    qkv = torch.randn(total, H + 2 * Hkv, d, generator=g).to(BF16).to(DEV)
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g).to(DEV) for _ in range(2))
    opts = dict(table=fa.fa_rope_table(512, d), q_weight=wq, k_weight=wk)
    q, k, v = qkv.split([H, Hkv, Hkv], dim=1)
    # everything at once
    qr, kr, vr = fa.fa_qk_norm_rope_fwd(q, k, v, **opts)
    ref, ref_lse = fa.fa_fwd_varlen(qr, kr, vr, i32([0, total]), total, causal=True)
    # the prompt, then single tokens
    kc = torch.full((8, Hkv, page, d), float("nan"), dtype=BF16, device=DEV)
    vc = kc.clone()
    table = i32([[5, 2, 7, 0, 3]])
    qp = fa.fa_kv_append(q[:prompt], k[:prompt], v[:prompt], kc, vc, table, i32([prompt]),
                         cu_seqlens=i32([0, prompt]), **opts)
    assert torch.equal(qp, qr[:prompt])
    parts = [fa.fa_fwd_paged(qp, kc, vc, table, i32([prompt]), cu_seqlens=i32([0, prompt]), max_q=prompt, causal=True)]
    for t in range(prompt, total):
        one = slice(t, t + 1)
        lens = i32([t + 1])
        qd = fa.fa_kv_append(q[one], k[one], v[one], kc, vc, table, lens, **opts)
        parts.append(fa.fa_fwd_paged(qd, kc, vc, table, lens))
    assert fa.fa_get_error() == fa.FA_OK
    out = torch.cat([p[0] for p in parts])
    lse = torch.cat([p[1] for p in parts], 1)
    K, V = f64(kr).transpose(1, 0, 2), f64(vr).transpose(1, 0, 2)
    check(out, lse, qr, [0, total], [(K, V, range(1, total + 1))], d ** -0.5, "run")
    assert torch.allclose(lse, ref_lse, atol=1e-5)
    assert torch.allclose(out.float(), ref.float(), atol=2.0 ** -5)
    # four sequences that continue from the prompt's first 128 keys (whole pages)
    shared, B = 128, 4
    kc2, vc2 = kc.clone(), vc.clone()
    kc2[[1, 4, 6]], vc2[[1, 4, 6]] = float("nan"), float("nan")
    pool = torch.cat([kc2, torch.full_like(kc2, float("nan"))])
    poolv = torch.cat([vc2, torch.full_like(vc2, float("nan"))])
    own = i32([[1], [4], [6], [9]])
    cu = i32([0, 2, 4, 6, 8])
    new = torch.randn(2 * B, H + 2 * Hkv, d, generator=g).to(BF16).to(DEV)
    qn, kn, vn = new.split([H, Hkv, Hkv], dim=1)
    qd = fa.fa_kv_append(qn, kn, vn, pool, poolv, own, i32([2] * B), cu_seqlens=cu,
                         pos_offset=i32([shared] * B), **opts)
    got, glse = fa.fa_fwd_shared_prefix(qd, pool, poolv, own, i32([2] * B), table[:, :4].contiguous(),
                                        i32([shared]), i32([0, B]), cu_seqlens=cu, max_q=2, max_kv=2, causal=True)
    pos = i32([shared, shared + 1] * B)
    q2, k2, v2 = fa.fa_qk_norm_rope_fwd(qn, kn, vn, positions=pos, **opts)
    assert torch.equal(q2, qd)
    per = [(np.concatenate([K[:, :shared], f64(k2[2 * b:2 * b + 2]).transpose(1, 0, 2)], 1),
            np.concatenate([V[:, :shared], f64(v2[2 * b:2 * b + 2]).transpose(1, 0, 2)], 1),
            [shared + 1, shared + 2]) for b in range(B)]
    check(got, glse, q2, [0, 2, 4, 6, 8], per, d ** -0.5, "shared")
    assert fa.fa_get_error() == fa.FA_OK
