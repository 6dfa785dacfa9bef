"""Accumulated attention weights and eviction (fa_kv_weights, fa_kv_evict) against the fp64 reference.

Weights: a term exp(x) has x = scale q.k - LSE from float32 products and sums, off by at most
2^-24 (d + 16) scale sum|q k| + 2^-22 (|LSE| + |x|), the exponential by 2^-22 of itself, and the sum
of T terms by 2^-24 T of it; the total is rounded once more.  Eviction copies: everything is equal."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import exact_io_aware_fwd_gb300 as fa
from oracle.serving import attend, evict, key_weights, page_bounds, page_scores, select_pages
from test_paged_gpu import Cache, _built, cumulative, f64, i32, limits_of  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16

HEADS = [(1, 1, 64, 16), (8, 2, 128, 64), (6, 2, 64, 32), (32, 1, 128, 128), (5, 5, 128, 16)]
by_heads = pytest.mark.parametrize("heads", HEADS, ids=lambda h: "H%dkv%dd%dpage%d" % h)


class Weighted:
    def __init__(self, nq, lens, heads, causal, seed, sigma=1.0):
        H, Hkv, d, page = heads
        self.cache = Cache(lens, Hkv, d, page, seed, sigma)
        self.nq, self.lens, self.cu, self.causal = nq, lens, cumulative(nq), causal
        g = torch.Generator().manual_seed(seed + 1)
        self.q = (sigma * torch.randn(self.cu[-1], H, d, generator=g)).to(BF16)
        self.lse = torch.zeros(H, self.cu[-1])
        for b, n in enumerate(nq):
            K, V = self.cache.keys(b)
            L = attend(f64(self.q[self.cu[b]:self.cu[b + 1]]), K, V, d ** -0.5, limits_of(n, lens[b], causal))[1]
            self.lse[:, self.cu[b]:self.cu[b + 1]] = torch.from_numpy(L.T).float()
        self.before = torch.exp(torch.randn(len(lens), Hkv, max(max(lens), 1) + 3, generator=g))
        self.scale, self.d = d ** -0.5, d

    def args(self):
        k, _, table, lens = self.cache.dev()
        return self.q.to(DEV), self.lse.to(DEV), k, table, lens

    def opts(self):
        return dict(cu_seqlens=i32(self.cu), max_q=max(self.nq), max_kv=max(self.lens), causal=self.causal)

    def check(self, got, before):
        got = f64(got)
        for b, n in enumerate(self.nq):
            a, e = self.cu[b], self.cu[b + 1]
            K = self.cache.keys(b)[0]
            w, err = key_weights(f64(self.q[a:e]), K, self.scale, f64(self.lse[:, a:e].T),
                                 limits_of(n, self.lens[b], self.causal))
            was = np.zeros(got.shape[1:]) if before is None else f64(before[b])
            ref = was.copy()
            ref[:, :self.lens[b]] += w
            terms = max(1, n * self.q.shape[1] // got.shape[1])
            bound = 2.0 ** -24 * (self.d + 16 + 8 + terms) * err + 2.0 ** -23 * (w + was[:, :self.lens[b]])
            assert np.all(np.abs(got[b, :, :self.lens[b]] - ref[:, :self.lens[b]]) <= bound), b
            assert np.array_equal(got[b, :, self.lens[b]:], ref[:, self.lens[b]:]), b


@by_heads
@pytest.mark.parametrize("causal", [False, True], ids=["all", "causal"])
@pytest.mark.parametrize("nq,lens", [([1], [1]), ([1, 1, 1], [31, 128, 129]), ([3, 0, 1, 5], [40, 9, 1, 700]),
                                     ([4, 2], [2, 0]), ([32, 40], [300, 40])], ids=str)
def test_weights(nq, lens, causal, heads):
    w = Weighted(nq, lens, heads, causal, sum(lens) + heads[0])
    before = w.before.to(DEV)
    w.check(fa.fa_kv_weights(*w.args(), before, **w.opts()), w.before)
    assert torch.equal(before, w.before.to(DEV))
    w.check(fa.fa_kv_weights(*w.args(), **w.opts()), None)
    fa.fa_kv_weights(*w.args(), before, out=before, **w.opts())
    w.check(before, w.before)
    assert fa.fa_get_error() == fa.FA_OK


@pytest.mark.parametrize("heads", [(8, 2, 128, 64), (4, 2, 64, 16), (16, 1, 64, 32)], ids=lambda h: "H%dkv%dd%dpage%d" % h)
@pytest.mark.parametrize("causal", [False, True], ids=["all", "causal"])
def test_weights_of_many_queries_and_of_many_sequences(heads, causal):
    """Several jobs of 128 queries a piece, shares that end inside sequences, and many pieces a CTA."""
    for nq, lens in (([100, 7, 130], [700, 129, 131]), ([33], [20000]), ([1, 0, 2] * 50, [300, 0, 40] * 50),
                     ([1, 0, 0, 0, 0, 0, 1], [9, 0, 0, 50, 0, 0, 400])):
        w = Weighted(nq, lens, heads, causal, sum(lens) + heads[0])
        before = w.before.to(DEV)
        w.check(fa.fa_kv_weights(*w.args(), before, **w.opts()), w.before)
        w.check(fa.fa_kv_weights(*w.args(), before, out=before, **w.opts()), w.before)
        assert fa.fa_get_error() == fa.FA_OK


@pytest.mark.parametrize("d", [64, 128])
def test_weights_time_out_and_recover(d, monkeypatch):
    """Waits of the pipeline that run out end the kernel, the call reports it, and the next call is
    right again (no fault, nothing left behind)."""
    w = Weighted([200, 90], [1500, 700], (4, 2, d, 32), True, 3)
    args, opts = w.args(), w.opts()
    monkeypatch.setenv("FA_WAIT_TIMEOUT_US", "1")
    fa.fa_kv_weights(*args, **opts)
    status = fa.fa_get_error()
    monkeypatch.delenv("FA_WAIT_TIMEOUT_US")
    assert status == fa.FA_ERR_TIMEOUT, fa.fa_status_string(status)
    w.check(fa.fa_kv_weights(*args, **opts), None)
    assert fa.fa_get_error() == fa.FA_OK


def test_weights_of_large_logits_and_after_the_attention_call():
    w = Weighted([2, 1], [500, 300], (8, 2, 128, 16), True, 3, sigma=4.0)
    w.check(fa.fa_kv_weights(*w.args(), **w.opts()), None)
    # with the attention's own LSE the weights of a head's keys sum to its queries
    q, _, k, table, lens = w.args()
    _, lse = fa.fa_fwd_paged(q, k, w.cache.dev()[1], table, lens, **w.opts())
    got = fa.fa_kv_weights(q, lse, k, table, lens, **w.opts())
    sums = got.double().sum(2).cpu().numpy()
    np.testing.assert_allclose(sums, [[2 * 4] * 2, [4] * 2], rtol=2.0 ** -8)  # logits of up to 200


def test_weights_of_rows_without_keys_and_of_other_statistics():
    """LSE = -inf adds nothing, +inf neither, NaN shows."""
    w = Weighted([1, 1], [40, 50], (4, 2, 64, 16), False, 4)
    for value, ok in ((float("-inf"), True), (float("inf"), True), (float("nan"), False)):
        lse = w.lse.clone()
        lse[0, 0] = value
        q, _, k, table, lens = w.args()
        got = fa.fa_kv_weights(q, lse.to(DEV), k, table, lens, max_kv=50)
        lse[0, 0] = float("-inf")
        ref = fa.fa_kv_weights(q, lse.to(DEV), k, table, lens, max_kv=50)
        assert torch.equal(got[:, 1], ref[:, 1]) and torch.equal(got[1], ref[1])
        assert torch.equal(got[0, 0], ref[0, 0]) if ok else torch.all(got[0, 0, :40].isnan())


@pytest.mark.parametrize("causal", [False, True], ids=["all", "causal"])
@pytest.mark.parametrize("heads", [(8, 2, 128, 64), (4, 2, 64, 16)], ids=lambda h: "H%dkv%dd%dpage%d" % h)
def test_weights_of_queries_that_are_left_out(heads, causal):
    """A query whose LSE is -inf adds nothing whatever it holds, next to 32 and more that do."""
    w = Weighted([70, 9, 3], [900, 300, 70], heads, causal, 21)
    out = [3, 33, 65, 70, 79, 80, 81]
    w.lse[:, out] = float("-inf")
    w.q[out] = 0.0
    before = w.before.to(DEV)
    want = fa.fa_kv_weights(*w.args(), before, **w.opts())
    w.check(want, w.before)
    for odd in (float("nan"), float("inf"), -float("inf"), 3e38):
        w.q[out] = odd
        assert torch.equal(fa.fa_kv_weights(*w.args(), before, **w.opts()), want)
    assert fa.fa_get_error() == fa.FA_OK


def test_weights_of_a_wide_array():
    """Columns far past the keys keep what they have, in place or not, and are zeros without weights."""
    w = Weighted([1, 3, 0], [700, 40, 9], (8, 2, 128, 64), True, 22)
    w.before = torch.exp(torch.randn(3, 2, 100003, generator=torch.Generator().manual_seed(22)))
    before = w.before.to(DEV)
    w.check(fa.fa_kv_weights(*w.args(), before, **w.opts()), w.before)
    out = torch.full_like(before, float("nan"))
    w.check(fa.fa_kv_weights(*w.args(), out=out, **w.opts()), None)
    w.check(fa.fa_kv_weights(*w.args(), before, out=before, **w.opts()), w.before)


def test_weights_repeat_in_a_graph_and_on_another_stream():
    w = Weighted([20, 3], [900, 400], (8, 2, 128, 64), True, 5)
    args, opts = w.args(), w.opts()
    want = fa.fa_kv_weights(*args, **opts)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = fa.fa_kv_weights(*args, **opts)
    got.zero_()
    g.replay()
    assert torch.equal(got, want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = fa.fa_kv_weights(*args, stream=side, **opts)
    side.synchronize()
    assert torch.equal(other, want)


def test_weights_out_of_range():
    w = Weighted([1, 1], [40, 50], (4, 2, 64, 16), False, 6)
    q, lse, k, table, lens = w.args()
    out = torch.full((2, 2, 45), 2.0, device=DEV)  # the second sequence has more keys than columns
    got = fa.fa_kv_weights(q, lse, k, table, lens, out)
    assert fa.fa_get_error() == fa.FA_ERR_INDEX and torch.all(got[0, :, 40:] == 2) and torch.all(got[1] > 2)
    wild = torch.full_like(table, 77)
    got = fa.fa_kv_weights(q, lse, k, wild, lens, max_kv=50)
    assert fa.fa_get_error() == fa.FA_ERR_INDEX and torch.all(got.isfinite())
    for cu in ([0, 1, 9], [2, 1, 0], [-4, 9, 1]):
        fa.fa_kv_weights(q, lse, k, table, lens, cu_seqlens=i32(cu), max_q=2, max_kv=50)
    fa.fa_get_error()
    for bad in (lse.t().contiguous(), lse.double(), lse.cpu()):
        with pytest.raises(ValueError):
            fa.fa_kv_weights(q, bad, k, table, lens)
    with pytest.raises(ValueError):
        fa.fa_kv_weights(q, lse, k, table, lens, torch.zeros(2, 1, 50, device=DEV))
    with pytest.raises(ValueError):
        fa.fa_kv_weights(q, lse, k, table, lens, torch.zeros(2, 2, 50, device=DEV), out=torch.zeros(2, 2, 51, device=DEV))


# ---------------------------------------------------------------------------------------- eviction
class Evicted:
    """A cache whose pool has shuffled new pages as well."""

    def __init__(self, lens, Hkv, d, page, budget, seed, weights=None):
        g = torch.Generator().manual_seed(seed)
        keep = [min(n, budget) for n in lens]
        both = Cache(list(lens) + keep, Hkv, d, page, seed)
        self.pages = both.k.shape[0]
        B = len(lens)
        width = max(1, max(-(-n // page) for n in lens)), max(1, max(-(-n // page) for n in keep))
        self.table, self.new = both.table[:B, :width[0]].contiguous(), both.table[B:, :width[1]].contiguous()
        self.cache, self.lens, self.page, self.budget = both, list(lens), page, budget
        self.w = torch.exp(2 * torch.randn(B, Hkv, max(max(lens), 1) + 2, generator=g)) if weights is None else weights
        self.Hkv = Hkv

    def run(self, recent, **kw):
        self.k, self.v = self.cache.k.to(DEV), self.cache.v.to(DEV)
        for b in range(len(self.lens)):  # the new pages hold nothing
            for p in self.new[b].tolist():
                if p >= 0:
                    self.k[p] = self.v[p] = float("nan")
        self.k0, self.v0 = self.k.clone(), self.v.clone()
        return fa.fa_kv_evict(self.w.to(DEV), self.k, self.v, self.table.to(DEV), i32(self.lens), self.new.to(DEV),
                              self.budget, recent, **kw)

    def check(self, recent, **kw):
        lens, kept, left = self.run(recent, **kw)
        assert fa.fa_get_error() == fa.FA_OK
        ref = [self.k0.clone(), self.v0.clone()]
        assert lens.tolist() == [min(n, self.budget) for n in self.lens]
        for b, n in enumerate(self.lens):
            for h in range(self.Hkv):
                pick = evict(self.w[b, h].double().numpy(), n, self.budget, recent)
                m = len(pick)
                assert kept[b, h].tolist() == pick.tolist() + [-1] * (self.budget - m), (b, h)
                got = left[b, h].cpu()
                assert torch.equal(got[:m].nan_to_num(7), self.w[b, h, pick].nan_to_num(7)) and torch.all(got[m:] == 0)
                src, dst = torch.from_numpy(pick).long(), torch.arange(m)
                sp, dp = self.table[b].long()[src // self.page].to(DEV), self.new[b].long()[dst // self.page].to(DEV)
                so, do = (src % self.page).to(DEV), (dst % self.page).to(DEV)
                for x, x0 in zip(ref, (self.k0, self.v0)):
                    x[dp, h, do] = x0[sp, h, so]
        bits = lambda t: t.view(torch.int16)  # noqa: E731
        assert torch.equal(bits(self.k), bits(ref[0])) and torch.equal(bits(self.v), bits(ref[1]))
        return lens, kept, left


@pytest.mark.parametrize("shape", [(1, 64, 16), (2, 128, 64), (4, 64, 128), (3, 128, 32)], ids=str)
@pytest.mark.parametrize("lens,budget", [([1], 1), ([10, 0, 100], 40), ([1500, 3, 700, 701], 700), ([5000], 17),
                                         ([2049, 1025], 1024)], ids=str)
def test_evict(lens, budget, shape):
    for recent in sorted({0, 1, budget // 3, budget}):
        Evicted(lens, *shape, budget, sum(lens) + recent).check(recent)


@pytest.mark.parametrize("n", [4096, 4097, 16384, 16385, 40000, 70001, 131072, 131073, 200001])
def test_evict_of_a_long_sequence(n):
    """A CTA's registers, a cluster's, and more than a cluster holds; next to a short sequence."""
    for budget, recent in ((9, 3), (n // 5, 100), (n - 2, 5)):
        Evicted([n, 50], 1, 64, 16, budget, n + budget).check(min(recent, budget), max_kv=n)
    few = torch.randint(0, 3, (1, 1, n), generator=torch.Generator().manual_seed(n)).float()
    Evicted([n], 1, 64, 16, n // 2, n, few).check(0)  # ties all along


def test_evict_of_equal_zero_and_odd_weights():
    """Ties keep the earlier key; zeros of both signs are equal; NaN and infinities are the largest."""
    g = torch.Generator().manual_seed(3)
    n = 3000
    cases = [torch.ones(1, 2, n), torch.zeros(1, 2, n), torch.randint(0, 4, (1, 2, n), generator=g).float(),
             torch.randn(1, 2, n, generator=g), 1 + 2.0 ** -23 * torch.randint(0, 3, (1, 2, n), generator=g).float(),
             torch.exp(30 * torch.randn(1, 2, n, generator=g))]
    signed = torch.zeros(1, 2, n)
    signed[..., ::2] = -0.0
    odd = torch.randn(1, 2, n, generator=g)
    odd[0, 0, 5:900:7] = float("nan")
    odd[0, 1, 3:800:9] = float("inf")
    odd[0, :, 4:800:11] = float("-inf")
    mixed = odd.clone()
    mixed[0, :, 6:700:5], mixed[0, :, 2:900:8] = float("inf"), float("nan")
    for w in cases + [signed, odd, mixed]:
        for budget in (1, 100, 1500, 2999):
            Evicted([n], 2, 64, 16, budget, 4, w).check(min(10, budget))


def test_evict_repeats_in_a_graph_and_on_another_stream():
    e = Evicted([900, 2000], 2, 128, 64, 300, 5)
    want = e.check(30)
    k, v = e.k0.clone(), e.v0.clone()
    args = (e.w.to(DEV), k, v, e.table.to(DEV), i32(e.lens), e.new.to(DEV), 300, 30)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = fa.fa_kv_evict(*args)
    for t in got:
        t.zero_()
    g.replay()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert torch.equal(k.view(torch.int16), e.k.view(torch.int16))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = fa.fa_kv_evict(*args, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_evict_of_a_long_sequence_in_a_graph():
    """A launch of clusters, captured and replayed for other weights and lengths."""
    e = Evicted([40000, 9000], 2, 64, 16, 1500, 15)
    e.check(100)
    args = (e.w.to(DEV), e.k0.clone(), e.v0.clone(), e.table.to(DEV), i32(e.lens), e.new.to(DEV), 1500, 100)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = fa.fa_kv_evict(*args)
    args[0].copy_(args[0].flip(2))
    args[4].copy_(i32([39990, 1200]))
    g.replay()
    want = fa.fa_kv_evict(*args)
    assert all(torch.equal(x, y) for x, y in zip(got, want)) and got[0].tolist() == [1500, 1200]
    assert fa.fa_get_error() == fa.FA_OK


def test_calls_on_two_streams_at_once():
    """Nothing is shared between calls: each has its own outputs and workspaces."""
    e, f = Evicted([3000, 700], 2, 64, 16, 300, 16), Evicted([20000], 2, 64, 16, 900, 17)
    want = [[t.clone() for t in x.check(20)] for x in (e, f)]
    w = Weighted([40, 3], [3000, 900], (8, 2, 64, 32), True, 18)
    a, o = w.args(), w.opts()
    ref = fa.fa_kv_weights(*a, **o)
    args = [(x.w.to(DEV), x.k, x.v, x.table.to(DEV), i32(x.lens), x.new.to(DEV), x.budget, 20) for x in (e, f)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got.append([fa.fa_kv_evict(*args[0], stream=streams[0]), fa.fa_kv_evict(*args[1], stream=streams[1]),
                    fa.fa_kv_weights(*a, **o, stream=streams[2])])
    torch.cuda.synchronize()
    for x, y, z in got:
        assert all(torch.equal(p, q) for p, q in zip(x, want[0])) and all(torch.equal(p, q) for p, q in zip(y, want[1]))
        assert torch.equal(z, ref)


def test_evict_out_of_range_and_refusals():
    e = Evicted([100, 60], 2, 64, 16, 32, 6)
    e.run(4)
    args = [e.w.to(DEV), e.k, e.v, e.table.to(DEV), i32(e.lens), e.new.to(DEV), 32, 4]
    # pages outside the pool are not written, or read as zeros; lengths past the columns are clamped
    wild = list(args)
    wild[5] = torch.full_like(args[5], 999)
    before = e.k.clone()
    fa.fa_kv_evict(*wild)
    assert fa.fa_get_error() == fa.FA_ERR_INDEX and torch.equal(e.k.view(torch.int16), before.view(torch.int16))
    wild = list(args)
    wild[3] = torch.full_like(args[3], -7)
    fa.fa_kv_evict(*wild)
    assert fa.fa_get_error() == fa.FA_ERR_INDEX and torch.all(e.k[e.new[0, 0].item()] == 0)
    wild = list(args)
    wild[4] = i32([1 << 30, -5])
    lens, kept, _ = fa.fa_kv_evict(*wild)
    assert fa.fa_get_error() == fa.FA_ERR_INDEX and lens.tolist() == [32, 0] and torch.all(kept[1] == -1)
    assert kept.max().item() < 102
    for at, bad in ((0, args[0].double()), (0, args[0][:, :1].contiguous()), (5, args[5][:, :1].contiguous()),
                    (5, args[5].long()), (6, 0), (7, 33), (7, -1), (2, e.v.float())):
        wrong = list(args)
        wrong[at] = bad
        with pytest.raises((ValueError, fa.FAError)):
            fa.fa_kv_evict(*wrong)


def test_evict_to_pages_for_the_keys_that_there_are():
    """No more keys are kept than the weights have columns for, however far the block table and the
    budget reach."""
    e = Evicted([100, 60], 2, 64, 16, 200, 23)
    e.table = torch.cat([e.table, torch.full((2, 13), -1, dtype=torch.int32)], 1).contiguous()  # 320 keys
    assert e.w.shape[2] == 102 and e.new.shape[1] == 7  # 112 keys
    e.check(10)
    e.new = e.new[:, :6].contiguous()
    with pytest.raises(ValueError):
        e.run(10)


# ------------------------------------------------------------------------------- as it is used
def test_weights_eviction_and_decoding_on():
    """Weights gathered over steps, an eviction, and attention over what is left: as plain attention
    over the kept keys, whose rotation is that of their first places; then on from there."""
    H, Hkv, d, page, budget = 8, 2, 64, 16, 48
    lens, steps = [100, 60], 6
    g = torch.Generator().manual_seed(9)
    cache = Cache([140, 140, 80, 80], Hkv, d, page, 10)
    kc, vc, table, _ = cache.dev()
    old, new = table[:2], table[2:, :5].contiguous()
    rope = fa.fa_rope_table(256, d, device=DEV)
    weights = torch.zeros(2, Hkv, 140, device=DEV)

    def token():
        x = torch.randn(2, H + 2 * Hkv, d, generator=g).to(BF16).to(DEV)
        return x.split([H, Hkv, Hkv], dim=1)

    for _ in range(steps):
        lens = [n + 1 for n in lens]
        q, k, v = token()
        q = fa.fa_kv_append(q, k, v, kc, vc, old, i32(lens), table=rope)
        o, lse = fa.fa_fwd_paged(q, kc, vc, old, i32(lens), max_kv=max(lens))
        fa.fa_kv_weights(q, lse, kc, old, i32(lens), weights, out=weights, max_kv=max(lens))
    sums = weights.double().sum(2).cpu().numpy()
    np.testing.assert_allclose(sums, steps * H / Hkv, rtol=2.0 ** -11)
    K, V = f64(kc), f64(vc)
    new_lens, kept, left = fa.fa_kv_evict(weights, kc, vc, old, i32(lens), new, budget, 8)
    assert new_lens.tolist() == [48, 48] and fa.fa_get_error() == fa.FA_OK
    offset = i32(lens) - new_lens
    q, k, v = token()
    q = fa.fa_kv_append(q, k, v, kc, vc, new, new_lens + 1, pos_offset=offset, table=rope)
    o, lse = fa.fa_fwd_paged(q, kc, vc, new, new_lens + 1, max_kv=budget + 1)
    assert fa.fa_get_error() == fa.FA_OK
    kn, vn = f64(kc), f64(vc)
    for b in range(2):
        for h in range(H):
            hk = h // (H // Hkv)
            src = kept[b, hk].cpu().numpy()
            kk = [K[old[b, j // page].item(), hk, j % page] for j in src]
            vv = [V[old[b, j // page].item(), hk, j % page] for j in src]
            at = new[b, budget // page].item(), hk, budget % page
            kk, vv = np.stack(kk + [kn[at]]), np.stack(vv + [vn[at]])
            O, L, A, _ = attend(f64(q[b:b + 1, h:h + 1]), kk[None], vv[None], d ** -0.5, [budget + 1])
            assert np.all(np.abs(f64(o[b, h]) - O[0, 0]) <= (2.0 ** -8 + 2.0 ** -14) * A[0, 0] + 2.0 ** -8 * np.abs(O[0, 0]))


def test_decoding_on_after_an_eviction():
    """An eviction of keys whose pages are selected: the new pages' bounds, the weights in their wider
    array, and steps of appending, selecting, attending and gathering from there, as the reference."""
    H, Hkv, d, page, budget, top, steps = 8, 2, 64, 16, 70, 3, 12
    lens = [150, 40, 99]
    kept_lens = [min(n, budget) for n in lens]
    g = torch.Generator().manual_seed(12)
    cache = Cache([*lens, *(n + steps for n in kept_lens)], Hkv, d, page, 13)
    kc, vc, table, _ = cache.dev()
    new_table = table[3:, :-(-(budget + steps) // page)].contiguous()
    bounds = torch.full((kc.shape[0], Hkv, 2, d), float("nan"), dtype=BF16, device=DEV)
    weights = torch.rand(3, Hkv, 160, generator=g).to(DEV)
    block_table, kv_lens = table[:3].contiguous(), i32(lens)
    new_lens, kept, new_weights = fa.fa_kv_evict(weights, kc, vc, block_table, kv_lens, new_table, budget, 9)
    pos_offset = kv_lens - new_lens
    block_table, kv_lens = new_table, new_lens
    weights.zero_()
    weights[:, :, :budget] = new_weights
    cu = torch.nn.functional.pad(kv_lens.cumsum(0, dtype=torch.int32), (1, 0))
    fa.fa_page_bounds(kc, block_table, kv_lens, bounds, cu_seqlens=cu)
    rope = fa.fa_rope_table(256, d, device=DEV)
    want, err = f64(weights), np.zeros(weights.shape)
    for step in range(steps):
        kv_lens = kv_lens + 1
        x = torch.randn(3, H + 2 * Hkv, d, generator=g).to(BF16).to(DEV)
        q, k, v = x.split([H, Hkv, Hkv], dim=1)
        q = fa.fa_kv_append(q, k, v, kc, vc, block_table, kv_lens, pos_offset=pos_offset, table=rope)
        fa.fa_page_bounds(kc, block_table, kv_lens, bounds)
        pages = fa.fa_select_pages(q, bounds, block_table, kv_lens, page, top)
        fa.fa_fwd_paged_selected(q, kc, vc, block_table, kv_lens, pages)
        o, lse = fa.fa_fwd_paged(q, kc, vc, block_table, kv_lens)
        fa.fa_kv_weights(q, lse, kc, block_table, kv_lens, weights, out=weights)
        assert fa.fa_get_error() == fa.FA_OK
        pool = f64(kc)
        for b, n in enumerate(kv_lens.tolist()):
            at = [(block_table[b, j // page].item(), j % page) for j in range(n)]
            K = np.stack([pool[p, :, r] for p, r in at], 1)
            score = page_scores(f64(q[b]), *page_bounds(K, page))
            for h in range(Hkv):
                pick = select_pages(score[h], -(-n // page), top, 1, 1).tolist()
                assert pages[b, h].tolist() == pick + [-1] * (top - len(pick))
            w, e = key_weights(f64(q[b:b + 1]), K, d ** -0.5, f64(lse[:, b:b + 1].T), [n])
            want[b, :, :n] += w
            err[b, :, :n] += 2.0 ** -24 * (d + 24 + H // Hkv) * e
    # the terms' errors, and a rounding of the whole a step
    assert np.all(np.abs(f64(weights) - want) <= err + 2.0 ** -23 * steps * want)
