"""Attention of trees of drafted tokens over the paged cache (fa_tree_mask, fa_fwd_paged_tree)
against the fp64 reference.  Tolerances: those of the paged attention (test_paged_gpu.py)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import exact_io_aware_fwd_gb300 as fa
from oracle.serving import attend_where, norm_rope, tree_sees
from test_paged_gpu import Cache, _built, cumulative, f64, i32  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16


def random_parents(n, rng, roots=0.1):
    return [-1 if i == 0 or rng.random() < roots else int(rng.integers(max(0, i - 8), i)) for i in range(n)]


def pack(rows, words):
    """int64 [t, words] of boolean rows [t, any]."""
    bits = np.zeros((len(rows), words * 64), dtype=np.uint8)
    for i, r in enumerate(rows):
        bits[i, :min(len(r), words * 64)] = r[:words * 64]
    return torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int64).reshape(-1, words))


def seen_by(rows, n, length):
    """[n, 1, length]: the context, and the new tokens of each row (new token j is key length - n + j)."""
    seen = np.zeros((n, 1, length), dtype=bool)
    for i in range(n):
        for key in range(length):
            j = key - (length - n)
            seen[i, 0, key] = j < 0 or (j < len(rows[i]) and rows[i][j])
    return seen


def check(out, lse, q, cu, per_seq, scale):
    """per_seq: (K, V, seen) of each sequence; the bounds of test_paged_gpu.check."""
    out, lse, q = f64(out), f64(lse), f64(q)
    d = q.shape[-1]
    for b, (K, V, seen) in enumerate(per_seq):
        a, e = cu[b], cu[b + 1]
        if a == e:
            continue
        O, L, A, size = attend_where(q[a:e], K, V, scale, seen)
        excess = np.abs(out[a:e] - O) - ((2.0 ** -8 + 2.0 ** -14) * A + 2.0 ** -8 * np.abs(O))
        assert np.all(excess <= 1e-30), (b, float(excess.max()))
        got, fin = lse[:, a:e].T, np.isfinite(L)
        assert np.array_equal(np.isfinite(got), fin) and np.all(got[~fin] == L[~fin]), b
        bound = 2.0 ** -24 * (d + 16) * size + 2.0 ** -20 * (1 + np.abs(np.where(fin, L, 0)))
        assert np.all(np.abs(got[fin] - L[fin]) <= bound[fin]), b


def run(nq, lens, heads, seed, rows=None, words=None, scale=None, sigma=1.0, **kw):
    H, Hkv, d, page = heads
    rng = np.random.default_rng(seed)
    cache = Cache(lens, Hkv, d, page, seed, sigma)
    cu = cumulative(nq)
    g = torch.Generator().manual_seed(seed + 1)
    q = (sigma * torch.randn(cu[-1], H, d, generator=g)).to(BF16)
    rows = rows or [tree_sees(random_parents(n, rng)) for n in nq]
    words = words or -(-max(nq) // 64)
    mask = torch.cat([pack(r, words) for r in rows if len(r)])
    args = dict(cu_seqlens=i32(cu), max_q=max(nq), max_kv=max(lens), scale=scale)
    args.update(kw)
    out, lse = fa.fa_fwd_paged_tree(q.to(DEV), *cache.dev(), mask.to(DEV), **args)
    assert fa.fa_get_error() == fa.FA_OK
    per = [(*cache.keys(b), seen_by([r[:words * 64] for r in rows[b]], nq[b], lens[b])) for b in range(len(lens))]
    check(out, lse, q, cu, per, d ** -0.5 if scale is None else scale)
    return cache, q, mask, out, lse


@pytest.mark.parametrize("heads", [(1, 1, 64, 16), (8, 2, 128, 64), (6, 2, 64, 32), (5, 1, 128, 128)],
                         ids=lambda h: "H%dkv%dd%dpage%d" % h)
@pytest.mark.parametrize("lengths", [
    ([1], [1]), ([1], [40]), ([3], [3]), ([2, 1, 4], [2, 17, 64]),        # few rows, whole segments
    ([4, 2], [2, 0]),                                                     # more tokens than keys
    ([3, 0, 4], [2500, 3, 1300]),                                         # split over the keys
    ([16, 7], [200, 1100]), ([26], [1000]), ([64, 33], [64, 1500]),       # more rows
    ([65, 1, 130], [900, 31, 130]), ([200], [1700]),                      # several words, two query tiles
], ids=lambda x: "-".join("%dof%d" % p for p in zip(*x)))
def test_tree(lengths, heads):
    for kw in (dict(), dict(max_kv=4000)):  # as they are, and too long for whole segments a CTA
        run(*lengths, heads, seed=sum(lengths[1]) + heads[0], **kw)


@pytest.mark.parametrize("heads", [(4, 2, 128, 16), (32, 1, 64, 64)], ids=lambda h: "H%dkv%dd%dpage%d" % h)
def test_masks_that_are_no_trees(heads):
    """Rows of zeros (with a context and without), rows that see later tokens, bits of tokens that do
    not exist, and fewer words than tokens."""
    rng = np.random.default_rng(3)
    for nq, lens in (([5, 3], [5, 300]), ([70, 9], [70, 900])):
        rows = [rng.random((n, n)) < 0.4 for n in nq]
        for r in rows:
            r[0] = False
            r[-1] = True
        run(nq, lens, heads, 5, rows)
        run(nq, lens, heads, 6, [np.concatenate([r, np.ones_like(r)], 1) for r in rows], words=3)
    run([70], [400], heads, 7, [rng.random((70, 70)) < 0.5], words=1)


def test_hidden_scores_of_any_size():
    """Large logits in front of and behind what a row sees, and a scale of 0."""
    run([9], [300], (4, 1, 128, 32), 8, sigma=6.0)
    run([9], [300], (4, 1, 128, 32), 8, scale=0.0)


def test_a_chain_is_causal_attention():
    nq, lens, heads = [7, 40, 1], [900, 1300, 77], (8, 2, 128, 64)
    chain = [np.tri(n, dtype=bool) for n in nq]
    cache, q, mask, out, lse = run(nq, lens, heads, 11, chain)
    ref, ref_lse = fa.fa_fwd_paged(q.to(DEV), *cache.dev(), cu_seqlens=i32(cumulative(nq)), max_q=40,
                                   max_kv=1300, causal=True)
    # both within the bounds of check(): sum p|v| and |O| are at most the largest |v|
    most = float(cache.v.nan_to_num(0).abs().max())
    assert float((out.float() - ref.float()).abs().max()) <= 2 * (2.0 ** -7 + 2.0 ** -14) * most
    assert float((lse - ref_lse).abs().max()) <= 2.0 ** -11


def test_bits_agree_from_run_to_run_and_in_a_graph():
    nq, lens, heads = [48, 64, 3], [3000, 5000, 64], (8, 2, 128, 64)
    cache, q, mask, out, lse = run(nq, lens, heads, 12)
    args = (q.to(DEV), *cache.dev(), mask.to(DEV))
    opts = dict(cu_seqlens=i32(cumulative(nq)), max_q=64, max_kv=5000)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o2, l2 = fa.fa_fwd_paged_tree(*args, **opts)
    o2.zero_()
    for _ in range(3):
        g.replay()
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    # the replay reads the mask and lengths that the tensors then hold
    args[5].fill_(-1)
    g.replay()
    o3, l3 = fa.fa_fwd_paged_tree(*args, **opts)
    assert torch.equal(o2, o3) and torch.equal(l2, l3) and not torch.equal(l2, lse)
    assert fa.fa_get_error() == fa.FA_OK


def test_another_stream_and_given_outputs():
    nq, lens, heads = [20, 9], [500, 800], (4, 2, 64, 32)
    cache, q, mask, out, lse = run(nq, lens, heads, 13)
    s = torch.cuda.Stream()
    args = [t.contiguous() for t in (q.to(DEV), *cache.dev(), mask.to(DEV))]
    torch.cuda.synchronize()
    o, l2 = torch.full_like(out, 7), torch.full_like(lse, 7)
    ws = torch.empty(fa.fa_fwd_paged_workspace_size(2, 29, 4, 2, 64), dtype=torch.uint8, device=DEV)
    got = fa.fa_fwd_paged_tree(*args, cu_seqlens=i32(cumulative(nq)), max_q=20, max_kv=800, out=o, lse=l2,
                               workspace=ws, stream=s)
    s.synchronize()
    assert got[0] is o or got[0].data_ptr() == o.data_ptr()
    assert torch.equal(o, out) and torch.equal(l2, lse)


def test_tokens_behind_the_last_sequence_stay():
    nq, lens, heads = [3, 4], [50, 60], (4, 2, 64, 16)
    cache, q, mask, out, lse = run(nq, lens, heads, 14)
    more = torch.cat([q, q[:2]]).to(DEV)
    o, l2 = torch.full((9, 4, 64), 3.0, dtype=BF16, device=DEV), torch.full((4, 9), 3.0, device=DEV)
    fa.fa_fwd_paged_tree(more, *cache.dev(), torch.cat([mask, mask[:2]]).to(DEV), cu_seqlens=i32([0, 3, 7]),
                         max_q=4, max_kv=60, out=o, lse=l2)
    assert torch.equal(o[:7], out) and torch.all(o[7:] == 3) and torch.all(l2[:, 7:] == 3)
    assert fa.fa_get_error() == fa.FA_OK


# ------------------------------------------------------------------------------------------- masks
@pytest.mark.parametrize("nq", [[1], [5, 0, 1, 64], [65, 3, 200], [0, 0, 33]], ids=str)
def test_tree_mask(nq):
    rng = np.random.default_rng(sum(nq))
    parents = [random_parents(n, rng) for n in nq]
    flat = i32([p for seq in parents for p in seq])
    for words in {-(-max(nq) // 64), 4}:
        ref = torch.cat([pack(tree_sees(p), words) for p in parents if p])
        got = fa.fa_tree_mask(flat, i32(cumulative(nq)), max_q=64 * words)
        assert torch.equal(got.cpu(), ref)
    assert fa.fa_get_error() == fa.FA_OK
    single = fa.fa_tree_mask(torch.full((5,), -1, dtype=torch.int32, device=DEV))
    assert torch.equal(single.cpu(), torch.ones(5, 1, dtype=torch.int64))


def test_tree_mask_of_parents_that_are_none():
    """A parent that is not in front of its token ends the branch; a token without a bit is left out."""
    got = fa.fa_tree_mask(i32([-1, 0, 2, -7, 9]), i32([0, 5]), max_q=5)
    assert got.flatten().tolist() == [1, 3, 4, 8, 16]
    assert fa.fa_get_error() == fa.FA_ERR_INDEX
    chain = i32([i - 1 for i in range(66)])
    got = fa.fa_tree_mask(chain, i32([0, 66]), max_q=64)
    assert got[65].item() == got[63].item() == -1 and fa.fa_get_error() == fa.FA_ERR_INDEX
    # tokens outside every sequence keep their rows
    out = torch.full((6, 1), 77, dtype=torch.int64, device=DEV)
    fa.fa_tree_mask(i32([0, -1, 0, -1, 0, 0]), i32([1, 3, 5]), max_q=2, out=out)
    assert out.flatten().tolist() == [77, 1, 3, 1, 3, 77]
    assert fa.fa_get_error() == fa.FA_OK


# ------------------------------------------------------------------------------- as it is used
def test_drafting_and_verifying_as_one_token_at_a_time():
    """A draft of a tree, its attention, and the accepted branch appended: each node's output is what
    decoding its branch one token at a time would give, and so is the cache after acceptance."""
    H, Hkv, d, page, ctx = 8, 2, 64, 16, 37
    g = torch.Generator().manual_seed(21)
    freq, _ = fa.rope_frequencies(d)
    table = fa.fa_rope_table(128, d, device=DEV)
    parents = [-1, -1, 0, 0, 2, 1, 4]
    depth = []
    for p in parents:
        depth.append(0 if p < 0 else depth[p] + 1)
    n = len(parents)
    x = torch.randn(ctx + n, H + 2 * Hkv, d, generator=g).to(BF16).to(DEV)
    q, k, v = x.split([H, Hkv, Hkv], dim=1)
    kc, vc = (torch.full((6, Hkv, page, d), float("nan"), dtype=BF16, device=DEV) for _ in range(2))
    blocks, cu = i32([[3, 0, 5, 1]]), i32([0, n])
    fa.fa_kv_append(q[:ctx], k[:ctx], v[:ctx], kc, vc, blocks, i32([ctx]), cu_seqlens=i32([0, ctx]), table=table)
    # the draft: rotated by depth, stored behind the context
    pos = i32([ctx + e for e in depth])
    qd, kd, vd = fa.fa_qk_norm_rope_fwd(q[ctx:], k[ctx:], v[ctx:], table=table, positions=pos)
    lens = i32([ctx + n])
    fa.fa_kv_append(None, kd, vd, kc, vc, blocks, lens, cu_seqlens=cu)
    mask = fa.fa_tree_mask(i32(parents), cu, max_q=n)
    o, lse = fa.fa_fwd_paged_tree(qd, kc, vc, blocks, lens, mask, cu_seqlens=cu, max_q=n, max_kv=ctx + n)
    assert fa.fa_get_error() == fa.FA_OK
    all_pos = np.concatenate([np.arange(ctx), ctx + np.array(depth)])
    to = lambda t: torch.tensor(t).to(BF16).double().numpy()  # noqa: E731
    K = to(norm_rope(f64(k), all_pos, inv_freq=f64(freq))).transpose(1, 0, 2)
    Q = to(norm_rope(f64(q), all_pos, inv_freq=f64(freq)))
    V = f64(v).transpose(1, 0, 2)
    seen = np.concatenate([np.ones((n, ctx), bool), tree_sees(parents)], 1)[:, None]
    ref = attend_where(Q[ctx:], K, V, d ** -0.5, seen)[0]
    # 2^-8 of sum p|v| (three times |O| here) and of |O|; rotated rows a rounding apart now and then
    assert np.linalg.norm(f64(o) - ref) <= 2.0 ** -5 * np.linalg.norm(ref)
    # the branch 0, 2, 4, 6 is accepted: its keys and values go behind the context, in order
    path = [0, 2, 4, 6]
    idx = torch.tensor([ctx + i for i in path], device=DEV)
    new = i32([ctx + len(path)])
    qa = fa.fa_kv_append(q[idx].contiguous(), k[idx].contiguous(), v[idx].contiguous(), kc, vc, blocks, new,
                         cu_seqlens=i32([0, len(path)]), table=table)
    oa, la = fa.fa_fwd_paged(qa, kc, vc, blocks, new, cu_seqlens=i32([0, len(path)]), max_q=len(path),
                             max_kv=ctx + len(path), causal=True)
    assert fa.fa_get_error() == fa.FA_OK
    # the same keys, but other tiles and another order of the sums
    assert torch.allclose(la, lse[:, path], atol=2.0 ** -12)
    assert np.linalg.norm(f64(oa) - f64(o)[path]) <= 2.0 ** -5 * np.linalg.norm(f64(o)[path])


def test_lengths_pages_and_offsets_out_of_range_are_reported():
    H, Hkv, d, page = 4, 2, 64, 16
    cache = Cache([40], Hkv, d, page, 30)
    q = torch.randn(3, H, d).to(BF16).to(DEV)
    mask = torch.ones(3, 1, dtype=torch.int64, device=DEV)
    kc, vc, table, _ = cache.dev()
    for lens, tab, cu in ((i32([400]), table, [0, 3]), (i32([40]), torch.full_like(table, 99), [0, 3]),
                          (i32([40]), table, [0, 5])):
        fa.fa_fwd_paged_tree(q, kc, vc, tab, lens, mask, cu_seqlens=i32(cu), max_q=3, max_kv=48)
        assert fa.fa_get_error() == fa.FA_ERR_INDEX


def test_refusals():
    cache = Cache([40], 2, 64, 16, 31)
    q = torch.randn(1, 4, 64).to(BF16).to(DEV)
    args = (q, *cache.dev())
    good = torch.ones(1, 1, dtype=torch.int64, device=DEV)
    fa.fa_fwd_paged_tree(*args, good)
    for bad in (good.int(), good.cpu(), good.flatten(), torch.ones(2, 1, dtype=torch.int64, device=DEV), None):
        with pytest.raises(ValueError):
            fa.fa_fwd_paged_tree(*args, bad)
    with pytest.raises(fa.FAError):
        fa.fa_fwd_paged_tree(*args, torch.ones(1, 0, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        fa.fa_tree_mask(torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        fa.fa_tree_mask(good)


# ------------------------------------------------------------- the largest weight (tensor-core kernel)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq", [5, 20])
def test_a_rows_largest_weight_is_not_rounded(nq, d):
    """One key outweighs the others, later than they come: 2^-7 of weight in each key tile, then a key
    128.5 times as heavy.  Every key has the same value, so O is that value.  Weights but the largest are
    off by 2^-8 of at most 11 / 128.5 of the sum, 2^-11.5, and float32 by 2^-14: less than the 2^-9 that
    a value of 255 / 128 times a power of two has to its next ones.  128.5 rounded to 8 bits is off by
    that much.  5 tokens of 8 heads a group are one query tile, 20 two."""
    H, Hkv, page, B, n = 32, 4, 16, 40, 1500
    cache = Cache([n] * B, Hkv, d, page, 40 + nq)
    keys = torch.zeros(n, d)
    keys[:, 0] = -30.0
    keys[5:1400:128, 0] = 0.0
    keys[1450, 0], keys[1450, 1] = 4.84375, float(np.log(128.5)) - 4.84375
    value = 1.9921875 * 2.0 ** torch.randint(-3, 3, (d,), generator=torch.Generator().manual_seed(d))
    for b in range(B):
        for i in range(-(-n // page)):
            p, part = int(cache.table[b, i]), keys[i * page:(i + 1) * page]
            cache.k[p, :, :len(part)] = part.to(BF16)
            cache.v[p, :, :len(part)] = value.to(BF16)
    q = torch.zeros(B * nq, H, d, dtype=BF16, device=DEV)
    q[:, :, :2] = 1.0
    mask = torch.cat([pack(np.tri(nq, dtype=bool), 1)] * B).to(DEV)
    out, _ = fa.fa_fwd_paged_tree(q, *cache.dev(), mask, cu_seqlens=i32([nq * b for b in range(B + 1)]), max_q=nq,
                                  max_kv=n, scale=1.0)
    assert fa.fa_get_error() == fa.FA_OK
    assert torch.equal(out, value.to(BF16).to(DEV).expand_as(out))


@pytest.mark.parametrize("sigma", [3.0, 6.0])
@pytest.mark.parametrize("heads", [(8, 2, 128, 64), (16, 2, 64, 16)], ids=lambda h: "H%dkv%dd%dpage%d" % h)
def test_large_logits_of_a_chain_as_those_of_a_causal_call(heads, sigma):
    """Both have the bound of check() without the largest weight, which is exactly 1: 2^-8 of the other
    weights times |v| and of |O|, and 2^-14 of sum p|v|; logits of up to 400 make exponents off by
    2^-24 (d + 16) sum|q k| scale, that is relative weights by as much."""
    H, Hkv, d, page = heads
    for nq, lens in (([6, 9], [2500, 1300]), ([40], [3000])):
        chain = [np.tri(n, dtype=bool) for n in nq]
        cache, q, mask, out, lse = run(nq, lens, heads, 50 + nq[0], chain, sigma=sigma)
        cu = cumulative(nq)
        ref, _ = fa.fa_fwd_paged(q.to(DEV), *cache.dev(), cu_seqlens=i32(cu), max_q=max(nq), max_kv=max(lens),
                                 causal=True)
        for b, n in enumerate(nq):
            K, V = cache.keys(b)
            for i in range(n):
                sees, qi = lens[b] - n + i + 1, f64(q[cu[b] + i])
                for h in range(H):
                    k, v = K[h * Hkv // H][:sees], V[h * Hkv // H][:sees]
                    s = k @ qi[h] * d ** -0.5
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    O, A, top = p @ v, p @ np.abs(v), int(p.argmax())
                    size = d ** -0.5 * float((np.abs(k) @ np.abs(qi[h])).max())
                    bound = (2.0 ** -8 * (A - p[top] * np.abs(v[top])) + 2.0 ** -8 * np.abs(O) +
                             (2.0 ** -14 + 2 * 2.0 ** -24 * (d + 16) * size) * (A + np.abs(O)))
                    for x in (out, ref):
                        assert np.all(np.abs(f64(x[cu[b] + i, h]) - O) <= bound), (b, i, h, x is out)
