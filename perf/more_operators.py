"""Workloads of what a serving program does with a paged key/value cache next to plain attention:
attention of trees of drafted tokens, attention over the pages that a cheap score selects for each
query (the pages' bounds, the selection, the attention), and eviction by accumulated attention
weight (the accumulation, the eviction).

``listed()`` and ``draw(rng)`` give cases; ``prepare(case, seed)`` makes what a program holds before
the call; ``run(state)`` is one pass, in elementary torch operations, or, where ``own`` is true,
through the package; ``exact(case, seed)`` is the definition in 64 bits; ``work(case)`` counts the
bytes and operations that a pass cannot do without.
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the smallest tree: a single user, 26 drafted tokens behind a short context
        dict(name="tree-1x26x1000", op="tree", B=1, nq=26, qlo=26, lo=1000, hi=1000, H=8, Hkv=8, d=64, page=16),
        # a serving batch that drafts 64 tokens a sequence, grouped-query
        dict(name="tree-32x64x8192-gqa", op="tree", B=32, nq=64, qlo=48, lo=2048, hi=8192, H=32, Hkv=8, d=128,
             page=64),
        # bounds of the pages that a decoding step of 64 sequences has written to
        dict(name="bounds-decode-64", op="bounds", B=64, nq=1, qlo=1, lo=512, hi=4096, Hkv=8, d=128, page=64),
        # bounds of all pages of a packed batch of prompts
        dict(name="bounds-prompt-16x4096", op="bounds", B=16, nq=4096, qlo=512, lo=4096, hi=4096, Hkv=16, d=128,
             page=16),
        # 32 of up to 256 pages for each query of a serving batch
        dict(name="select-64x16384-gqa", op="select", B=64, nq=1, qlo=1, lo=4096, hi=16384, H=32, Hkv=8, d=128,
             page=64, top=32, first=1, last=2),
        # 128 of 4096 pages: few long contexts
        dict(name="select-4x131072-gqa", op="select", B=4, nq=1, qlo=1, lo=100000, hi=131072, H=32, Hkv=8, d=128,
             page=32, top=128, first=1, last=4),
        # the attention over 2048 selected keys of each sequence and head of the serving batch
        dict(name="selected-64x16384-gqa", op="selected", B=64, nq=1, qlo=1, lo=4096, hi=16384, H=32, Hkv=8, d=128,
             page=64, top=32),
        # over 4096 keys of few long contexts: the work has to be split over the keys
        dict(name="selected-4x131072-gqa", op="selected", B=4, nq=1, qlo=1, lo=100000, hi=131072, H=32, Hkv=8,
             d=128, page=32, top=128),
        # attention weights of one decoding step of a serving batch, added to what the keys had
        dict(name="weights-64x4096-gqa", op="weights", B=64, nq=1, qlo=1, lo=512, hi=4096, H=32, Hkv=8, d=128,
             page=64),
        # the votes of a prompt's last 32 tokens for the keys to keep
        dict(name="weights-8x16384-window", op="weights", B=8, nq=32, qlo=32, lo=8192, hi=16384, H=32, Hkv=8, d=128,
             page=64),
        # a serving batch cut down to 1024 keys a sequence
        dict(name="evict-64x4096", op="evict", B=64, lo=512, hi=4096, Hkv=8, d=128, page=64, budget=1024,
             recent=128),
        # one long context cut down to an eighth
        dict(name="evict-1x131072", op="evict", B=1, lo=131072, hi=131072, Hkv=8, d=128, page=16, budget=16384,
             recent=1024),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "bounds", "select", "selected", "weights", "evict"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 3, 4, 8] if Hkv < 8 else [1, 4])
    page = rng.choice([16, 32, 64, 128])
    c = dict(op=op, H=H, Hkv=Hkv, d=d, page=page)
    if op == "tree":
        B = _log(rng, 1, 32)
        hi = _log(rng, 32, 262144 // max(B, 8))
        nq = _log(rng, 2, min(200, hi, max(2, (1 << 23) // (B * hi))))
        return dict(c, B=B, nq=nq, qlo=rng.randint(1, nq), lo=max(nq, hi // rng.choice([1, 2, 8])), hi=hi)
    if op == "bounds":
        B = _log(rng, 1, 128)
        nq = 1 if rng.random() < 0.5 else _log(rng, 2, max(2, 32768 // B))
        hi = nq + _log(rng, 1, 512)
        return dict(c, B=B, nq=nq, qlo=rng.randint(1, nq), lo=nq, hi=hi)
    if op in ("select", "selected"):
        B = _log(rng, 1, 64)
        hi = _log(rng, 64, 524288 // max(B, 4))
        nq = rng.choice([1, 1, 1, 2, 5])
        pages = -(-hi // page)
        top = max(2, min(_log(rng, 2, 128), 4096 // page, pages))
        c = dict(c, B=B, nq=nq, qlo=1, lo=max(nq, hi // rng.choice([1, 2, 8])), hi=hi + nq, top=top)
        if op == "select":
            first = rng.randint(0, min(2, top - 1))
            c.update(first=first, last=rng.randint(0, min(4, top - first - 1)))
        return c
    if op == "weights":
        B = _log(rng, 1, 64)
        nq = 1 if rng.random() < 0.5 else _log(rng, 2, 64)
        hi = nq + _log(rng, 1, 131072 // max(B, 8))
        return dict(c, B=B, nq=nq, qlo=rng.randint(1, nq), lo=max(nq, hi // rng.choice([1, 2, 8])), hi=hi)
    B = _log(rng, 1, 64)
    hi = _log(rng, 64, 131072 // B if B > 1 else 131072)
    budget = max(2, _log(rng, max(2, hi // 16), hi))
    return dict(c, B=B, lo=max(1, hi // rng.choice([1, 2, 8])), hi=hi, budget=budget,
                recent=rng.randint(0, budget // rng.choice([1, 2, 8])))


def _lengths(case):
    """The lengths of a case are part of it, not of its inputs: (new tokens, keys) of each sequence."""
    r = random.Random("%s %d %d %d" % (case["op"], case["B"], case["lo"], case["hi"]))
    B, top = case["B"], case.get("nq", 0)
    nq = [r.randint(case.get("qlo", 0), top) for _ in range(B)]
    nq[r.randrange(B)] = top
    kv = [max(n, r.randint(case["lo"], case["hi"])) for n in nq]
    kv[r.randrange(B)] = case["hi"]
    if case["op"] == "bounds" and case["lo"] == case["hi"]:  # prompts: all keys are new
        kv = list(nq)
    return nq, kv


def _parents(case):
    """A tree over each sequence's drafted tokens (-1: behind the context): wide at the top and
    thinner below, the shape of drafts that continue the likelier tokens."""
    r = random.Random("tree %d %d %d" % (case["B"], case["nq"], case["hi"]))
    out = []
    for n in _lengths(case)[0]:
        out.append([-1 if i == 0 or r.random() < 0.05 else min(i - 1, int(i * r.random() ** 1.5)) for i in range(n)])
    return out


def work(case):
    Hkv, d, page = case["Hkv"], case["d"], case["page"]
    nq, kv = _lengths(case)
    T, keys = sum(nq), sum(kv)
    if case["op"] == "bounds":
        read = written = 0
        for n, k in zip(nq, kv):
            first = (k - n) // page
            read += k - first * page
            written += -(-k // page) - first
        return {"bytes": Hkv * d * 2 * (read + 2 * written), "flops": 2 * read * Hkv * d}
    if case["op"] == "evict":
        kept = sum(min(k, case["budget"]) for k in kv)
        return {"bytes": Hkv * (4 * keys + kept * (2 * 2 * d * 2 + 8)), "flops": Hkv * keys}
    H = case["H"]
    io = 2 * T * H * d * 2 + T * H * 4
    if case["op"] == "tree":
        pairs = 0
        for n, k, parents in zip(nq, kv, _parents(case)):
            depth = []
            for p in parents:
                depth.append(1 if p < 0 else depth[p] + 1)
            pairs += n * (k - n) + sum(depth)
        return {"bytes": keys * Hkv * d * 2 * 2 + io + T * 8 * -(-case["nq"] // 64), "flops": 4 * pairs * H * d}
    if case["op"] == "weights":
        pairs = sum(n * k - n * (n - 1) // 2 for n, k in zip(nq, kv))
        return {"bytes": keys * Hkv * (d * 2 + 8) + T * H * (d * 2 + 4), "flops": 2 * pairs * H * d}
    pages = [-(-k // page) for k in kv]
    if case["op"] == "select":
        scored = sum(n * p for n, p in zip(nq, pages))
        return {"bytes": sum(pages) * Hkv * d * 2 * 2 + T * H * d * 2 + T * Hkv * case["top"] * 4,
                "flops": 4 * scored * H * d}
    # each token's keys, at most once for each page of a sequence however many tokens read it
    picked = sum(min(n * min(case["top"] * page, k), k) for n, k in zip(nq, kv))
    pairs = sum(n * min(case["top"] * page, k) for n, k in zip(nq, kv))
    return {"bytes": picked * Hkv * d * 2 * 2 + io + T * Hkv * case["top"] * 4, "flops": 4 * pairs * H * d}


# ------------------------------------------------------------------------------------------ inputs
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _tables(lens, page, g, first=0):
    """Block table of sequences of these lengths over shuffled pages first, first + 1, ... (-1 where
    there is no page), and how many pages that is."""
    need = [-(-n // page) for n in lens]
    total, width = sum(need), max(1, max(need))
    pages = (first + torch.randperm(total, generator=g, device=DEV)).to(torch.int32)
    inside = torch.arange(width, device=DEV)[None] < torch.tensor(need, device=DEV)[:, None]
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    table[inside] = pages
    return table, total


def _visible(s):
    """(sequence, index among its new tokens, keys it sees) of each packed token."""
    n = s["cu"].diff().long()
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=DEV), n, output_size=s["T"])
    i = torch.arange(s["T"], device=DEV) - s["cu"].long()[seq]
    return seq, i, s["kv_lens"].long()[seq] - n[seq] + i + 1


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)

    def rand(*shape):
        return torch.rand(shape, generator=g, device=DEV)

    Hkv, d, page, B = case["Hkv"], case["d"], case["page"], case["B"]
    nq, kv = _lengths(case)
    cu = [0]
    for n in nq:
        cu.append(cu[-1] + n)
    s = dict(case=case, cu=_i32(cu), kv_lens=_i32(kv), T=cu[-1], max_q=max(nq), max_kv=max(kv))
    s["block_table"], pages = _tables(kv, page, g)
    if case["op"] == "evict":
        # the pool holds the pages that the kept keys go to, and one that nobody uses
        s["new_table"], more = _tables([min(k, case["budget"]) for k in kv], page, g, pages)
        pages += more + 1
        # sums of attention weights: many tiny, a few large, some keys never looked at
        w = torch.exp(3 * randn(B, Hkv, s["max_kv"], dtype=torch.float32))
        s["weights"] = w * (rand(B, Hkv, s["max_kv"]) < 0.9)
    if case["op"] == "select":
        # each page's keys lie around a point of their own
        mid = randn(pages, Hkv, 1, d, dtype=torch.float32)
        off = randn(pages, Hkv, 2, d, dtype=torch.float32).abs() * torch.tensor([-1.0, 1.0], device=DEV)[:, None]
        s["bounds"] = (0.6 * mid + off).bfloat16()
    else:
        s["k_cache"] = randn(pages, Hkv, page, d)
    if case["op"] in ("tree", "selected", "evict"):
        s["v_cache"] = randn(pages, Hkv, page, d)
    if case["op"] == "bounds":
        s["bounds"] = torch.zeros(pages, Hkv, 2, d, dtype=torch.bfloat16, device=DEV)
    if case["op"] in ("tree", "select", "selected", "weights"):
        s["q"] = randn(s["T"], case["H"], d)
    if case["op"] == "tree":
        words = -(-s["max_q"] // 64)
        rows = np.zeros((s["T"], words * 64), dtype=np.uint8)
        for at, parents in zip(cu, _parents(case)):
            for i, p in enumerate(parents):
                if p >= 0:
                    rows[at + i] = rows[at + p]
                rows[at + i, i] = 1
        bits = np.packbits(rows, axis=1, bitorder="little").view(np.int64)
        s["tree_mask"] = torch.from_numpy(bits).to(DEV)
    if case["op"] == "selected":  # distinct pages, ascending, the first and the last among them
        seq, _, sees = _visible(s)
        have = (sees + page - 1) // page
        at = torch.arange(s["block_table"].shape[1], device=DEV)
        key = rand(s["T"], Hkv, at.numel())
        key[:, :, 0] = -1.0
        key = torch.where(at == have[:, None, None] - 1, -1.0, key)
        key = torch.where(at >= have[:, None, None], 2.0, key)
        low, idx = key.topk(min(case["top"], at.numel()), largest=False)
        idx = torch.where(low < 1.5, idx, at.numel()).sort(-1).values
        pick = torch.full((s["T"], Hkv, case["top"]), -1, dtype=torch.int32, device=DEV)
        pick[:, :, :idx.shape[2]] = torch.where(idx < at.numel(), idx, -1).to(torch.int32)
        s["pages"] = pick
    if case["op"] == "weights":
        s["weights"] = torch.exp(randn(B, Hkv, s["max_kv"], dtype=torch.float32))
        # what the attention call before has left: the log-sum-exp of each query's scores
        lse = []
        for b in range(B):
            x = _case_scores(s, b, torch.float32)
            lse.append(torch.logsumexp(x, -1).flatten(0, 1))
        s["lse"] = torch.cat(lse, 1).contiguous()
    return s


def _case_scores(s, b, dtype):
    """Scaled and causally masked scores [Hkv, group, tokens, keys] of one sequence."""
    c = s["case"]
    lo, hi = s["cu"][b:b + 2].tolist()
    n, k = hi - lo, int(s["kv_lens"][b])
    K = s["k_cache"][s["block_table"][b, :-(-k // c["page"])].long()].to(dtype).transpose(1, 2).flatten(0, 1)[:k]
    q = s["q"][lo:hi].to(dtype).unflatten(1, (c["Hkv"], -1)).permute(1, 2, 0, 3)
    x = (q.flatten(1, 2) @ K.permute(1, 2, 0)).unflatten(1, (-1, n)) * c["d"] ** -0.5
    sees = k - n + torch.arange(n, device=DEV)
    return x.masked_fill(torch.arange(k, device=DEV) > sees[:, None], -math.inf)


# ------------------------------------------------------------------------------- the package's calls
def _own(s):
    import exact_io_aware_fwd_gb300 as fa

    c = s["case"]
    table, lens, cu = s["block_table"], s["kv_lens"], s["cu"]
    if c["op"] == "tree":
        return fa.fa_fwd_paged_tree(s["q"], s["k_cache"], s["v_cache"], table, lens, s["tree_mask"],
                                    cu_seqlens=cu, max_q=s["max_q"], max_kv=s["max_kv"])
    if c["op"] == "bounds":
        return fa.fa_page_bounds(s["k_cache"], table, lens, s["bounds"], cu_seqlens=cu, total=s["T"])
    if c["op"] == "select":
        return fa.fa_select_pages(s["q"], s["bounds"], table, lens, c["page"], c["top"], first=c["first"],
                                  last=c["last"], cu_seqlens=cu, max_kv=s["max_kv"])
    if c["op"] == "selected":
        return fa.fa_fwd_paged_selected(s["q"], s["k_cache"], s["v_cache"], table, lens, s["pages"], cu_seqlens=cu)
    if c["op"] == "weights":
        return fa.fa_kv_weights(s["q"], s["lse"], s["k_cache"], table, lens, s["weights"], cu_seqlens=cu,
                                max_q=s["max_q"], max_kv=s["max_kv"], causal=True)
    out = fa.fa_kv_evict(s["weights"], s["k_cache"], s["v_cache"], table, lens, s["new_table"], c["budget"],
                         c["recent"], max_kv=s["max_kv"])
    return [s["k_cache"], s["v_cache"], *out]


# ---------------------------------------------------------------------------------------- plain form
def _gather(cache, table, n):
    """[rows, n, Hkv, d] in 32 bits of a block table's pages."""
    x = cache[table.clamp(min=0).long()].transpose(2, 3)
    return x.flatten(1, 2)[:, :n].float()


def _pad(s, x, seq, i):
    out = x.new_zeros((s["case"]["B"], s["max_q"]) + x.shape[1:])
    out[seq, i] = x
    return out


def _scores(s, seq, i):
    """Scaled scores [B, Hkv, group, tokens, keys] of padded queries with all keys of their sequence."""
    c = s["case"]
    q = _pad(s, s["q"].float(), seq, i).unflatten(2, (c["Hkv"], -1)).permute(0, 2, 3, 1, 4)
    k = _gather(s["k_cache"], s["block_table"], s["max_kv"]).permute(0, 2, 3, 1)
    return (q.flatten(2, 3) @ k).unflatten(2, (-1, s["max_q"])) * c["d"] ** -0.5


def _soft(x):
    """(exponentials, sums, log-sum-exps) over the last dimension; zeros where nothing is seen."""
    m = x.amax(-1, keepdim=True)
    p = torch.where(torch.isinf(m), torch.zeros_like(x), torch.exp(x - m))
    total = p.sum(-1)
    return p, total, m.squeeze(-1) + total.log()


def _plain_tree(s):
    c = s["case"]
    seq, i, _ = _visible(s)
    x = _scores(s, seq, i)
    mask = _pad(s, s["tree_mask"], seq, i)                                   # [B, tokens, words]
    n = s["cu"].diff().long()[:, None, None]
    key = torch.arange(s["max_kv"], device=DEV)
    bit = key - (s["kv_lens"].long()[:, None, None] - n)                     # [B, 1, keys]: index in the draft
    word = mask.gather(2, (bit // 64).clamp(0, mask.shape[2] - 1).expand(-1, s["max_q"], -1))
    seen = (bit < 0) | ((bit < n) & ((word >> (bit % 64)) & 1).bool())
    p, total, lse = _soft(x.masked_fill(~seen[:, None, None], -math.inf))
    v = _gather(s["v_cache"], s["block_table"], s["max_kv"]).permute(0, 2, 1, 3)
    o = (p.flatten(2, 3) @ v).unflatten(2, (c["H"] // c["Hkv"], -1))
    o = torch.where(total[..., None] > 0, o / total[..., None], torch.zeros_like(o))
    return [o.flatten(1, 2)[seq, :, i].bfloat16(), lse.flatten(1, 2)[seq, :, i].t().contiguous()]


def _plain_bounds(s):
    page, lens = s["case"]["page"], s["kv_lens"].long()[:, None]
    first = (lens - s["cu"].diff().long()[:, None]) // page
    # a sequence with fewer pages to renew than another renews its last one again
    at = torch.arange((s["max_q"] + page - 2) // page + 1, device=DEV)
    at = torch.minimum(first + at, (lens - 1) // page)                       # [B, pages]
    phys = s["block_table"].long().gather(1, at)
    k = s["k_cache"][phys]                                                   # [B, pages, Hkv, page, d]
    key = at[:, :, None] * page + torch.arange(page, device=DEV)
    valid = (key < lens[:, :, None])[:, :, None, :, None]
    lo = torch.where(valid, k, math.inf).amin(3)
    hi = torch.where(valid, k, -math.inf).amax(3)
    s["bounds"][phys] = torch.stack([lo, hi], 3)
    return s["bounds"]


def _pick(score, have, first, last, top):
    """Indices of the `top` largest scores below `have`, ascending (-1: fewer); the first and last
    ones always, ties to the lowest index.  score [rows, Hkv, P], have [rows]."""
    P = score.shape[-1]
    at = torch.arange(P, device=DEV)
    have = have[:, None, None]
    score = torch.where((at < first) | (at >= have - last), math.inf, score)
    score = torch.where(at < have, score, -math.inf)
    idx = score.sort(dim=-1, descending=True, stable=True).indices[..., :top]
    idx = torch.where(idx < have, idx, P).sort(-1).values
    out = torch.full(score.shape[:2] + (top,), -1, dtype=torch.int32, device=DEV)
    out[..., :idx.shape[-1]] = torch.where(idx < P, idx, -1).to(torch.int32)
    return out


def _plain_select(s):
    c = s["case"]
    seq, i, sees = _visible(s)
    # 64 bits: a page is in or out by a comparison
    box = s["bounds"][s["block_table"].clamp(min=0).long()].double().permute(0, 2, 3, 4, 1)  # [B, Hkv, 2, d, P]
    q = _pad(s, s["q"].double(), seq, i).unflatten(2, (c["Hkv"], -1)).permute(0, 2, 3, 1, 4)
    q = q.flatten(2, 3)
    x = q.clamp(max=0) @ box[:, :, 0] + q.clamp(min=0) @ box[:, :, 1]
    x = x.unflatten(2, (-1, s["max_q"])).amax(2)[seq, :, i]                  # [T, Hkv, P]
    return _pick(x, (sees + c["page"] - 1) // c["page"], c["first"], c["last"], c["top"])


def _plain_selected(s):
    c = s["case"]
    page = c["page"]
    seq, _, sees = _visible(s)
    pages = s["pages"].long()                                                # [T, Hkv, top]
    phys = s["block_table"].long()[seq[:, None, None], pages.clamp(min=0)]
    head = torch.arange(c["Hkv"], device=DEV)[None, :, None]
    k = s["k_cache"][phys, head].flatten(2, 3).float()                       # [T, Hkv, top * page, d]
    v = s["v_cache"][phys, head].flatten(2, 3).float()
    at = (pages[..., None] * page + torch.arange(page, device=DEV)).flatten(2)
    seen = (pages >= 0).repeat_interleave(page, 2) & (at < sees[:, None, None])
    q = s["q"].float().unflatten(1, (c["Hkv"], -1))
    x = (q @ k.transpose(2, 3)) * c["d"] ** -0.5
    p, total, lse = _soft(x.masked_fill(~seen[:, :, None], -math.inf))
    o = p @ v
    o = torch.where(total[..., None] > 0, o / total[..., None], torch.zeros_like(o))
    return [o.flatten(1, 2).bfloat16(), lse.flatten(1, 2).t().contiguous()]


def _plain_weights(s):
    c = s["case"]
    seq, i, _ = _visible(s)
    x = _scores(s, seq, i)
    n = s["cu"].diff().long()[:, None]
    token = torch.arange(s["max_q"], device=DEV)
    key = torch.arange(s["max_kv"], device=DEV)
    seen = (key <= (s["kv_lens"].long()[:, None] - n + token)[..., None]) & (token < n)[..., None]
    lse = _pad(s, s["lse"].t().contiguous(), seq, i).unflatten(2, (c["Hkv"], -1)).permute(0, 2, 3, 1)
    p = torch.exp(x - lse[..., None]).masked_fill(~seen[:, None, None], 0.0)
    return s["weights"] + p.sum((2, 3))


def _plain_evict(s):
    c = s["case"]
    page, budget = c["page"], c["budget"]
    lens = s["kv_lens"].long()
    # a sequence within the budget keeps everything: all of its keys count as recent
    w = s["weights"]
    at = torch.arange(w.shape[2], device=DEV)
    w = torch.where(at >= (lens - c["recent"])[:, None, None], math.inf, w)
    kept = _pick(w, lens, 0, 0, budget)
    there = kept >= 0
    src = kept.clamp(min=0).long()
    new_weights = torch.where(there, s["weights"].gather(2, src), 0.0)
    # places of the copies; what is not there is a slot of the unused page, copied onto itself
    spare = s["k_cache"].shape[0] - 1
    b = torch.arange(c["B"], device=DEV)[:, None, None]
    head = torch.arange(c["Hkv"], device=DEV)[None, :, None].expand_as(src)
    dst = torch.arange(budget, device=DEV).expand_as(src)
    zero = torch.zeros_like(src)
    page_src = torch.where(there, s["block_table"].long()[b, src // page], spare)
    page_dst = torch.where(there, s["new_table"].long()[b, (dst // page).clamp(max=s["new_table"].shape[1] - 1)], spare)
    slot_src, slot_dst = torch.where(there, src % page, zero), torch.where(there, dst % page, zero)
    for cache in (s["k_cache"], s["v_cache"]):
        cache[page_dst, head, slot_dst] = cache[page_src, head, slot_src]
    new_lens = lens.clamp(max=budget).to(torch.int32)
    return [s["k_cache"], s["v_cache"], new_lens, kept, new_weights]


def run(state):
    if own:
        return _own(state)
    return {"tree": _plain_tree, "bounds": _plain_bounds, "select": _plain_select, "selected": _plain_selected,
            "weights": _plain_weights, "evict": _plain_evict}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------- 64-bit definition
def _keys(cache, table, n, page):
    """[Hkv, n, d] of the first n keys of one block-table row, in 64 bits."""
    used = table[: -(-n // page)].long()
    return cache[used].double().transpose(1, 2).flatten(0, 1)[:n].transpose(0, 1)


def _attend(q, K, V, hidden, d):
    """(O, LSE) of rows q over keys K [n, d]; hidden [rows, n]."""
    x = (q @ K.t()) / math.sqrt(d)
    x.masked_fill_(hidden, -math.inf)
    return torch.softmax(x, -1) @ V, x.logsumexp(-1)


def _exact_attention(case, s):
    H, Hkv, d, page = case["H"], case["Hkv"], case["d"], case["page"]
    G = H // Hkv
    cu, kv = s["cu"].tolist(), s["kv_lens"].tolist()
    O = torch.zeros(s["T"], H, d, dtype=torch.float64, device=DEV)
    LSE = torch.zeros(H, s["T"], dtype=torch.float64, device=DEV)
    parents = _parents(case) if case["op"] == "tree" else None
    for b in range(case["B"]):
        n, k = cu[b + 1] - cu[b], kv[b]
        K = _keys(s["k_cache"], s["block_table"][b], k, page)
        V = _keys(s["v_cache"], s["block_table"][b], k, page)
        hidden = np.zeros((n, k), dtype=bool)
        if parents is not None:
            hidden[:, k - n:] = True
            for i in range(n):
                j = i
                while j >= 0:  # the token, its parent, and so on up to the context
                    hidden[i, k - n + j] = False
                    j = parents[b][j]
            hidden = torch.from_numpy(hidden).to(DEV)
            for h in range(H):
                O[cu[b]:cu[b + 1], h], LSE[h, cu[b]:cu[b + 1]] = _attend(
                    s["q"][cu[b]:cu[b + 1], h].double(), K[h // G], V[h // G], hidden, d)
            continue
        for i in range(n):
            t, sees = cu[b] + i, k - n + i + 1
            for h in range(Hkv):
                pick = [p for p in s["pages"][t, h].tolist() if p >= 0]
                at = torch.tensor([j for p in pick for j in range(p * page, min((p + 1) * page, sees))], device=DEV)
                q = s["q"][t, h * G:(h + 1) * G].double()
                none = torch.zeros(G, at.numel(), dtype=torch.bool, device=DEV)
                O[t, h * G:(h + 1) * G], LSE[h * G:(h + 1) * G, t] = _attend(q, K[h, at], V[h, at], none, d)
    return [O, LSE]


def _exact_bounds(case, s):
    page = case["page"]
    out = s["bounds"].double()
    cu, kv, table = s["cu"].tolist(), s["kv_lens"].tolist(), s["block_table"].tolist()
    for b in range(case["B"]):
        new = kv[b] - (cu[b + 1] - cu[b])
        first = new // page
        for i in range(first, -(-kv[b] // page)):
            k = s["k_cache"][table[b][i], :, :min(page, kv[b] - i * page)].double()
            out[table[b][i], :, 0], out[table[b][i], :, 1] = k.min(1).values, k.max(1).values
    return out


def _top(values, count):
    """Indices of the `count` largest values of a numpy vector, ties to the lowest index, ascending."""
    return np.sort(np.lexsort((np.arange(values.size), -values))[:count])


def _exact_select(case, s):
    G, page, top = case["H"] // case["Hkv"], case["page"], case["top"]
    cu, kv = s["cu"].tolist(), s["kv_lens"].tolist()
    out = np.full((s["T"], case["Hkv"], top), -1, dtype=np.int32)
    for b in range(case["B"]):
        P = -(-kv[b] // page)
        box = s["bounds"][s["block_table"][b, :P].long()].double()
        for t in range(cu[b], cu[b + 1]):
            have = -(-(kv[b] - cu[b + 1] + t + 1) // page)
            q = s["q"][t].double().unflatten(0, (case["Hkv"], G))            # [Hkv, G, d]
            best = torch.maximum(q * box[:, :, None, 0], q * box[:, :, None, 1])  # largest of each element's products
            score = best.sum(-1).amax(-1).t().cpu().numpy()[:, :have]
            for h in range(case["Hkv"]):
                w = score[h]
                if have > top:
                    mid = _top(w[case["first"]:have - case["last"]], top - case["first"] - case["last"])
                    pick = np.concatenate([np.arange(case["first"]), case["first"] + mid,
                                           np.arange(have - case["last"], have)])
                else:
                    pick = np.arange(have)
                out[t, h, :pick.size] = pick
    return torch.from_numpy(out).to(DEV)


def _exact_weights(case, s):
    out = s["weights"].double()
    cu = s["cu"].tolist()
    for b in range(case["B"]):
        x = _case_scores(s, b, torch.float64)
        lse = s["lse"][:, cu[b]:cu[b + 1]].double().unflatten(0, (case["Hkv"], -1))
        out[b, :, :x.shape[-1]] += torch.exp(x - lse[..., None]).sum((1, 2))
    return out


def _exact_evict(case, s):
    page, budget, recent = case["page"], case["budget"], case["recent"]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    kv = s["kv_lens"].tolist()
    w = s["weights"].double().cpu().numpy()
    kept = np.full((case["B"], case["Hkv"], budget), -1, dtype=np.int32)
    left = np.zeros(kept.shape)
    for b, n in enumerate(kv):
        m = min(n, budget)
        for h in range(case["Hkv"]):
            if n > budget:
                pick = np.concatenate([_top(w[b, h, :n - recent], budget - recent), np.arange(n - recent, n)])
            else:
                pick = np.arange(n)
            kept[b, h, :m], left[b, h, :m] = pick, w[b, h, pick]
            at, to = torch.from_numpy(pick).long().to(DEV), torch.arange(m, device=DEV)
            frm, into = s["block_table"][b, at // page].long(), s["new_table"][b, to // page].long()
            kc[into, h, to % page] = kc[frm, h, at % page]
            vc[into, h, to % page] = vc[frm, h, at % page]
    lens = torch.tensor([min(n, budget) for n in kv], dtype=torch.int32, device=DEV)
    return [kc, vc, lens, torch.from_numpy(kept).to(DEV), torch.from_numpy(left).to(DEV)]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("tree", "selected"):
        return _exact_attention(case, s)
    return {"bounds": _exact_bounds, "select": _exact_select, "weights": _exact_weights,
            "evict": _exact_evict}[case["op"]](case, s)
