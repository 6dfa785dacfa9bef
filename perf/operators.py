"""Workloads of the operators around attention: the norms and rotary positions of queries and keys
(forward and backward), appending to a paged key/value cache, attention that reads the cache, and
attention of a batch that shares a prefix.

``listed()`` and ``draw(rng)`` give cases; ``prepare(case, seed)`` makes what a program holds before
the call; ``run(state)`` is one pass, in elementary torch operations, or, where ``own`` is true,
through the package; ``exact(case, seed)`` is the definition in 64 bits; ``work(case)`` counts the
bytes and operations that a pass cannot do without.
"""

import math
import random

import torch

own = False

EPS = 1e-6
DEV = "cuda"


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # training, long grouped-query shape: norms + rotation of a fused projection, to [B, H, N, d]
        dict(name="rope-fwd-1x16384-gqa", op="rope_fwd", B=1, N=16384, H=32, Hkv=8, d=128, rot=128,
             interleaved=False, norm=True, packed=False, theta=500000.0, factor=1.0),
        # its backward: gradients in the projection's layout and of both norms' weights
        dict(name="rope-bwd-1x16384-gqa", op="rope_bwd", B=1, N=16384, H=32, Hkv=8, d=128, rot=128,
             interleaved=False, norm=True, packed=False, theta=500000.0, factor=1.0),
        # a small packed batch: interleaved pairs in part of a 64-wide head, no norms, linear scaling
        dict(name="rope-fwd-packed-1000", op="rope_fwd", B=1, N=1000, H=12, Hkv=12, d=64, rot=32,
             interleaved=True, norm=False, packed=True, theta=10000.0, factor=4.0),
        # one decoding step of 64 sequences: 64 tokens into the cache
        dict(name="append-decode-64", op="append", B=64, nq=1, qlo=1, lo=1, hi=512, H=32, Hkv=8, d=128, page=64,
             rot=128, interleaved=False, norm=True, theta=500000.0, factor=1.0),
        # the prompts of a packed batch of 512..4096 tokens into pages of 16
        dict(name="append-prompt-16x4096", op="append", B=16, nq=4096, qlo=512, lo=4096, hi=4608, H=16, Hkv=16, d=128,
             page=16, rot=64, interleaved=False, norm=False, theta=10000.0, factor=1.0),
        # the smallest call: one short sequence, one token
        dict(name="paged-1x100", op="paged", B=1, nq=1, qlo=1, lo=100, hi=100, H=8, Hkv=8, d=64, page=16),
        # a usual serving batch: 64 sequences of 512..4096 tokens, grouped-query
        dict(name="paged-64x4096-gqa", op="paged", B=64, nq=1, qlo=1, lo=512, hi=4096, H=32, Hkv=8, d=128, page=64),
        # few long contexts: the work has to be split over the keys
        dict(name="paged-4x131072-gqa", op="paged", B=4, nq=1, qlo=1, lo=100000, hi=131072, H=32, Hkv=8, d=128,
             page=128),
        # four drafted tokens for each of 16 ragged sequences, all heads with their own keys
        dict(name="paged-16x2000-draft", op="paged", B=16, nq=4, qlo=2, lo=1000, hi=2000, H=12, Hkv=12, d=128, page=32),
        # a chunk of two long prompts against what the cache holds of them already
        dict(name="paged-2x16384-chunk", op="paged", B=2, nq=512, qlo=400, lo=16000, hi=16384, H=32, Hkv=8, d=128,
             page=64),
        # a few short answers to one short instruction
        dict(name="prefix-8x1000", op="prefix", B=8, groups=1, plo=1000, phi=1000, nq=1, qlo=1, lo=0, hi=64, H=12, Hkv=4,
             d=64, page=16),
        # 128 sequences behind two long shared documents
        dict(name="prefix-128x32768-gqa", op="prefix", B=128, groups=2, plo=30000, phi=32768, nq=1, qlo=1, lo=1, hi=1024,
             H=32, Hkv=8, d=128, page=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope_fwd", "rope_bwd", "append", "paged", "paged", "prefix"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 3, 4, 8] if Hkv < 8 else [1, 4])
    page = rng.choice([16, 32, 64, 128])
    if op in ("rope_fwd", "rope_bwd"):
        B = rng.choice([1, 1, 2, 5])
        return dict(op=op, B=B, N=_log(rng, 1, 16384 // B), H=H, Hkv=Hkv, d=d,
                    rot=rng.choice([32, d // 2, d]), interleaved=rng.random() < 0.5,
                    norm=rng.random() < 0.6, packed=rng.random() < 0.5,
                    theta=rng.choice([10000.0, 500000.0]), factor=rng.choice([1.0, 4.0]))
    if op == "append":
        B = _log(rng, 1, 128)
        nq = 1 if rng.random() < 0.5 else _log(rng, 2, max(2, 32768 // B))
        hi = nq + _log(rng, 1, 512)
        return dict(op=op, B=B, nq=nq, qlo=rng.randint(1, nq), lo=nq, hi=hi, H=H, Hkv=Hkv, d=d, page=page,
                    rot=rng.choice([32, d // 2, d]), interleaved=rng.random() < 0.5,
                    norm=rng.random() < 0.6, theta=rng.choice([10000.0, 500000.0]), factor=1.0)
    if op == "paged":
        B = _log(rng, 1, 128)
        hi = _log(rng, 64, 262144 // max(B, 2))
        nq = 1
        if rng.random() < 0.4:
            nq = _log(rng, 2, max(2, min(hi, 512, 1024 // B, (1 << 24) // (B * hi))))
        return dict(op=op, B=B, nq=nq, qlo=rng.randint(1, nq), lo=max(nq, hi // rng.choice([1, 2, 8])), hi=hi, H=H,
                    Hkv=Hkv, d=d, page=page)
    B = _log(rng, 2, 128)
    groups = min(B, rng.choice([1, 1, 2, 5]))
    phi = _log(rng, 64, 65536 // groups)
    hi = _log(rng, 1, 1024)
    nq = max(1, min(rng.choice([1, 1, 1, 2, 3]), (1 << 23) // (B * phi)))
    return dict(op=op, B=B, groups=groups, plo=max(1, phi // rng.choice([1, 2])), phi=phi, nq=nq, qlo=1,
                lo=rng.choice([nq, hi + nq]), hi=hi + nq, H=H, Hkv=Hkv, d=d, page=page)


def _lengths(case, seed=7):
    """The lengths of a case are part of it, not of its inputs: (new tokens, keys) of each sequence."""
    r = random.Random("%d %d %d %d %d" % (seed, case["B"], case["nq"], case["lo"], case["hi"]))
    nq = [r.randint(case["qlo"], case["nq"]) for _ in range(case["B"])]
    nq[r.randrange(case["B"])] = case["nq"]
    kv = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    kv[r.randrange(case["B"])] = case["hi"]
    return nq, kv


def _groups(case, seed=9):
    """(first sequence of each group and the end, prefix length of each group)."""
    r = random.Random("%d %d %d %d" % (seed, case["B"], case["groups"], case["phi"]))
    cuts = sorted(r.sample(range(1, case["B"]), case["groups"] - 1))
    pre = [r.randint(case["plo"], case["phi"]) for _ in range(case["groups"])]
    pre[r.randrange(case["groups"])] = case["phi"]
    return [0] + cuts + [case["B"]], pre


def work(case):
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    if case["op"] in ("rope_fwd", "rope_bwd"):
        T = case["B"] * case["N"]
        rows = T * (H + 2 * Hkv)
        table = (case["N"] if not case["packed"] else T) * case["rot"] * 4
        moved = 2 * rows * d * 2
        if case["op"] == "rope_bwd" and case["norm"]:
            moved += T * (H + Hkv) * d * 2
        return {"bytes": moved + table, "flops": rows * d * (10 if case["norm"] else 4)}
    nq, kv = _lengths(case)
    T = sum(nq)
    if case["op"] == "append":
        rows = T * (H + 2 * Hkv)
        return {"bytes": 2 * rows * d * 2 + T * case["rot"] * 4, "flops": rows * d * 6}
    io = 2 * T * H * d * 2 + T * H * 4
    own_keys = [max(0, k) for k in kv]
    pairs = sum(n * k - n * (n - 1) // 2 if k >= n else k * (k + 1) // 2 for n, k in zip(nq, own_keys))
    keys = sum(own_keys)
    if case["op"] == "prefix":
        cut, pre = _groups(case)
        keys += sum(pre)
        pairs += sum(p * sum(nq[a:b]) for p, a, b in zip(pre, cut, cut[1:]))
    return {"bytes": keys * Hkv * d * 2 * 2 + io, "flops": 4 * pairs * H * d}


# ------------------------------------------------------------------------------------------ inputs
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _frequencies(case):
    i = torch.arange(case["rot"] // 2, dtype=torch.float64)
    return (case["theta"] ** (-2.0 * i / case["rot"]) / case["factor"]).to(DEV)


def _table(inv_freq, n):
    """cos and sin of every position, as a program computes them once: [n, rot] in 32 bits."""
    angle = torch.arange(n, dtype=torch.float64, device=DEV)[:, None] * inv_freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _tables(lens, page, g):
    """Block table of sequences of these lengths over a shuffled pool (-1 where there is no page)."""
    need = [-(-n // page) for n in lens]
    total, width = sum(need), max(1, max(need))
    pages = torch.randperm(total + 3, generator=g, device=DEV)[:total].to(torch.int32)
    have = torch.tensor(need, device=DEV)
    col = torch.arange(width, device=DEV)
    inside = col[None, :] < have[:, None]
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    table[inside] = pages
    return table.contiguous(), total + 3


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)

    s = dict(case=case)
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    if case["op"] in ("rope_fwd", "rope_bwd"):
        B, N = case["B"], case["N"]
        s["inv_freq"] = _frequencies(case)
        s["table"] = _table(s["inv_freq"], N)
        lead = (B * N,) if case["packed"] else (B, N)
        s["qkv"] = randn(*lead, H + 2 * Hkv, d)
        if case["packed"]:  # documents of different lengths, one behind the other
            at = torch.arange(B * N, device=DEV)
            first = torch.rand(B * N, generator=g, device=DEV) < 3.0 / max(N, 1)
            first[::N] = True
            s["positions"] = (at - torch.where(first, at, 0).cummax(0).values).to(torch.int32)
        if case["norm"]:
            s["wq"] = 1 + 0.2 * randn(d, dtype=torch.float32)
            s["wk"] = 1 + 0.2 * randn(d, dtype=torch.float32)
        if case["op"] == "rope_bwd":
            shape = (lambda h: (B * N, h, d)) if case["packed"] else (lambda h: (B, h, N, d))
            s["dq"], s["dk"], s["dv"] = randn(*shape(H)), randn(*shape(Hkv)), randn(*shape(Hkv))
        return s
    nq, kv = _lengths(case)
    cu = [0]
    for n in nq:
        cu.append(cu[-1] + n)
    s["cu"], s["kv_lens"], s["T"] = _i32(cu), _i32(kv), cu[-1]
    s["max_q"], s["max_kv"] = max(nq), max(kv)
    table, pages = _tables(kv, case["page"], g)
    s["block_table"] = table
    if case["op"] == "prefix":
        cut, pre = _groups(case)
        ptable, more = _tables(pre, case["page"], g)
        s["prefix_table"] = torch.where(ptable >= 0, ptable + pages, ptable)
        pages += more
        s["group_cu"], s["prefix_lens"], s["max_prefix"] = _i32(cut), _i32(pre), max(pre)
        s["group_tokens"] = [cu[b] - cu[a] for a, b in zip(cut, cut[1:])]
    s["k_cache"] = randn(pages, Hkv, case["page"], d)
    s["v_cache"] = randn(pages, Hkv, case["page"], d)
    if case["op"] == "append":
        s["inv_freq"] = _frequencies(case)
        s["table"] = _table(s["inv_freq"], case["hi"])
        s["qkv"] = randn(s["T"], H + 2 * Hkv, d)
        if case["norm"]:
            s["wq"] = 1 + 0.2 * randn(d, dtype=torch.float32)
            s["wk"] = 1 + 0.2 * randn(d, dtype=torch.float32)
    else:
        s["q"] = randn(s["T"], H, d)
    return s


# ------------------------------------------------------------------------------- the package's calls
def _own(s):
    import exact_io_aware_fwd_gb300 as fa

    c = s["case"]
    H, Hkv = c["H"], c["Hkv"]
    if c["op"] in ("rope_fwd", "rope_bwd"):
        q, k, v = s["qkv"].split([H, Hkv, Hkv], dim=-2)
        opts = dict(table=s["table"], positions=s.get("positions"), interleaved=c["interleaved"],
                    q_weight=s.get("wq"), k_weight=s.get("wk"), eps=EPS)
        if c["op"] == "rope_fwd":
            return fa.fa_qk_norm_rope_fwd(q, k, v, **opts)
        dq, dk, dv, dwq, dwk = fa.fa_qk_norm_rope_bwd(s["dq"], s["dk"], s["dv"], q, k, **opts)
        return [dq, dk, dv] + ([dwq, dwk] if c["norm"] else [])
    if c["op"] == "append":
        q, k, v = s["qkv"].split([H, Hkv, Hkv], dim=-2)
        out = fa.fa_kv_append(q, k, v, s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"],
                              cu_seqlens=s["cu"], table=s["table"], interleaved=c["interleaved"],
                              q_weight=s.get("wq"), k_weight=s.get("wk"), eps=EPS)
        return [out, s["k_cache"], s["v_cache"]]
    if c["op"] == "paged":
        return fa.fa_fwd_paged(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"],
                               cu_seqlens=s["cu"], max_q=s["max_q"], max_kv=s["max_kv"], causal=True)
    return fa.fa_fwd_shared_prefix(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"],
                                   s["prefix_table"], s["prefix_lens"], s["group_cu"],
                                   cu_seqlens=s["cu"], max_q=s["max_q"], max_kv=s["max_kv"],
                                   max_prefix=s["max_prefix"], causal=True)


# ---------------------------------------------------------------------------------------- plain form
def _turn(y, cos, sin, rot, interleaved):
    """The rotation of the first `rot` elements of each head; cos, sin [..., 1, rot / 2]."""
    head, tail = y[..., :rot], y[..., rot:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        out = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = head[..., : rot // 2], head[..., rot // 2:]
        out = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([out, tail], -1)


def _norm(x, w):
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w


def _cos_sin(s, pos):
    c, sn = s["table"][pos.long()].unsqueeze(-2).chunk(2, -1)
    return c, sn


def _positions(s):
    return s["positions"] if "positions" in s else torch.arange(s["case"]["N"], device=DEV)


def _plain_rope_fwd(s):
    c = s["case"]
    q, k, v = s["qkv"].split([c["H"], c["Hkv"], c["Hkv"]], dim=-2)
    cos, sin = _cos_sin(s, _positions(s))
    q = _turn(_norm(q.float(), s.get("wq")), cos, sin, c["rot"], c["interleaved"])
    k = _turn(_norm(k.float(), s.get("wk")), cos, sin, c["rot"], c["interleaved"])
    out = [q.bfloat16(), k.bfloat16(), v]
    return [t.contiguous() if c["packed"] else t.transpose(1, 2).contiguous() for t in out]


def _norm_bwd(g, x, w):
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    h = x * r
    u = g * w
    return r * (u - h * (u * h).mean(-1, keepdim=True)), (g * h).flatten(0, -2).sum(0)


def _plain_rope_bwd(s):
    c = s["case"]
    q, k, _ = s["qkv"].split([c["H"], c["Hkv"], c["Hkv"]], dim=-2)
    cos, sin = _cos_sin(s, _positions(s))
    dq, dk, dv = (t if c["packed"] else t.transpose(1, 2) for t in (s["dq"], s["dk"], s["dv"]))
    dq = _turn(dq.float(), cos, -sin, c["rot"], c["interleaved"])
    dk = _turn(dk.float(), cos, -sin, c["rot"], c["interleaved"])
    if not c["norm"]:
        return [dq.bfloat16(), dk.bfloat16(), dv.contiguous()]
    dq, dwq = _norm_bwd(dq, q.float(), s["wq"])
    dk, dwk = _norm_bwd(dk, k.float(), s["wk"])
    return [dq.bfloat16(), dk.bfloat16(), dv.contiguous(), dwq, dwk]


def _token_places(s):
    """(sequence, index in its new tokens, how many it has) of each packed token."""
    n = s["cu"].diff().long()
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=DEV), n, output_size=s["T"])
    return seq, torch.arange(s["T"], device=DEV) - s["cu"].long()[seq], n


def _plain_append(s):
    c = s["case"]
    q, k, v = s["qkv"].split([c["H"], c["Hkv"], c["Hkv"]], dim=-2)
    seq, i, n = _token_places(s)
    pos = s["kv_lens"].long()[seq] - n[seq] + i
    cos, sin = _cos_sin(s, pos)
    q = _turn(_norm(q.float(), s.get("wq")), cos, sin, c["rot"], c["interleaved"]).bfloat16()
    k = _turn(_norm(k.float(), s.get("wk")), cos, sin, c["rot"], c["interleaved"]).bfloat16()
    page = s["block_table"][seq, pos // c["page"]].long()
    s["k_cache"][page, :, pos % c["page"]] = k
    s["v_cache"][page, :, pos % c["page"]] = v
    return [q, s["k_cache"], s["v_cache"]]


def _gather(cache, table, n):
    """[rows, n, Hkv, d] in 32 bits of a block table's pages."""
    x = cache[table.clamp(min=0).long()].transpose(2, 3)
    return x.flatten(1, 2)[:, :n].float()


def _scores(q, k, seen, c):
    """Scaled scores of padded queries [b, t, H, d] and keys [b, n, Hkv, d], masked where not seen."""
    b, t = q.shape[:2]
    q = q.reshape(b, t, c["Hkv"], -1, c["d"]).permute(0, 2, 3, 1, 4).flatten(2, 3)
    x = (q @ k.permute(0, 2, 3, 1)).unflatten(2, (-1, t)) * c["d"] ** -0.5
    return x.masked_fill(~seen[:, None, None], float("-inf"))


def _softmax_sums(x, v):
    """(max, sum of exponentials, their product with the values) over the keys."""
    m = x.amax(-1, keepdim=True)
    p = torch.where(torch.isinf(m), torch.zeros_like(x), torch.exp(x - m))
    o = (p.flatten(2, 3) @ v.permute(0, 2, 1, 3)).unflatten(2, p.shape[2:4])
    return m.squeeze(-1), p.sum(-1), o


def _padded(s, x, row, col, rows, cols):
    out = x.new_zeros((rows, cols) + x.shape[1:])
    out[row, col] = x
    return out


def _finish(m, l, o, row, col):
    """Packed O [T, H, d] and LSE [H, T] of padded sums [rows, Hkv, group, t(, d)]."""
    o = torch.where(l[..., None] > 0, o / l[..., None], torch.zeros_like(o))
    lse = (m + l.log()).flatten(1, 2)
    o = o.flatten(1, 2)[row, :, col]
    return [o.bfloat16(), lse[row, :, col].t().contiguous()]


def _own_sums(s):
    """The padded sums of each sequence over its own pages."""
    c = s["case"]
    seq, i, n = _token_places(s)
    q = _padded(s, s["q"].float(), seq, i, c["B"], s["max_q"])
    key = torch.arange(s["max_kv"], device=DEV)
    last = s["kv_lens"].long()[:, None] - n[:, None] + torch.arange(s["max_q"], device=DEV)
    seen = (key <= last[..., None]) & (key < s["kv_lens"][:, None, None])
    k = _gather(s["k_cache"], s["block_table"], s["max_kv"])
    v = _gather(s["v_cache"], s["block_table"], s["max_kv"])
    return (*_softmax_sums(_scores(q, k, seen, c), v), seq, i)


def _plain_paged(s):
    m, l, o, seq, i = _own_sums(s)
    return _finish(m, l, o, seq, i)


def _plain_prefix(s):
    c = s["case"]
    m, l, o, seq, i = _own_sums(s)
    # the prefix: all queries of a group together against its pages
    cut = s["group_cu"].long()
    grp = torch.searchsorted(cut, seq, right=True) - 1
    at = torch.arange(s["T"], device=DEV) - s["cu"].long()[cut[grp]]
    q = _padded(s, s["q"].float(), grp, at, c["groups"], max(s["group_tokens"]))
    seen = torch.arange(s["max_prefix"], device=DEV) < s["prefix_lens"][:, None]
    k = _gather(s["k_cache"], s["prefix_table"], s["max_prefix"])
    v = _gather(s["v_cache"], s["prefix_table"], s["max_prefix"])
    pm, pl, po = _softmax_sums(_scores(q, k, seen[:, None].expand(-1, q.shape[1], -1), c), v)
    # joined token by token: [T, Hkv, group(, d)]
    m, l, o = m[seq, :, :, i], l[seq, :, :, i], o[seq, :, :, i]
    pm, pl, po = pm[grp, :, :, at], pl[grp, :, :, at], po[grp, :, :, at]
    top = torch.maximum(m, pm)
    a = torch.where(torch.isinf(m), torch.zeros_like(m), torch.exp(m - top))
    b = torch.where(torch.isinf(pm), torch.zeros_like(pm), torch.exp(pm - top))
    total = a * l + b * pl
    out = (a[..., None] * o + b[..., None] * po) / total[..., None]
    return [out.flatten(1, 2).bfloat16(), (top + total.log()).flatten(1).t().contiguous()]


def run(state):
    if own:
        return _own(state)
    return {"rope_fwd": _plain_rope_fwd, "rope_bwd": _plain_rope_bwd, "append": _plain_append,
            "paged": _plain_paged, "prefix": _plain_prefix}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------- 64-bit definition
def _exact_rotation(pos, s):
    """Complex numbers e^(i angle) [tokens, 1, rot / 2] of the positions, in 64 bits."""
    angle = pos.double().reshape(-1, 1) * s["inv_freq"]
    return torch.polar(torch.ones_like(angle), angle).unsqueeze(1)


def _exact_turn(y, z, c):
    """Rotates [tokens, heads, d]: each pair is a complex number times z."""
    y = y.clone()
    r = c["rot"]
    first = slice(0, r, 2) if c["interleaved"] else slice(0, r // 2)
    second = slice(1, r, 2) if c["interleaved"] else slice(r // 2, r)
    w = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * z
    y[..., first], y[..., second] = w.real, w.imag
    return y


def _exact_qk(x, w, z, c):
    x = x.double()
    if w is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / c["d"] + EPS).sqrt() * w.double()
    return _exact_turn(x, z, c)


def _exact_rope(case, s):
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    B, N = case["B"], case["N"]
    pos = s["positions"] if case["packed"] else torch.arange(N, device=DEV).repeat(B)
    z = _exact_rotation(pos, s)
    x = s["qkv"].reshape(B * N, H + 2 * Hkv, d)
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    there = (lambda t: t) if case["packed"] else (lambda t: t.unflatten(0, (B, N)).transpose(1, 2))
    if case["op"] == "rope_fwd":
        return [there(_exact_qk(q, s.get("wq"), z, case)), there(_exact_qk(k, s.get("wk"), z, case)),
                there(v.double())]
    back = (lambda t: t) if case["packed"] else (lambda t: t.transpose(1, 2).flatten(0, 1))
    out, dws = [], []
    for dy, x_, w in ((s["dq"], q, s.get("wq")), (s["dk"], k, s.get("wk"))):
        g = _exact_turn(back(dy).double(), z.conj(), case)
        if w is not None:
            x64 = x_.double()
            rms = (x64.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt()
            dws.append((g * x64 / rms).sum((0, 1)))
            u = g * w.double()
            g = u / rms - x64 * (u * x64).sum(-1, keepdim=True) / (d * rms ** 3)
        out.append(g)
    out.append(back(s["dv"]).double())
    shape = (lambda t: t) if case["packed"] else (lambda t: t.unflatten(0, (B, N)))
    return [shape(t) for t in out] + dws


def _exact_append(case, s):
    H, Hkv = case["H"], case["Hkv"]
    cu, kv = s["cu"].tolist(), s["kv_lens"].tolist()
    pos = torch.cat([torch.arange(kv[b] - (cu[b + 1] - cu[b]), kv[b], device=DEV) for b in range(case["B"])])
    z = _exact_rotation(pos, s)
    x = s["qkv"]
    q = _exact_qk(x[:, :H], s.get("wq"), z, case)
    k = _exact_qk(x[:, H:H + Hkv], s.get("wk"), z, case)
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    for b in range(case["B"]):
        p = pos[cu[b]:cu[b + 1]]
        page, at = s["block_table"][b].long()[p // case["page"]], p % case["page"]
        kc[page, :, at] = k[cu[b]:cu[b + 1]]
        vc[page, :, at] = x[cu[b]:cu[b + 1], H + Hkv:].double()
    return [q, kc, vc]


def _keys(cache, table, n, page):
    """[Hkv, n, d] of the first n tokens of one block table row, in 64 bits."""
    used = table[: -(-n // page)].long()
    return cache[used].double().transpose(1, 2).flatten(0, 1)[:n].transpose(0, 1)


def _exact_attention(case, s):
    H, Hkv, d, page = case["H"], case["Hkv"], case["d"], case["page"]
    cu, kv = s["cu"].tolist(), s["kv_lens"].tolist()
    O = torch.zeros(s["T"], H, d, dtype=torch.float64, device=DEV)
    LSE = torch.zeros(H, s["T"], dtype=torch.float64, device=DEV)
    prefix = [None] * case["B"]
    if case["op"] == "prefix":
        cut, pre = s["group_cu"].tolist(), s["prefix_lens"].tolist()
        for g in range(case["groups"]):
            both = [_keys(s[n], s["prefix_table"][g], pre[g], page) for n in ("k_cache", "v_cache")]
            prefix[cut[g]:cut[g + 1]] = [both] * (cut[g + 1] - cut[g])
    for b in range(case["B"]):
        n = cu[b + 1] - cu[b]
        K = _keys(s["k_cache"], s["block_table"][b], kv[b], page)
        V = _keys(s["v_cache"], s["block_table"][b], kv[b], page)
        before = 0
        if prefix[b] is not None:
            before = prefix[b][0].shape[1]
            K, V = (torch.cat([p, t], 1) for p, t in zip(prefix[b], (K, V)))
        limit = before + kv[b] - n + torch.arange(n, device=DEV)
        hidden = torch.arange(K.shape[1], device=DEV)[None] > limit.clamp(min=before - 1)[:, None]
        for h in range(Hkv):
            G = H // Hkv
            q = s["q"][cu[b]:cu[b + 1], h * G:(h + 1) * G].double().transpose(0, 1)
            x = (q @ K[h].t()) / math.sqrt(d)
            x.masked_fill_(hidden, float("-inf"))
            lse = x.logsumexp(-1)
            O[cu[b]:cu[b + 1], h * G:(h + 1) * G] = (torch.softmax(x, -1) @ V[h]).transpose(0, 1)
            LSE[h * G:(h + 1) * G, cu[b]:cu[b + 1]] = lse
    return [O, LSE]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rope_fwd", "rope_bwd"):
        return _exact_rope(case, s)
    return _exact_append(case, s) if case["op"] == "append" else _exact_attention(case, s)
