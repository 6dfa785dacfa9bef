"""Norms and rotary positions of queries and keys (fa_qk_norm_rope_fwd / _bwd, fa_rope_table)
against the fp64 reference.

Tolerances.  A bf16 output is off by at most half a step, 2^-8 of its value, plus what float32
did before the rounding: each of the about 16 roundings on the way (norm, weight, products, the
table's entries) is 2^-24 of a number no larger than the row's largest, so 2^-19 of that covers
them.  In the backward the mean of u x r sums d products: 2^-24 (d + 16) of the mean of their
magnitudes, below 2^-16 of max|u| max|x r|.  A weight gradient sums rows in chains of at most
(rows a thread walks + 8 + 38 + 32) float32 additions of terms with about 8 roundings: 2^-24 x 128
= 7.6e-6 of the sum of the terms' magnitudes."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import exact_io_aware_fwd_gb300 as fa
from oracle.serving import norm_rope, norm_rope_backward

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
HALF = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    fa.build()
    fa.load_library()


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, ref, slack, label):
    """Every element within half a bf16 step and `slack` (an array or a number)."""
    got = f64(got)
    assert np.isfinite(got).all(), label
    excess = np.abs(got - ref) - (HALF * np.abs(ref) + slack)
    assert excess.max() <= 0, (label, float(excess.max()))


def make(T, H, Hkv, d, seed, norm):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, H + 2 * Hkv, d, generator=g).to(torch.bfloat16).to(DEV)
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(DEV) if norm else None for _ in range(2)]
    return qkv, *w


CASES = [
    # B, N, H, Hkv, d, rot, interleaved, norm, packed
    (1, 1, 1, 1, 64, 64, False, True, True),
    (2, 37, 4, 2, 128, 128, False, True, False),
    (2, 37, 4, 2, 128, 128, True, True, False),
    (1, 130, 5, 1, 64, 32, False, True, True),
    (1, 130, 3, 3, 64, 16, True, False, True),
    (3, 65, 8, 1, 128, 96, False, False, False),
    (3, 65, 7, 2, 128, 48, True, True, False),
    (1, 9, 32, 8, 128, 0, False, True, True),   # norms alone
    (1, 1000, 32, 8, 128, 64, False, True, True),
    (2, 3, 64, 4, 64, 0, False, False, False),  # the layout alone
]
IDS = ["B%dN%dH%dkv%dd%dr%d%s%s%s" % (*c[:6], "i" if c[6] else "", "n" if c[7] else "", "p" if c[8] else "")
       for c in CASES]


def setup(case, seed):
    B, N, H, Hkv, d, rot, inter, norm, packed = case
    qkv, wq, wk = make(B * N, H, Hkv, d, seed, norm)
    inv, table = None, None
    if rot:
        inv, _ = fa.rope_frequencies(rot, base=10000.0, scaling="linear", factor=2.0)
        table = fa.fa_rope_table(5000, rot, inv_freq=inv)
    g = torch.Generator().manual_seed(seed + 1)
    pos = torch.randint(0, 5000, (B * N,), generator=g).to(torch.int32) if seed % 2 else None
    where = pos.numpy() if pos is not None else np.tile(np.arange(N), B) if not packed else np.arange(N)
    x = qkv if packed else qkv.view(B, N, H + 2 * Hkv, d)
    if pos is not None:
        pos = pos.to(DEV) if packed else pos.view(B, N).to(DEV)
    opts = dict(table=table, positions=pos, interleaved=inter, q_weight=wq, k_weight=wk, eps=1e-5)
    ref = dict(inv_freq=None if inv is None else inv.numpy(), interleaved=inter, eps=1e-5)
    return x, opts, where, ref


@pytest.mark.parametrize("seed", [20, 21], ids=["index", "positions"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case, seed):
    B, N, H, Hkv, d, rot, inter, norm, packed = case
    x, opts, where, ref = setup(case, seed)
    q, k, v = x.split([H, Hkv, Hkv], dim=-2)
    out = fa.fa_qk_norm_rope_fwd(q, k, v, **opts)
    assert fa.fa_get_error() == fa.FA_OK
    for o, t, w, name in ((out[0], q, opts["q_weight"], "q"), (out[1], k, opts["k_weight"], "k")):
        h = t.shape[-2]
        assert o.is_contiguous() and o.shape == ((N, h, d) if packed else (B, h, N, d))
        r = norm_rope(f64(t).reshape(B * N, h, d), where, None if w is None else f64(w), **ref)
        slack = 2.0 ** -19 * np.abs(r).max(-1, keepdims=True) * 2  # a pair is at most sqrt 2 larger
        got = o if packed else o.transpose(1, 2).reshape(B * N, h, d)
        if rot == 0 and not norm:
            assert np.array_equal(f64(got), r)
        close(got, r, slack, name)
        if rot:  # what lies past the rotated part is passed on
            if not norm:
                assert torch.equal(got[..., rot:], t.reshape(B * N, h, d)[..., rot:])
    assert torch.equal(out[2], v if packed else v.transpose(1, 2))


@pytest.mark.parametrize("seed", [20, 21], ids=["index", "positions"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case, seed):
    B, N, H, Hkv, d, rot, inter, norm, packed = case
    x, opts, where, ref = setup(case, seed)
    q, k, v = x.split([H, Hkv, Hkv], dim=-2)
    g = torch.Generator().manual_seed(seed + 2)
    shape = (lambda h: (N, h, d)) if packed else (lambda h: (B, h, N, d))
    dz = [torch.randn(shape(h), generator=g).to(torch.bfloat16).to(DEV) for h in (H, Hkv, Hkv)]
    dq, dk, dv, dwq, dwk = fa.fa_qk_norm_rope_bwd(*dz, q, k, **opts)
    again = fa.fa_qk_norm_rope_bwd(*dz, q, k, **opts)
    assert fa.fa_get_error() == fa.FA_OK
    assert dq.stride() == x.stride() and dk.data_ptr() == dq.data_ptr() + 2 * H * d  # one tensor
    flat = (lambda t: f64(t)) if packed else (lambda t: f64(t.transpose(1, 2)).reshape(B * N, t.shape[1], d))
    for got, dwg, z, t, w in ((dq, dwq, dz[0], q, opts["q_weight"]), (dk, dwk, dz[1], k, opts["k_weight"])):
        h = t.shape[-2]
        x64 = f64(t).reshape(B * N, h, d)
        r, dw, size = norm_rope_backward(flat(z), x64, where, None if w is None else f64(w), **ref)
        slack = 2.0 ** -18 * np.abs(flat(z)).max(-1, keepdims=True)
        if norm:
            rs = 1 / np.sqrt((x64 ** 2).mean(-1, keepdims=True) + 1e-5)
            u = np.abs(flat(z)).max(-1, keepdims=True) * 1.5 * np.abs(f64(w)).max()
            slack = 2.0 ** -16 * rs * u * (1 + (np.abs(x64) * rs).max(-1, keepdims=True) ** 2)
            assert np.all(np.abs(f64(dwg) - dw) <= 7.6e-6 * size + 1e-30)
        close(got.reshape(B * N, h, d), r, slack, "dx")
    assert torch.equal(dv, dz[2] if packed else dz[2].transpose(1, 2))
    assert (dwq is None) == (not norm)
    for a, b in zip((dq, dk, dv, dwq, dwk), again):  # bit-identical from run to run
        assert a is None or torch.equal(a, b)


def test_backward_weight_gradient_over_many_rows():
    """More rows than one pass of the persistent grid: the partials of every block are summed."""
    T, H, Hkv, d = 6000, 8, 2, 128
    qkv, wq, wk = make(T, H, Hkv, d, 3, True)
    q, k, v = qkv.split([H, Hkv, Hkv], dim=-2)
    dz = [torch.randn(T, h, d, device=DEV).to(torch.bfloat16) for h in (H, Hkv, Hkv)]
    _, _, _, dwq, dwk = fa.fa_qk_norm_rope_bwd(*dz, q, k, q_weight=wq, k_weight=wk)
    for dw, z, t, w in ((dwq, dz[0], q, wq), (dwk, dz[1], k, wk)):
        _, ref, size = norm_rope_backward(f64(z), f64(t), np.zeros(T), f64(w))
        assert np.all(np.abs(f64(dw) - ref) <= 7.6e-6 * size)


@pytest.mark.parametrize("scale", [1e-18, 1e-12, 1e15, 1e18])
@pytest.mark.parametrize("d,inter", [(64, True), (128, False)])
def test_norms_of_very_small_and_large_rows(d, inter, scale):
    """Rows whose mean square is far from 1 but a float32 (the mean of d squares at 1e18: at most
    3e37), without eps: results and gradients, of the size of 1 and of 1 / scale, keep the bounds of
    the other tests, which are relative."""
    T, H, Hkv = 50, 4, 2
    g = torch.Generator().manual_seed(d)
    x = (scale * torch.randn(T, H + Hkv, d, generator=g)).to(torch.bfloat16).to(DEV)
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g)).to(DEV) for _ in range(2))
    inv, _ = fa.rope_frequencies(d)
    opts = dict(table=fa.fa_rope_table(T, d, inv_freq=inv), interleaved=inter, q_weight=wq, k_weight=wk, eps=0.0)
    ref = dict(inv_freq=inv.numpy(), interleaved=inter, eps=0.0)
    q, k = x.split([H, Hkv], dim=-2)
    out = fa.fa_qk_norm_rope_fwd(q, k, **opts)
    dz = [torch.randn(T, h, d, generator=g).to(torch.bfloat16).to(DEV) for h in (H, Hkv)]
    dq, dk, _, dwq, dwk = fa.fa_qk_norm_rope_bwd(*dz, None, q, k, **opts)
    assert fa.fa_get_error() == fa.FA_OK
    for o, got, dwg, z, t, w in ((out[0], dq, dwq, dz[0], q, wq), (out[1], dk, dwk, dz[1], k, wk)):
        r = norm_rope(f64(t), np.arange(T), f64(w), **ref)
        close(o, r, 2.0 ** -19 * np.abs(r).max(-1, keepdims=True) * 2, "z")
        r, dw, size = norm_rope_backward(f64(z), f64(t), np.arange(T), f64(w), **ref)
        rs = 1 / np.sqrt((f64(t) ** 2).mean(-1, keepdims=True))
        u = np.abs(f64(z)).max(-1, keepdims=True) * 1.5 * np.abs(f64(w)).max()
        slack = 2.0 ** -16 * rs * u * (1 + (np.abs(f64(t)) * rs).max(-1, keepdims=True) ** 2)
        close(got, r, slack, "dx")
        assert np.all(np.abs(f64(dwg) - dw) <= 7.6e-6 * size + 1e-30)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_backward_in_place(d, inter, norm):
    T, H, Hkv = 1000, 6, 2
    dz = [torch.randn(T, h, d, device=DEV).to(torch.bfloat16) for h in (H, Hkv, Hkv)]
    x, wq, wk = make(T, H, Hkv, d, 13, norm)
    q, k, _ = x.split([H, Hkv, Hkv], dim=-2)
    opts = dict(table=fa.fa_rope_table(T, d), interleaved=inter, q_weight=wq, k_weight=wk)
    want = fa.fa_qk_norm_rope_bwd(*dz, q, k, **opts)
    got = fa.fa_qk_norm_rope_bwd(*dz, q, k, **opts, dq_in=dz[0], dk_in=dz[1], dv_in=dz[2])
    assert all(a is b for a, b in zip(got, dz))
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, want))
    assert fa.fa_get_error() == fa.FA_OK


def test_table_far_positions_and_amplitude():
    """cos and sin of positions up to 10^6 to half a float32 step of a value of at most 1.2 (the
    angle is a float64 product, off by 2^-53 x 10^6), with yarn's amplitude."""
    rot = 64
    inv, amp = fa.rope_frequencies(rot, 500000.0, "yarn", 8.0, 8192)
    table = fa.fa_rope_table(1 << 20, rot, 500000.0, "yarn", 8.0, 8192)
    for p in (0, 1, 4095, 123457, (1 << 20) - 1):
        row = f64(table[p])
        ang = p * inv.numpy()
        assert np.abs(row[:32] - amp * np.cos(ang)).max() < 2.0 ** -23 * 1.25
        assert np.abs(row[32:] - amp * np.sin(ang)).max() < 2.0 ** -23 * 1.25
    # float32 amplitude: one more rounding is inside the bound above


def test_positions_out_of_range_are_reported():
    table = fa.fa_rope_table(50, 64)
    q = torch.randn(4, 2, 64, device=DEV).to(torch.bfloat16)
    pos = torch.tensor([0, 49, 50, -7], dtype=torch.int32, device=DEV)
    out = fa.fa_qk_norm_rope_fwd(q, q, None, table=table, positions=pos)
    assert fa.fa_get_error() == fa.FA_ERR_INDEX
    assert fa.fa_get_error() == fa.FA_OK  # cleared
    near = fa.fa_qk_norm_rope_fwd(q, q, None, table=table, positions=pos.clamp(0, 49))
    assert torch.equal(out[0], near[0]) and out[2] is None


def test_infinity_stays_where_it_is():
    """Past the rotated part elements are passed on; an infinity there reaches nothing else."""
    table = fa.fa_rope_table(8, 32)
    q = torch.randn(8, 2, 64, device=DEV).to(torch.bfloat16)
    want = fa.fa_qk_norm_rope_fwd(q, q, table=table)[0]
    q[..., 40] = float("inf")
    got = fa.fa_qk_norm_rope_fwd(q, q, table=table)[0]
    assert torch.isinf(got[..., 40]).all()
    got[..., 40], want[..., 40] = 0, 0
    assert torch.equal(got, want)


def test_strides_in_place_streams_and_graph():
    T, H, Hkv, d = 70, 6, 2, 64
    qkv, wq, wk = make(T, H, Hkv, d, 11, True)
    table = fa.fa_rope_table(T, d)
    opts = dict(table=table, q_weight=wq, k_weight=wk)
    q, k, v = qkv.split([H, Hkv, Hkv], dim=-2)
    want = fa.fa_qk_norm_rope_fwd(q, k, v, **opts)
    # heads in front of tokens, and padded rows
    hm = torch.empty(H + 2 * Hkv, T, d + 8, dtype=torch.bfloat16, device=DEV)[..., :d]
    hm.copy_(qkv.transpose(0, 1))
    got = fa.fa_qk_norm_rope_fwd(*(hm.transpose(0, 1).split([H, Hkv, Hkv], dim=-2)), **opts)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # another stream than the tensors' own
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fa.fa_qk_norm_rope_fwd(q, k, v, **opts, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # captured and replayed on new values
    static = qkv.clone()
    qs, ks, vs = static.split([H, Hkv, Hkv], dim=-2)
    dz = [torch.randn_like(t) for t in want]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = fa.fa_qk_norm_rope_fwd(qs, ks, vs, **opts)
        grads = fa.fa_qk_norm_rope_bwd(*dz, qs, ks, **opts)
    static.copy_(qkv.flip(0))
    g.replay()
    ref = fa.fa_qk_norm_rope_fwd(*(qkv.flip(0).split([H, Hkv, Hkv], dim=-2)), **opts)
    assert all(torch.equal(a, b) for a, b in zip(ref, out))
    refg = fa.fa_qk_norm_rope_bwd(*dz, qs, ks, **opts)
    assert all(torch.equal(a, b) for a, b in zip(refg, grads))
    # in place
    inp = qkv.clone()
    qi, ki, vi = inp.split([H, Hkv, Hkv], dim=-2)
    fa.fa_qk_norm_rope_fwd(qi, ki, vi, **opts, q_out=qi, k_out=ki, v_out=vi)
    assert torch.equal(qi, want[0]) and torch.equal(ki, want[1]) and torch.equal(vi, want[2])
    assert fa.fa_get_error() == fa.FA_OK


def test_table_made_on_another_stream_is_kept_while_the_current_one_may_read_it():
    """A table dropped while work on the caller's stream is still ahead is not handed to the next
    call on the side stream that made it."""
    side, first = torch.cuda.Stream(), fa.fa_rope_table(4096, 64)
    torch.cuda.synchronize()
    table = fa.fa_rope_table(4096, 64, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(200_000_000)  # about a tenth of a second
    got, where = table.clone(), table.data_ptr()
    del table
    other = fa.fa_rope_table(4096, 64, base=100.0, stream=side)
    assert other.data_ptr() != where
    torch.cuda.synchronize()
    assert torch.equal(got, first) and not torch.equal(other, first)


def test_empty_and_refusals():
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    k = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, device=DEV)
    out = fa.fa_qk_norm_rope_fwd(q, k, k, q_weight=w, k_weight=w)
    assert [tuple(t.shape) for t in out] == [(0, 4, 64), (0, 2, 64), (0, 2, 64)]
    _, _, _, dwq, dwk = fa.fa_qk_norm_rope_bwd(q, k, k, q, k, q_weight=w, k_weight=w)
    assert not dwq.any() and not dwk.any()
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    table = fa.fa_rope_table(2, 64)
    with pytest.raises(fa.binding.FAError):
        fa.fa_qk_norm_rope_fwd(q, k, table=table)  # 3 tokens, 2 positions
    for bad in (dict(q_weight=w), dict(q_weight=w.bfloat16(), k_weight=w), dict(table=table.double()),
                dict(positions=torch.zeros(4, dtype=torch.int32, device=DEV)),
                dict(positions=torch.zeros(3, dtype=torch.int64, device=DEV)),
                dict(q_out=torch.empty(3, 5, 64, dtype=torch.bfloat16, device=DEV))):
        with pytest.raises(ValueError):
            fa.fa_qk_norm_rope_fwd(q, k, **bad)
    with pytest.raises(ValueError):
        fa.fa_qk_norm_rope_bwd(q, k, q_weight=w, k_weight=w)  # the forward's q and k are missing
    with pytest.raises(ValueError):
        fa.fa_qk_norm_rope_fwd(q[..., :32], k[..., :32][..., ::2])


@pytest.mark.parametrize("shape", [(0, 5), (2, 0), (0,)], ids=str)
def test_empty_calls_return_the_given_outputs(shape):
    """Calls without tokens check and return the outputs they are given, like the others."""
    d, H, Hkv = 64, 4, 2
    new = lambda h: torch.empty(*shape, h, d, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    att = lambda h: new(h) if len(shape) == 1 else new(h).transpose(1, 2).contiguous()  # noqa: E731
    x, out, grads = [[f(h) for h in (H, Hkv, Hkv)] for f in (new, att, new)]
    got = fa.fa_qk_norm_rope_fwd(*x, q_out=out[0], k_out=out[1], v_out=out[2])
    assert all(a is b for a, b in zip(got, out))
    got = fa.fa_qk_norm_rope_bwd(*out, dq_in=grads[0], dk_in=grads[1], dv_in=grads[2])
    assert all(a is b for a, b in zip(got, grads)) and got[3] is None
    assert [t.shape for t in fa.fa_qk_norm_rope_fwd(*x)] == [t.shape for t in out]
    assert [t.shape for t in fa.fa_qk_norm_rope_bwd(*out)[:3]] == [t.shape for t in x]
    with pytest.raises(ValueError):
        fa.fa_qk_norm_rope_fwd(*x, q_out=out[1])
    with pytest.raises(ValueError):
        fa.fa_qk_norm_rope_bwd(*out, dk_in=grads[0])
    assert fa.fa_get_error() == fa.FA_OK


@pytest.mark.parametrize("norm", [False, True])
def test_training_step_around_attention(norm):
    """Projection -> norms, rotation -> attention -> loss, and all gradients back to the fused
    projection, against the same graph in float64 (the gradient tolerance of the attention
    tests, 2e-2 in the Frobenius norm)."""
    B, N, H, Hkv, d = 2, 150, 4, 2, 64
    qkv, wq, wk = make(B * N, H, Hkv, d, 31, norm)
    x = qkv.view(B, N, H + 2 * Hkv, d)
    inv, _ = fa.rope_frequencies(d)
    table = fa.fa_rope_table(N, d)
    opts = dict(table=table, q_weight=wq, k_weight=wk)
    q, k, v = fa.fa_qk_norm_rope_fwd(*x.split([H, Hkv, Hkv], dim=-2), **opts)
    o, lse = fa.fa_fwd_gqa(q, k, v, causal=True)
    do = torch.randn(B, H, N, d, device=DEV).to(torch.bfloat16)
    dq, dk, dv = fa.fa_bwd_gqa(q, k, v, o, do, lse, causal=True)
    xq, xk, _ = x.split([H, Hkv, Hkv], dim=-2)
    got = fa.fa_qk_norm_rope_bwd(dq, dk, dv, xq, xk, **opts)
    assert fa.fa_get_error() == fa.FA_OK

    x64 = x.double().cpu().requires_grad_()
    ws = [None if w is None else w.double().cpu().requires_grad_() for w in (wq, wk)]
    ang = torch.arange(N, dtype=torch.float64)[:, None] * inv
    c, s = ang.cos()[:, None], ang.sin()[:, None]

    def path(t, w):
        if w is not None:
            t = t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
        a, b = t.chunk(2, -1)
        return torch.cat([a * c - b * s, a * s + b * c], -1).transpose(1, 2)

    q6, k6, v6 = x64.split([H, Hkv, Hkv], dim=-2)
    q6, k6, v6 = path(q6, ws[0]), path(k6, ws[1]), v6.transpose(1, 2)
    k6, v6 = (t.repeat_interleave(H // Hkv, 1) for t in (k6, v6))
    sc = (q6 @ k6.transpose(-1, -2)) * d ** -0.5
    sc = sc.masked_fill(torch.ones(N, N).triu(1).bool(), float("-inf"))
    (torch.softmax(sc, -1) @ v6 * do.double().cpu()).sum().backward()
    refs = [x64.grad[..., :H, :], x64.grad[..., H:H + Hkv, :], x64.grad[..., H + Hkv:, :]]
    refs += [w.grad for w in ws if w is not None]
    for g, r in zip(got, refs):
        assert torch.linalg.norm(g.double().cpu() - r) <= 2e-2 * torch.linalg.norm(r)
