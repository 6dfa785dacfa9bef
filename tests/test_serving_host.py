"""CPU checks of the operators around attention: the index functions of the paged kernels compiled
for the host, argument refusals of the C ABI and of the binding, the rotary frequencies, and the
fp64 reference (its gradients against differences)."""

import math
import os
import struct
import subprocess
import sysconfig

import numpy as np
import pytest
import torch

import exact_io_aware_fwd_gb300 as fa
from exact_io_aware_fwd_gb300 import build_lib, serving
from oracle import attention_forward
from oracle.serving import attend, norm_rope, norm_rope_backward, paged_keys, rotate

HERE = os.path.dirname(os.path.abspath(__file__))
P = 0x10000  # aligned fake pointer, never dereferenced on the refusal paths


@pytest.fixture(scope="module")
def lib():
    fa.build()
    return fa.load_library()


def test_plan_functions_on_the_host(tmp_path):
    exe = tmp_path / "checks"
    subprocess.run([build_lib._nvcc(), *build_lib.ARCH, "-O1", "-std=c++17", "-I", build_lib.CSRC,
                    os.path.join(HERE, "csrc", "paged_plan_checks.cu"), "-o", str(exe)],
                   check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout


def test_index_functions_on_the_host(tmp_path):
    exe = tmp_path / "checks"
    subprocess.run([build_lib._nvcc(), *build_lib.ARCH, "-O1", "-std=c++17", "-I", build_lib.CSRC,
                    os.path.join(HERE, "csrc", "paged_host_checks.cu"), "-o", str(exe)],
                   check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout


# ------------------------------------------------------------------------------- C ABI refusals
# the structures of include/fa.h, in native alignment
VIEW, TRANSFORM = struct.Struct("@Pqqq"), struct.Struct("@PiiiPPf4x")
PAGED_KV, PREFIX = struct.Struct("@PPiiPiP"), struct.Struct("@PiPPii")


def _view(p=P, batch=8, token=8, head=8):
    return VIEW.pack(p or 0, batch, token, head)


def _pack(layout, values):
    return layout.pack(*(0 if v is None else v for v in values))


def _transform(**kw):
    d = dict(table=P, n_pos=64, rot=64, interleaved=0, q_weight=None, k_weight=None, eps=1e-6)
    d.update(kw)
    return _pack(TRANSFORM, d.values())


def test_rope_table_refusals(lib):
    ok = [P, 64, 100, 1.0, P, None]
    for at, bad in ((0, None), (4, None), (1, 0), (1, 63), (1, 2000), (2, 0), (2, -3),
                    (3, math.inf), (0, P + 4), (4, P + 2)):
        args = list(ok)
        args[at] = bad
        assert lib.fa_rope_table(*args) == fa.FA_ERR_INVALID_ARG, (at, bad)


def test_norm_rope_refusals(lib):
    def fwd(views=None, B=1, N=8, H=4, Hkv=2, d=64, t=None, pos=None):
        v = views or [_view() for _ in range(6)]
        return lib.fa_qk_norm_rope_fwd(b"".join(v[:3]), b"".join(v[3:]), pos, B, N, H, Hkv, d,
                                       t or _transform(), None)

    bad = fa.FA_ERR_INVALID_ARG
    assert fwd(d=96) == fa.FA_ERR_UNSUPPORTED
    assert fwd(H=0) == bad and fwd(Hkv=-1) == bad and fwd(B=0) == bad and fwd(N=-1) == bad
    assert fwd(N=65) == bad  # more tokens than the table has positions
    assert fwd(N=0) == fa.FA_OK
    assert fwd(B=1 << 20, N=1 << 20, pos=P) == bad
    for kw in (dict(rot=24), dict(rot=0), dict(rot=128), dict(n_pos=0), dict(table=P + 4),
               dict(q_weight=P), dict(k_weight=P), dict(q_weight=P, k_weight=P + 8),
               dict(q_weight=P, k_weight=P, eps=-1.0), dict(q_weight=P, k_weight=P, eps=math.nan)):
        assert fwd(t=_transform(**kw)) == bad, kw
    for i in (0, 1, 3, 4, 5):  # null, misaligned and odd strides of each view
        for v in (_view(None), _view(P + 8), _view(token=12), _view(head=4)):
            views = [_view() for _ in range(6)]
            views[i] = v
            assert fwd(views) == bad, i
    views = [_view() for _ in range(6)]
    views[0] = _view(batch=4)
    assert fwd(views, B=2, pos=P) == bad

    def bwd(views=None, dw=(P, P), ws=P, nbytes=1 << 24, t=None, N=8):
        v = views or [_view() for _ in range(8)]
        return lib.fa_qk_norm_rope_bwd(b"".join(v[:3]), b"".join(v[3:5]), b"".join(v[5:]), *dw, None,
                                       1, N, 4, 2, 64, t or _transform(q_weight=P, k_weight=P), ws,
                                       nbytes, None)

    assert lib.fa_qk_norm_rope_bwd_workspace_size(96) == 0
    need = lib.fa_qk_norm_rope_bwd_workspace_size(64)
    assert need >= 2 * 64 * 4
    assert bwd(dw=(None, P)) == bad and bwd(dw=(P, None)) == bad
    assert bwd(ws=None) == fa.FA_ERR_WORKSPACE and bwd(nbytes=need - 1) == fa.FA_ERR_WORKSPACE
    assert bwd(ws=P + 16) == bad
    for i in range(8):
        views = [_view() for _ in range(8)]
        views[i] = _view(P + 2)
        assert bwd(views) == bad, i
    assert bwd(t=_transform(), ws=None, dw=(None, None), N=0) == fa.FA_OK


def _kv(**kw):
    d = dict(k_cache=P, v_cache=P, num_pages=8, page_size=16, block_table=P, max_pages=4, kv_lens=P)
    d.update(kw)
    return _pack(PAGED_KV, d.values())


CACHE_FAULTS = [dict(k_cache=None), dict(v_cache=None), dict(k_cache=P + 8), dict(num_pages=0),
                dict(max_pages=-1), dict(block_table=None), dict(kv_lens=None)]


def test_append_refusals(lib):
    def call(cache=None, views=None, B=2, total=5, cu=P, t=None):
        v = views or [_view() for _ in range(4)]
        return lib.fa_kv_append(b"".join(v[:3]), v[3], cache or _kv(), cu, None, B, total, 4, 2, 64,
                                t or _transform(), None)

    bad = fa.FA_ERR_INVALID_ARG
    for kw in CACHE_FAULTS + [dict(max_pages=0)]:
        assert call(_kv(**kw)) == bad, kw
    assert call(_kv(page_size=48)) == fa.FA_ERR_UNSUPPORTED
    assert call(B=0) == bad and call(total=-1) == bad
    assert call(cu=None) == bad  # one token per sequence needs total == B
    assert call(total=0) == fa.FA_OK
    assert call(t=_transform(rot=8)) == bad
    for i in (1, 2, 3):
        views = [_view() for _ in range(4)]
        views[i] = _view(None)
        assert call(views=views) == bad, i


def test_paged_attention_refusals(lib):
    def call(cache=None, q=P, o=P, lse=P, cu=P, B=2, max_q=3, max_kv=64, total=5, H=4, Hkv=2, d=64,
             scale=-1.0, ws=P, nbytes=1 << 30):
        return lib.fa_fwd_paged(q, cache or _kv(), o, lse, cu, B, max_q, max_kv,
                                total, H, Hkv, d, 1, scale, ws, nbytes, None)

    bad = fa.FA_ERR_INVALID_ARG
    for kw in CACHE_FAULTS:
        assert call(_kv(**kw)) == bad, kw
    assert call(_kv(page_size=256)) == fa.FA_ERR_UNSUPPORTED
    assert call(d=32) == fa.FA_ERR_UNSUPPORTED
    assert call(H=3) == bad and call(H=0) == bad and call(Hkv=0) == bad and call(B=0) == bad
    assert call(H=258, Hkv=2) == fa.FA_ERR_UNSUPPORTED  # 129 query heads per key/value head
    assert call(max_q=0) == bad and call(max_kv=-1) == bad and call(total=-1) == bad
    assert call(cu=None) == bad and call(scale=math.nan) == bad
    assert call(q=None) == bad and call(o=P + 4) == bad and call(lse=None) == bad
    assert call(ws=None) == fa.FA_ERR_WORKSPACE and call(ws=P + 8) == bad
    need = lib.fa_fwd_paged_workspace_size(2, 5, 4, 2, 64)
    assert need > 0 and call(nbytes=need - 1) == fa.FA_ERR_WORKSPACE
    assert call(total=0, q=None, o=None, lse=None, ws=None) == fa.FA_OK
    assert call(total=1 << 29, H=32, Hkv=8) == bad  # (token, head) rows past 32 bits
    assert call(total=1 << 24, B=64, H=64, Hkv=8, max_kv=1 << 20, nbytes=1 << 50) == fa.FA_ERR_UNSUPPORTED
    assert call(_kv(num_pages=1 << 30)) == bad  # pages x heads past 32 bits
    assert lib.fa_fwd_paged_workspace_size(0, 5, 4, 2, 64) == 0
    assert lib.fa_fwd_paged_workspace_size(2, 5, 4, 3, 64) == 0

    def shared(prefix, nbytes=1 << 30):
        return lib.fa_fwd_shared_prefix(P, _kv(), prefix, P, P, P, 2, 3, 64, 5, 4, 2,
                                        64, 1, -1.0, P, nbytes, None)

    def pre(**kw):
        d = dict(table=P, max_pages=4, lens=P, group_cu=P, groups=2, max_len=64)
        d.update(kw)
        return _pack(PREFIX, d.values())

    assert shared(None) == bad
    for kw in (dict(table=None), dict(max_pages=-1), dict(lens=None), dict(group_cu=None),
               dict(groups=0), dict(max_len=-1)):
        assert shared(pre(**kw)) == bad, kw
    need = lib.fa_fwd_shared_prefix_workspace_size(2, 2, 5, 4, 2, 64)
    assert need > lib.fa_fwd_paged_workspace_size(2, 5, 4, 2, 64)
    assert shared(pre(), need - 1) == fa.FA_ERR_WORKSPACE
    assert lib.fa_fwd_shared_prefix_workspace_size(2, 0, 5, 4, 2, 64) == 0


def test_binding_refuses_host_tensors_and_other_objects(lib):
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.fa_qk_norm_rope_fwd(q, q)
    cache = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(4, 1, dtype=torch.int32), torch.ones(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.fa_kv_append(q, q, q, cache, cache, table, lens)
    with pytest.raises(ValueError):
        fa.fa_fwd_paged(q, cache, cache, table, lens)
    with pytest.raises(ValueError):
        fa.fa_fwd_paged([1.0], cache, cache, table, lens)
    with pytest.raises(ValueError):
        fa.fa_qk_norm_rope_bwd(q, None)
    with pytest.raises(TypeError):
        fa.fa_fwd_paged(q, cache, cache, table)


def test_binding_belongs_to_one_pytorch_and_python(lib, monkeypatch):
    """A binding built with another PyTorch or Python is another file: it is neither taken for this
    one nor loaded in its place."""
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert build_lib.BINDING_PATH == build_lib.binding_path(torch.__version__, suffix)
    assert os.path.exists(build_lib.BINDING_PATH)
    others = [build_lib.binding_path("1.0", suffix), build_lib.binding_path(torch.__version__, ".cpython-30.so")]
    assert len({build_lib.BINDING_PATH, *others}) == 3
    monkeypatch.setattr(serving, "BINDING_PATH", others[0])
    monkeypatch.setattr(serving, "_ext", None)
    with pytest.raises(RuntimeError, match="not built"):
        serving._binding()


def test_rope_table_refuses_a_stream_of_another_device():
    class Elsewhere:
        device = torch.device("cuda", 1)

    with pytest.raises(ValueError):
        fa.fa_rope_table(8, 64, device="cuda:0", stream=Elsewhere())


# ----------------------------------------------------------------------------- rotary frequencies
def test_rope_frequencies():
    inv, amp = fa.rope_frequencies(8, base=10000.0)
    assert amp == 1.0
    np.testing.assert_allclose(inv.numpy(), [1.0, 0.1, 0.01, 0.001], rtol=1e-15)
    lin, _ = fa.rope_frequencies(8, scaling="linear", factor=4.0)
    np.testing.assert_allclose(lin.numpy(), inv.numpy() / 4, rtol=1e-15)
    ntk, _ = fa.rope_frequencies(8, scaling="ntk", factor=4.0)  # fastest kept, slowest stretched
    np.testing.assert_allclose(ntk.numpy()[[0, -1]], [1.0, 0.001 / 4], rtol=1e-13)
    assert np.all(np.diff(ntk.numpy()) < 0)
    yarn, amp = fa.rope_frequencies(64, scaling="yarn", factor=8.0, original_len=4096)
    inv, _ = fa.rope_frequencies(64)
    ratio = (yarn / inv).numpy()
    turns = (4096 * inv / (2 * math.pi)).numpy()
    assert np.allclose(ratio[turns >= 32], 1.0) and np.allclose(ratio[turns <= 1], 1 / 8)
    mid = (turns < 32) & (turns > 1)
    assert mid.any() and np.all(np.diff(ratio[mid]) < 0) and np.all(ratio[mid] < 1)
    assert amp == pytest.approx(0.1 * math.log(8.0) + 1)
    for bad in (dict(rot=7), dict(rot=8, scaling="cubic"), dict(rot=8, scaling="yarn"),
                dict(rot=8, factor=0.5), dict(rot=8, base=1.0)):
        with pytest.raises(ValueError):
            fa.rope_frequencies(**bad)


def test_yarn_ramp_between_whole_pairs():
    """The ends of the ramp by hand: (rot / 2) ln(len / (2 pi turns)) / ln(base) is 23.6 and 39.65 for
    rot 128, base 10^6 over 32768 positions at 32 turns and 1, and 20.9 and 45.03 for base 10^4 over
    4096; rounded outwards 23, 40 and 20, 46."""
    i = np.arange(64)
    for base, factor, length, lo, hi in ((1e6, 4.0, 32768, 23, 40), (1e4, 16.0, 4096, 20, 46)):
        inv = base ** (-i / 64)
        keep = 1 - np.clip((i - lo) / (hi - lo), 0, 1)
        got, _ = fa.rope_frequencies(128, base, "yarn", factor, length)
        np.testing.assert_allclose(got.numpy(), inv * (keep + (1 - keep) / factor), rtol=1e-13)
        # ends between pairs, on request
        lo, hi = (64 * math.log(length / (2 * math.pi * t)) / math.log(base) for t in (32, 1))
        keep = 1 - np.clip((i - lo) / (hi - lo), 0, 1)
        cut, _ = fa.rope_frequencies(128, base, "yarn", factor, length, whole_pairs=False)
        np.testing.assert_allclose(cut.numpy(), inv * (keep + (1 - keep) / factor), rtol=1e-13)
        assert np.abs((cut / got).numpy() - 1).max() > 0.04
    # every pair turns less than 32 times over 128 positions: the ramp begins at pair 0; short and
    # long lengths leave it a length
    got, _ = fa.rope_frequencies(128, 1e4, "yarn", 2.0, 128)
    assert got[0] == 1.0 and 0.5 < got[1] * 1e4 ** (1 / 64) < 1.0
    for length in (1, 5, 1 << 40):
        got, _ = fa.rope_frequencies(64, 1e4, "yarn", 8.0, length)
        ratio = got.numpy() * 1e4 ** (np.arange(32) / 32)
        assert np.all((ratio > 1 / 8 - 1e-12) & (ratio < 1 + 1e-12)) and np.all(np.diff(ratio) < 1e-12)
    assert np.allclose(ratio, 1.0)


# ------------------------------------------------------------------------------- the reference
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_reference_gradients_are_differences(interleaved, norm):
    rng = np.random.default_rng(5)
    T, H, d, rot = 3, 2, 16, 8
    x, dz = rng.normal(size=(T, H, d)), rng.normal(size=(T, H, d))
    w = 1 + 0.3 * rng.normal(size=d) if norm else None
    pos, inv = np.array([0, 5, 70]), 100.0 ** (-np.arange(rot // 2) / (rot // 2))
    kw = dict(inv_freq=inv, interleaved=interleaved, amplitude=1.1)
    dx, dw, _ = norm_rope_backward(dz, x, pos, w, 1e-3, **kw)
    f = lambda x_, w_: (norm_rope(x_, pos, w_, 1e-3, **kw) * dz).sum()  # noqa: E731
    h = 1e-6
    for _ in range(20):
        e = np.zeros_like(x)
        i = tuple(rng.integers(0, n) for n in x.shape)
        e[i] = h
        assert (f(x + e, w) - f(x - e, w)) / (2 * h) == pytest.approx(dx[i], rel=1e-6, abs=1e-8)
    for i in range(d if norm else 0):
        e = np.zeros(d)
        e[i] = h
        assert (f(x, w + e) - f(x, w - e)) / (2 * h) == pytest.approx(dw[i], rel=1e-6, abs=1e-8)


def test_reference_rotation_depends_on_distance_only():
    rng = np.random.default_rng(6)
    q, k = rng.normal(size=(1, 1, 32)), rng.normal(size=(1, 1, 32))
    inv = 50.0 ** (-np.arange(16) / 16)
    dots = [float((rotate(q, [a], inv, il) * rotate(k, [b], inv, il)).sum())
            for a, b in ((3, 1), (103, 101), (5002, 5000)) for il in (False,)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-9)


def test_reference_attention_is_the_oracle():
    rng = np.random.default_rng(7)
    n, d, page = 37, 16, 8
    q, k, v = (rng.normal(size=(n, d)) for _ in range(3))
    table = rng.permutation(9)
    kc, vc = (rng.normal(size=(9, 1, page, d)) for _ in range(2))
    for j in range(n):
        kc[table[j // page], 0, j % page], vc[table[j // page], 0, j % page] = k[j], v[j]
    K, V = paged_keys(kc, table, n), paged_keys(vc, table, n)
    assert np.array_equal(K[0], k) and np.array_equal(V[0], v)
    O, LSE, _, _ = attend(q[:, None], K, V, d ** -0.5, [i + 1 for i in range(n)])
    ref = attention_forward(q, k, v, d ** -0.5, True)
    ref = ref if isinstance(ref, dict) else {"O": ref[0], "LSE": ref[1]}
    np.testing.assert_allclose(O[:, 0], ref["O"], atol=1e-12)
    np.testing.assert_allclose(LSE[:, 0], ref["LSE"], atol=1e-12)
