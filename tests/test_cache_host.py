"""CPU checks of the operators that choose and drop keys of the paged cache, and of trees: argument
refusals of the C ABI and of the binding, the index functions compiled for the host, and the fp64
reference against closed forms."""

import math
import os
import subprocess

import numpy as np
import pytest
import torch

import exact_io_aware_fwd_gb300 as fa
from exact_io_aware_fwd_gb300 import build_lib
from oracle.serving import (attend, attend_where, evict, key_weights, largest, page_bounds, page_scores,
                            select_pages, tree_sees)
from test_serving_host import CACHE_FAULTS, P, _kv

HERE = os.path.dirname(os.path.abspath(__file__))
BAD = fa.FA_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    fa.build()
    return fa.load_library()


def test_index_functions_on_the_host(tmp_path):
    exe = tmp_path / "checks"
    subprocess.run([build_lib._nvcc(), *build_lib.ARCH, "-O1", "-std=c++17", "-I", build_lib.CSRC,
                    os.path.join(HERE, "csrc", "cache_host_checks.cu"), "-o", str(exe)],
                   check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout


# ------------------------------------------------------------------------------- C ABI refusals
NO_V = [kw for kw in CACHE_FAULTS if "v_cache" not in kw]
NO_KV = [kw for kw in NO_V if "k_cache" not in kw]


def test_tree_refusals(lib):
    def mask(parents=P, cu=P, B=2, total=5, words=1, out=P):
        return lib.fa_tree_mask(parents, cu, B, total, words, out, None)

    assert mask(parents=None) == BAD and mask(out=None) == BAD and mask(out=P + 4) == BAD
    assert mask(words=0) == BAD and mask(words=(1 << 24) + 1) == BAD
    assert mask(B=0) == BAD and mask(total=-1) == BAD and mask(cu=None) == BAD
    assert mask(total=0, parents=None, out=None) == fa.FA_OK

    def tree(cache=None, q=P, mask=P, words=1, o=P, lse=P, cu=P, B=2, max_q=3, max_kv=64, total=5, H=4, Hkv=2,
             d=64, scale=-1.0, ws=P, nbytes=1 << 30):
        return lib.fa_fwd_paged_tree(q, cache or _kv(), mask, words, o, lse, cu, B, max_q, max_kv, total, H, Hkv, d,
                                     scale, ws, nbytes, None)

    for kw in CACHE_FAULTS:
        assert tree(_kv(**kw)) == BAD, kw
    assert tree(mask=None) == BAD and tree(mask=P + 4) == BAD and tree(words=0) == BAD and tree(words=-1) == BAD
    assert tree(q=None) == BAD and tree(o=P + 4) == BAD and tree(lse=None) == BAD and tree(scale=math.nan) == BAD
    assert tree(H=3) == BAD and tree(B=0) == BAD and tree(cu=None) == BAD and tree(max_q=0) == BAD
    assert tree(d=32) == fa.FA_ERR_UNSUPPORTED and tree(_kv(page_size=48)) == fa.FA_ERR_UNSUPPORTED
    assert tree(H=258) == fa.FA_ERR_UNSUPPORTED
    need = lib.fa_fwd_paged_workspace_size(2, 5, 4, 2, 64)
    assert tree(nbytes=need - 1) == fa.FA_ERR_WORKSPACE and tree(ws=None) == fa.FA_ERR_WORKSPACE
    assert tree(total=0, q=None, mask=None, o=None, lse=None, ws=None) == fa.FA_OK


def test_page_refusals(lib):
    def bounds(cache=None, out=P, cu=P, B=2, total=5, Hkv=2, d=64):
        return lib.fa_page_bounds(cache or _kv(v_cache=None), out, cu, B, total, Hkv, d, None)

    for kw in NO_V:
        assert bounds(_kv(**kw)) == BAD, kw
    assert bounds(out=None) == BAD and bounds(out=P + 8) == BAD and bounds(B=0) == BAD and bounds(cu=None) == BAD
    assert bounds(total=-1) == BAD and bounds(Hkv=0) == BAD and bounds(d=96) == fa.FA_ERR_UNSUPPORTED
    assert bounds(_kv(page_size=8)) == fa.FA_ERR_UNSUPPORTED
    assert bounds(B=1 << 28, Hkv=8) == fa.FA_ERR_UNSUPPORTED  # pages x heads past 31 bits
    assert bounds(total=0) == fa.FA_OK

    def select(cache=None, q=P, b=P, out=P, top=4, first=1, last=1, cu=P, B=2, max_kv=640, total=5, H=4, Hkv=2, d=64,
               ws=P, nbytes=1 << 30):
        return lib.fa_select_pages(q, b, cache or _kv(k_cache=None, v_cache=None), out, top, first, last, cu, B,
                                   max_kv, total, H, Hkv, d, ws, nbytes, None)

    for kw in NO_KV:
        assert select(_kv(**kw)) == BAD, kw
    for kw in (dict(q=None), dict(b=None), dict(out=None), dict(q=P + 8), dict(b=P + 2), dict(top=0), dict(first=-1),
               dict(last=-1), dict(first=3, last=2), dict(first=1 << 30, last=1 << 30), dict(B=0), dict(cu=None),
               dict(total=-1), dict(H=3), dict(max_kv=-1)):
        assert select(**kw) == BAD, kw
    assert select(d=32) == fa.FA_ERR_UNSUPPORTED and select(H=258) == fa.FA_ERR_UNSUPPORTED
    assert select(B=1 << 20, total=1 << 20, max_kv=1 << 20) == fa.FA_ERR_UNSUPPORTED
    need = lib.fa_select_pages_workspace_size(2, 5, 2, 16, 640)
    assert need > 5 * 2 * 40 * 12 and select(nbytes=need - 1) == fa.FA_ERR_WORKSPACE
    assert select(ws=None) == fa.FA_ERR_WORKSPACE
    for args in ((0, 5, 2, 16, 640), (2, -1, 2, 16, 640), (2, 5, 0, 16, 640), (2, 5, 2, 17, 640), (2, 5, 2, 16, -1)):
        assert lib.fa_select_pages_workspace_size(*args) == 0
    assert select(total=0, q=None, b=None, out=None, ws=None) == fa.FA_OK

    def selected(cache=None, q=P, pages=P, top=4, o=P, lse=P, cu=P, B=2, total=5, H=4, Hkv=2, d=64, scale=-1.0, ws=P,
                 nbytes=1 << 30):
        return lib.fa_fwd_paged_selected(q, cache or _kv(), pages, top, o, lse, cu, B, total, H, Hkv, d, scale, ws,
                                         nbytes, None)

    for kw in CACHE_FAULTS:
        assert selected(_kv(**kw)) == BAD, kw
    for kw in (dict(q=None), dict(pages=None), dict(top=0), dict(o=None), dict(lse=None), dict(o=P + 2), dict(B=0),
               dict(cu=None), dict(total=-1), dict(H=3), dict(scale=math.inf)):
        assert selected(**kw) == BAD, kw
    assert selected(d=32) == fa.FA_ERR_UNSUPPORTED and selected(H=258) == fa.FA_ERR_UNSUPPORTED
    assert selected(top=1 << 28) == fa.FA_ERR_UNSUPPORTED  # keys past 31 bits
    need = lib.fa_fwd_paged_selected_workspace_size(5, 4, 2, 64)
    assert need > 0 and selected(nbytes=need - 1) == fa.FA_ERR_WORKSPACE
    assert lib.fa_fwd_paged_selected_workspace_size(-1, 4, 2, 64) == 0
    assert selected(total=0, q=None, pages=None, o=None, lse=None, ws=None) == fa.FA_OK


def test_eviction_refusals(lib):
    def weights(cache=None, q=P, lse=P, w=P, out=P, cap=64, cu=P, B=2, max_q=3, max_kv=64, total=5, H=4, Hkv=2, d=64,
                scale=-1.0):
        return lib.fa_kv_weights(q, lse, cache or _kv(v_cache=None), w, out, cap, cu, B, max_q, max_kv, total, H, Hkv,
                                 d, 1, scale, None)

    for kw in NO_V:
        assert weights(_kv(**kw)) == BAD, kw
    for kw in (dict(q=None), dict(lse=None), dict(out=None), dict(q=P + 4), dict(cap=-1), dict(B=0), dict(cu=None),
               dict(max_q=0), dict(max_kv=-1), dict(total=-1), dict(H=3), dict(scale=math.nan)):
        assert weights(**kw) == BAD, kw
    assert weights(d=32) == fa.FA_ERR_UNSUPPORTED and weights(H=258) == fa.FA_ERR_UNSUPPORTED
    assert weights(_kv(num_pages=1 << 30), Hkv=4) == fa.FA_ERR_UNSUPPORTED
    assert weights(total=1 << 29, H=4, Hkv=1) == fa.FA_ERR_UNSUPPORTED  # queries past the plan's
    assert weights(B=1 << 24, cap=1 << 20, max_kv=1 << 20) == fa.FA_ERR_UNSUPPORTED
    assert weights(cap=0, out=None) == fa.FA_OK

    def drop(cache=None, w=P, cap=64, table=P, pages=2, budget=20, recent=4, lens=P, kept=P, left=P, B=2, max_kv=64,
             Hkv=2, d=64):
        return lib.fa_kv_evict(w, cap, cache or _kv(), table, pages, budget, recent, lens, kept, left, B, max_kv, Hkv,
                               d, None)

    for kw in CACHE_FAULTS:
        assert drop(_kv(**kw)) == BAD, kw
    for kw in (dict(w=None), dict(table=None), dict(lens=None), dict(kept=None), dict(left=None), dict(cap=-1),
               dict(pages=-1), dict(budget=0), dict(recent=-1), dict(recent=21), dict(B=0), dict(max_kv=-1)):
        assert drop(**kw) == BAD, kw
    assert drop(d=32) == fa.FA_ERR_UNSUPPORTED and drop(_kv(page_size=1)) == fa.FA_ERR_UNSUPPORTED
    assert drop(B=1 << 20, budget=1 << 20) == fa.FA_ERR_UNSUPPORTED


def test_binding_refuses_host_tensors(lib):
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(4, 1, dtype=torch.int32), torch.ones(4, dtype=torch.int32)
    w, box = torch.zeros(4, 2, 16), torch.zeros(2, 2, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: fa.fa_tree_mask(lens), lambda: fa.fa_page_bounds(cache, table, lens, box),
                 lambda: fa.fa_fwd_paged_tree(q, cache, cache, table, lens, torch.zeros(4, 1, dtype=torch.int64)),
                 lambda: fa.fa_select_pages(q, box, table, lens, 16, 2),
                 lambda: fa.fa_fwd_paged_selected(q, cache, cache, table, lens, torch.zeros(4, 2, 1, dtype=torch.int32)),
                 lambda: fa.fa_kv_weights(q, torch.zeros(2, 4), cache, table, lens),
                 lambda: fa.fa_kv_evict(w, cache, cache, table, lens, table, 4, 1),
                 lambda: fa.fa_tree_mask([1, 2]), lambda: fa.fa_page_bounds(None, table, lens, box)):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------------------- the reference
def test_reference_masks_are_limits():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(3, 4, 8)), rng.normal(size=(2, 10, 8)), rng.normal(size=(2, 10, 8))
    seen = np.arange(10) < np.array([0, 4, 10])[:, None, None]
    for a, b in zip(attend(q, k, v, 0.3, [0, 4, 10]), attend_where(q, k, v, 0.3, seen)):
        np.testing.assert_allclose(a, b, atol=1e-12)
    assert tree_sees([-1, 0, 1, 0, -1]).tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 1, 1, 0, 0],
                                                     [1, 0, 0, 1, 0], [0, 0, 0, 0, 1]]


def test_reference_bounds_bound_every_key():
    """A page's score is at least q.k of every key of it, and is reached by a page of one key."""
    rng = np.random.default_rng(1)
    q, k = rng.normal(size=(6, 8)), rng.normal(size=(2, 37, 8))
    lo, hi = page_bounds(k, 16)
    s = page_scores(q, lo, hi)
    for h in range(2):
        dots = (k[h] @ q[3 * h:3 * h + 3].T).max(1)
        for p in range(3):
            assert dots[16 * p:16 * p + 16].max() <= s[h, p] + 1e-12
    one = page_scores(q, *page_bounds(k, 1))
    np.testing.assert_allclose(one, [(k[h] @ q[3 * h:3 * h + 3].T).max(1) for h in range(2)])
    assert largest([1.0, 3.0, 3.0, 2.0, 3.0], 2).tolist() == [1, 2]
    assert select_pages(np.array([9.0, 1, 5, 5, 7, 0]), 6, 4, 1, 1).tolist() == [0, 2, 4, 5]
    assert select_pages(np.array([9.0, 1]), 2, 4, 1, 1).tolist() == [0, 1]


def test_reference_weights_are_the_softmax():
    rng = np.random.default_rng(2)
    q, k, v = rng.normal(size=(3, 4, 8)), rng.normal(size=(2, 10, 8)), rng.normal(size=(2, 10, 8))
    limits = [0, 4, 10]
    lse = attend(q, k, v, 0.3, limits)[1]
    w, _ = key_weights(q, k, 0.3, lse, limits)
    np.testing.assert_allclose(w.sum(1), [4.0, 4.0])  # two of three tokens see keys, two heads a group
    assert np.all(w[:, 4:] < w[:, :4].max()) and np.all(w > 0)
    assert evict(np.array([5.0, 1, 4, 4, 0, 9, 9]), 7, 4, 2).tolist() == [0, 2, 5, 6]
    assert evict(np.array([5.0, 1]), 2, 4, 2).tolist() == [0, 1]
    assert evict(np.array([5.0, np.nan, 7, 1, 1]), 5, 2, 0).tolist() == [1, 2]
