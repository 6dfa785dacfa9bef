"""The operators around attention: norms and rotary positions of queries and keys, the paged
key/value cache, and the attention that reads it (the calls of include/fa.h with the same names).

As in binding.py only argument checks and marshalling happen on the way to the library; here they
are compiled (csrc/serving_binding.cpp), because the smallest of these calls are a few
microseconds of kernel.  Calls launch on the tensors' device, on its current stream or on
``stream``; what a call allocates is allocated on the stream it launches on, and outputs are
recorded on the current one as well.  Inputs are not recorded on ``stream``: as everywhere in
PyTorch, a tensor that is freed while another stream may still read it is the caller's to keep.
"""

from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import math
import os

import torch

from .binding import FAError, _check, load_library
from .build_lib import BINDING_PATH

_BF16 = torch.bfloat16
_ENTRIES = ["fa_qk_norm_rope_fwd", "fa_qk_norm_rope_bwd", "fa_qk_norm_rope_bwd_workspace_size",
            "fa_kv_append", "fa_fwd_paged", "fa_fwd_paged_workspace_size", "fa_fwd_shared_prefix",
            "fa_fwd_shared_prefix_workspace_size", "fa_tree_mask", "fa_fwd_paged_tree",
            "fa_page_bounds", "fa_select_pages", "fa_select_pages_workspace_size",
            "fa_fwd_paged_selected", "fa_fwd_paged_selected_workspace_size", "fa_kv_weights",
            "fa_kv_evict"]
_ext = None


def _binding():
    """The compiled binding, loaded once and bound to the library."""
    global _ext
    if _ext is None:
        if not os.path.exists(BINDING_PATH):
            raise RuntimeError(f"{BINDING_PATH} is not built: run "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        loader = importlib.machinery.ExtensionFileLoader("_serving_binding", BINDING_PATH)
        module = importlib.util.module_from_spec(
            importlib.util.spec_from_loader("_serving_binding", loader))
        loader.exec_module(module)
        lib = load_library()
        module.bind(FAError, *(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value
                               for n in _ENTRIES))
        _ext = module
    return _ext


def _on(stream, call, q, *args):
    """The binding's call with `stream` as the current one.  A block that the allocator hands out
    is free in the order of the stream it belongs to, so outputs and workspaces have to belong to
    the stream that writes them."""
    if not isinstance(q, torch.Tensor) or q.device != stream.device:
        raise ValueError("stream must be one of the tensors' device")
    caller = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        out = call(q, *args)
    for t in out if isinstance(out, tuple) else (out,):
        if t is not None and caller != stream:
            t.record_stream(caller)
    return out


# ------------------------------------------------------------------------------------------ rotary
def rope_frequencies(rot, base=10000.0, scaling=None, factor=1.0, original_len=None,
                     beta_fast=32.0, beta_slow=1.0, whole_pairs=True):
    """(frequencies float64 [rot / 2] on the CPU, amplitude) of the rotation's pairs.

    scaling: None; "linear" (positions divided by `factor`); "ntk" (the base raised so that the
    slowest pair is stretched by `factor` and the fastest not at all); "yarn" (pairs that turn
    more than `beta_fast` times over `original_len` positions are kept, those that turn less than
    `beta_slow` times are divided by `factor`, a ramp between; cos and sin scaled by
    0.1 ln(factor) + 1).

    yarn's ramp is linear in the pair's index (in the number of turns, as in the method's paper,
    it would be another).  It runs from the pair that turns `beta_fast` times, rounded down, to the
    one that turns `beta_slow` times, rounded up, which is how most checkpoints were trained;
    whole_pairs=False leaves the ends between pairs.  The two differ: 36% in one frequency of
    rot 128, base 10^4, factor 16 over 4096 positions."""
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even")
    if not factor >= 1.0 or not base > 1.0:
        raise ValueError("factor must be at least 1 and base more than 1")
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    inv = base ** (-2.0 * i / rot)
    if scaling in (None, "ntk"):
        return inv, 1.0
    if scaling == "linear":
        return inv / factor, 1.0
    if scaling != "yarn":
        raise ValueError("scaling must be None, 'linear', 'ntk' or 'yarn'")
    if original_len is None or original_len < 1 or not beta_fast > beta_slow > 0:
        raise ValueError("yarn needs original_len and beta_fast > beta_slow > 0")
    # the ramp is linear in the pair's index, between the pairs that turn beta_fast and beta_slow
    # times over original_len positions
    index = lambda t: (rot / 2) * math.log(original_len / (2 * math.pi * t)) / math.log(base)  # noqa: E731
    lo, hi = index(beta_fast), index(beta_slow)
    if whole_pairs:
        lo, hi = math.floor(lo), math.ceil(hi)
    lo = max(lo, 0)  # the ramp begins at a pair and has a length, also where no pair turns that often
    hi = max(min(hi, rot - 1), lo + 1e-3)
    keep = 1.0 - ((i - lo) / (hi - lo)).clamp(0.0, 1.0)
    return inv * keep + inv / factor * (1.0 - keep), 0.1 * math.log(factor) + 1.0


def fa_rope_table(n_pos, rot, base=10000.0, scaling=None, factor=1.0, original_len=None,
                  inv_freq=None, amplitude=1.0, device="cuda", stream=None):
    """float32 [n_pos, rot] table of cos and sin, from rope_frequencies(rot, base, scaling, ...)
    or from `inv_freq` (float64 [rot / 2]) and `amplitude`; angles in float64."""
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError("device must be a CUDA device")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    n_pos, rot = int(n_pos), int(rot)
    if n_pos < 1 or rot < 2 or rot % 2:
        raise ValueError("n_pos must be positive and rot even")
    if inv_freq is None:
        inv_freq, amplitude = rope_frequencies(rot, base, scaling, factor, original_len)
    if inv_freq.dtype != torch.float64 or tuple(inv_freq.shape) != (rot // 2,):
        raise ValueError("inv_freq must be float64 [rot / 2]")
    if stream is not None and stream.device != device:
        raise ValueError("stream must be one of the table's device")
    caller = torch.cuda.current_stream(device)
    with torch.cuda.device(device), torch.cuda.stream(stream):
        freq = inv_freq.to(device).contiguous()
        table = torch.empty((n_pos, rot), dtype=torch.float32, device=device)
        st = load_library().fa_rope_table(freq.data_ptr(), rot, n_pos, float(amplitude),
                                          table.data_ptr(),
                                          torch.cuda.current_stream(device).cuda_stream)
    _check(st, "fa_rope_table")
    if stream is not None and stream != caller:
        table.record_stream(caller)
    return table


def fa_qk_norm_rope_fwd(q, k, v=None, table=None, positions=None, interleaved=False,
                        q_weight=None, k_weight=None, eps=1e-6, q_out=None, k_out=None,
                        v_out=None, stream=None):
    """Norms and rotation of q and k, from the projection's layout to the attention's (see
    include/fa.h): [B, N, heads, d] views -> [B, heads, N, d], or packed [total, heads, d] views
    -> contiguous [total, heads, d].  Inputs (and given outputs) may be strided, such as slices
    of a fused projection; v, if given, is copied to the same layout.  table: fa_rope_table's,
    or None; positions: int32 [B, N] or [total], default each token's index n in its row.
    Returns (q, k, v or None)."""
    ext = _ext or _binding()
    if stream is None:
        return ext.norm_rope_fwd(q, k, v, table, positions, interleaved, q_weight, k_weight, eps,
                                 q_out, k_out, v_out)
    return _on(stream, ext.norm_rope_fwd, q, k, v, table, positions, interleaved, q_weight,
               k_weight, eps, q_out, k_out, v_out)


def fa_qk_norm_rope_bwd_workspace_size(d) -> int:
    return int(load_library().fa_qk_norm_rope_bwd_workspace_size(int(d)))


def fa_qk_norm_rope_bwd(dq, dk, dv=None, q=None, k=None, table=None, positions=None,
                        interleaved=False, q_weight=None, k_weight=None, eps=1e-6, dq_in=None,
                        dk_in=None, dv_in=None, workspace=None, stream=None):
    """Gradients of fa_qk_norm_rope_fwd (see include/fa.h): dq, dk (and dv) of its outputs
    ([B, heads, N, d] or packed [total, heads, d]) to the projection's layout ([B, N, heads, d]
    or packed), with the forward's q and k when there are norms (else not needed).  Without given
    outputs the three gradients are slices of one new tensor [..., H + 2 Hkv, d], the gradient of
    a fused projection.  Returns (dq, dk, dv or None, dq_weight, dk_weight); the last two are
    float32 [d], None without norms."""
    ext = _ext or _binding()
    if stream is None:
        return ext.norm_rope_bwd(dq, dk, dv, q, k, table, positions, interleaved, q_weight,
                                 k_weight, eps, dq_in, dk_in, dv_in, workspace)
    return _on(stream, ext.norm_rope_bwd, dq, dk, dv, q, k, table, positions, interleaved,
               q_weight, k_weight, eps, dq_in, dk_in, dv_in, workspace)


# ------------------------------------------------------------------------------------- paged cache
def fa_kv_append(q, k, v, k_cache, v_cache, block_table, kv_lens, cu_seqlens=None,
                 pos_offset=None, table=None, interleaved=False, q_weight=None, k_weight=None,
                 eps=1e-6, q_out=None, stream=None):
    """Norms and rotation of the new tokens' q and k [total, heads, d] (strided views allowed),
    k and v written into the paged cache [pages, Hkv, page_size, d], q (or None) into a packed
    tensor, in one launch (see include/fa.h).  kv_lens counts the new tokens; cu_seqlens: their
    offsets, default one token per sequence; pos_offset: int32 [B] added to the rotation's
    positions.  Returns the transformed q (None without q)."""
    ext = _ext or _binding()
    if stream is None:
        return ext.kv_append(q, k, v, k_cache, v_cache, block_table, kv_lens, cu_seqlens,
                             pos_offset, table, interleaved, q_weight, k_weight, eps, q_out)
    return _on(stream, lambda kk, *rest: ext.kv_append(q, kk, *rest), k, v, k_cache, v_cache,
               block_table, kv_lens, cu_seqlens, pos_offset, table, interleaved, q_weight,
               k_weight, eps, q_out)


def fa_fwd_paged_workspace_size(B, total, H, Hkv, d) -> int:
    return int(load_library().fa_fwd_paged_workspace_size(int(B), int(total), int(H), int(Hkv),
                                                          int(d)))


def fa_fwd_shared_prefix_workspace_size(B, groups, total, H, Hkv, d) -> int:
    return int(load_library().fa_fwd_shared_prefix_workspace_size(
        int(B), int(groups), int(total), int(H), int(Hkv), int(d)))


def fa_fwd_paged(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens=None, max_q=None,
                 max_kv=None, causal=False, scale=None, out=None, lse=None, workspace=None,
                 stream=None):
    """O [total, H, d] and LSE [H, total] of packed queries over the paged cache (see
    include/fa.h).  cu_seqlens: offsets of each sequence's query tokens, default one per
    sequence; causal aligns them to the end of the sequence.  max_q and max_kv bound the query
    tokens and keys of a sequence (defaults: total, or 1 without cu_seqlens, and the block table's
    reach).  They choose the kernel and how keys are split, so a loose bound costs time: single
    tokens passed with cu_seqlens and no max_q are taken for chunks."""
    ext = _ext or _binding()
    if stream is None:
        return ext.fwd_paged(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens, max_q, max_kv,
                             causal, scale, out, lse, workspace)
    return _on(stream, ext.fwd_paged, q, k_cache, v_cache, block_table, kv_lens, cu_seqlens, max_q,
               max_kv, causal, scale, out, lse, workspace)


def fa_fwd_shared_prefix(q, k_cache, v_cache, block_table, kv_lens, prefix_table, prefix_lens,
                         group_cu, cu_seqlens=None, max_q=None, max_kv=None, max_prefix=None,
                         causal=False, scale=None, out=None, lse=None, workspace=None,
                         stream=None):
    """fa_fwd_paged for sequences that share prefixes held in the same cache (see include/fa.h):
    sequences [group_cu[g], group_cu[g + 1]) begin with the prefix_lens[g] keys in pages
    prefix_table[g]; block_table and kv_lens are their own keys behind it."""
    ext = _ext or _binding()
    if stream is None:
        return ext.fwd_shared_prefix(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens, max_q,
                                     max_kv, causal, scale, out, lse, workspace, prefix_table,
                                     prefix_lens, group_cu, max_prefix)
    return _on(stream, ext.fwd_shared_prefix, q, k_cache, v_cache, block_table, kv_lens,
               cu_seqlens, max_q, max_kv, causal, scale, out, lse, workspace, prefix_table,
               prefix_lens, group_cu, max_prefix)


# ------------------------------------------------------------------------------------------- trees
def fa_tree_mask(parents, cu_seqlens=None, max_q=None, out=None, stream=None):
    """int64 [total, words] masks of trees of new tokens: bit k of a token's row says whether it sees
    the k-th new token of its sequence (itself and its ancestors).  parents: int32 [total], each
    token's parent as an index among its sequence's new tokens, smaller than its own, or -1 behind
    the context.  cu_seqlens: the sequences' offsets, default one token each; max_q (default: total,
    or 1 without cu_seqlens) bounds a sequence's tokens and gives the words, 64 tokens each."""
    ext = _ext or _binding()
    if stream is None:
        return ext.tree_mask(parents, cu_seqlens, max_q, out)
    return _on(stream, ext.tree_mask, parents, cu_seqlens, max_q, out)


def fa_fwd_paged_tree(q, k_cache, v_cache, block_table, kv_lens, tree_mask, cu_seqlens=None,
                      max_q=None, max_kv=None, scale=None, out=None, lse=None, workspace=None,
                      stream=None):
    """fa_fwd_paged of trees of drafted tokens (see include/fa.h): a query sees the keys in front of
    its sequence's new tokens, and those new tokens whose bit is set in its row of tree_mask (int64
    [total, words], fa_tree_mask's or any other).  The drafted tokens' keys and values are in the
    cache; their rotary position is that of their depth, so they go there in two steps:
    fa_qk_norm_rope_fwd with positions, then fa_kv_append without a table."""
    ext = _ext or _binding()
    if stream is None:
        return ext.fwd_paged_tree(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens, max_q,
                                  max_kv, False, scale, out, lse, workspace, tree_mask)
    return _on(stream, ext.fwd_paged_tree, q, k_cache, v_cache, block_table, kv_lens, cu_seqlens,
               max_q, max_kv, False, scale, out, lse, workspace, tree_mask)


# ---------------------------------------------------------------------------------- selected pages
def fa_page_bounds(k_cache, block_table, kv_lens, bounds, cu_seqlens=None, total=None, stream=None):
    """Renews the bounds (bf16 [pages, Hkv, 2, d]: the smallest and the largest of each element of a
    page's keys) of the pages that hold one of the last n keys of each sequence (see include/fa.h).
    cu_seqlens: offsets whose differences are n, default 1 each; total: at least their last one, which
    bounds the launch (default: what the block table has room for, a warp for each of its pages; pages
    that a smaller one leaves out are reported).  Returns bounds."""
    ext = _ext or _binding()
    if stream is None:
        return ext.page_bounds(k_cache, block_table, kv_lens, bounds, cu_seqlens, total)
    return _on(stream, ext.page_bounds, k_cache, block_table, kv_lens, bounds, cu_seqlens, total)


def fa_select_pages_workspace_size(B, total, Hkv, page_size, max_kv) -> int:
    return int(load_library().fa_select_pages_workspace_size(int(B), int(total), int(Hkv),
                                                             int(page_size), int(max_kv)))


def fa_select_pages(q, bounds, block_table, kv_lens, page_size, top, first=1, last=1,
                    cu_seqlens=None, max_kv=None, out=None, workspace=None, stream=None):
    """int32 [total, Hkv, top]: the pages that each query token attends to (see include/fa.h): the
    `first` first and `last` last of those it sees and, of the others, those whose keys may score
    highest by their bounds; ascending indices into the sequence's row of block_table, -1 where
    there are fewer.  max_kv bounds a sequence's keys (default: the block table's reach): the
    workspace grows with it."""
    ext = _ext or _binding()
    if stream is None:
        return ext.select_pages(q, bounds, block_table, kv_lens, page_size, top, first, last,
                                cu_seqlens, max_kv, out, workspace)
    return _on(stream, ext.select_pages, q, bounds, block_table, kv_lens, page_size, top, first,
               last, cu_seqlens, max_kv, out, workspace)


def fa_fwd_paged_selected_workspace_size(total, H, Hkv, d) -> int:
    return int(load_library().fa_fwd_paged_selected_workspace_size(int(total), int(H), int(Hkv),
                                                                   int(d)))


def fa_fwd_paged_selected(q, k_cache, v_cache, block_table, kv_lens, pages, cu_seqlens=None,
                          scale=None, out=None, lse=None, workspace=None, stream=None):
    """O [total, H, d] and LSE [H, total] of packed queries over the keys of selected pages (see
    include/fa.h): each token and key/value head reads the pages in its row of pages (int32 [total,
    Hkv, top], fa_select_pages' or any other), causally."""
    ext = _ext or _binding()
    if stream is None:
        return ext.fwd_paged_selected(q, k_cache, v_cache, block_table, kv_lens, pages, cu_seqlens,
                                      scale, out, lse, workspace)
    return _on(stream, ext.fwd_paged_selected, q, k_cache, v_cache, block_table, kv_lens, pages,
               cu_seqlens, scale, out, lse, workspace)


# ---------------------------------------------------------------------------------------- eviction
def fa_kv_weights(q, lse, k_cache, block_table, kv_lens, weights=None, cu_seqlens=None, max_q=None,
                  max_kv=None, causal=False, scale=None, out=None, stream=None):
    """float32 [B, Hkv, capacity]: weights (None: zeros) plus the attention weights that the queries q
    [total, H, d] gave to each key, summed over a key/value head's queries (see include/fa.h); lse:
    the attention's [H, total].  The capacity is that of weights or out, else max_kv; out may be
    weights.  cu_seqlens, max_q, max_kv, causal, scale: as in the attention call."""
    ext = _ext or _binding()
    if stream is None:
        return ext.kv_weights(q, lse, k_cache, block_table, kv_lens, weights, cu_seqlens, max_q,
                              max_kv, causal, scale, out)
    return _on(stream, ext.kv_weights, q, lse, k_cache, block_table, kv_lens, weights, cu_seqlens,
               max_q, max_kv, causal, scale, out)


def fa_kv_evict(weights, k_cache, v_cache, block_table, kv_lens, new_table, budget, recent,
                max_kv=None, stream=None):
    """Each sequence and key/value head keeps `budget` keys, the last `recent` and those of the rest
    with the largest weights (float32 [B, Hkv, capacity]), in their order (see include/fa.h).  They
    and their values are copied to the pages new_table (int32 [B, pages], unused pages of the
    cache).  Returns (new_lens int32 [B], kept int32 [B, Hkv, budget]: which keys, -1 behind the
    last, new_weights float32 [B, Hkv, budget]).  The next token's rotary position stays kv_lens[b]:
    kv_lens - new_lens is what fa_kv_append's pos_offset grows by.  The new pages have no bounds yet
    (fa_page_bounds with cu_seqlens that count new_lens tokens), and new_weights has no columns for
    further keys."""
    ext = _ext or _binding()
    if stream is None:
        return ext.kv_evict(weights, k_cache, v_cache, block_table, kv_lens, new_table, budget,
                            recent, max_kv)
    return _on(stream, ext.kv_evict, weights, k_cache, v_cache, block_table, kv_lens, new_table,
               budget, recent, max_kv)
