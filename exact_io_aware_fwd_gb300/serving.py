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
            "fa_fwd_shared_prefix_workspace_size"]
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
