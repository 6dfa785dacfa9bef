"""Binding of the operators around attention: norms and rotary positions of queries and keys, the
paged key/value cache, and the attention that reads it (the calls of include/fa.h with the same
names).  As in binding.py only argument checks and marshalling happen here.

Calls launch on the tensors' device, on its current stream or on ``stream``; outputs and
workspaces allocated here for another stream than the current one are recorded on it.
"""

from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from .binding import (PagedKV, Prefix, QKTransform, View, _check, _out, _scale, _want, _workspace,
                      load_library)

_BF16 = torch.bfloat16
_NO_VIEW = View(None, 0, 0, 0)
_NO_GUARD = contextlib.nullcontext()


class _Launch:
    """Device guard, stream handle and the stream that fresh tensors have to be recorded on."""

    def __init__(self, device, stream):
        self.guard = (_NO_GUARD if device.index == torch.cuda.current_device()
                      else torch.cuda.device(device))
        current = torch.cuda.current_stream(device)
        self.stream = current if stream is None else stream
        self.handle = ctypes.c_void_p(self.stream.cuda_stream)
        self.foreign = self.stream.cuda_stream != current.cuda_stream

    def keep(self, *tensors):
        if self.foreign:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.stream)


def _at(t):
    return None if t is None else t.data_ptr()


def _rows(t, order, device, name):
    """View of a bf16 tensor whose dimensions are (batch, token, head) in `order` ("bnh", "bhn",
    or "nh" without a batch), then the head's contiguous elements."""
    if (not isinstance(t, torch.Tensor) or t.dtype != _BF16 or t.device != device
            or t.dim() != len(order) + 1 or t.stride(-1) != 1):
        raise ValueError(f"{name} must be a bfloat16 tensor on {device} of {len(order) + 1} "
                         "dimensions with contiguous rows")
    strides = {"b": 0, "n": 0, "h": 0}
    for i, c in enumerate(order):
        if t.shape[i] > 1:
            strides[c] = t.stride(i)
            if strides[c] % 8:
                raise ValueError(f"{name}: strides must be multiples of 8 elements")
    if t.data_ptr() % 16:
        raise ValueError(f"{name} must be 16-byte aligned")
    return View(t.data_ptr(), strides["b"], strides["n"], strides["h"])


def _own_rows(t, shape, order, device, name):
    """(tensor, view) of an output: a new contiguous tensor, or the caller's, whose elements must
    be distinct (no expanded or overlapping dimensions)."""
    if t is None:
        t = torch.empty(shape, dtype=_BF16, device=device)
    else:
        if not isinstance(t, torch.Tensor) or tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must have shape {tuple(shape)}")
        reach = 1
        for st, n in sorted((t.stride(i), t.shape[i]) for i in range(t.dim()) if t.shape[i] > 1):
            if st < reach:
                raise ValueError(f"{name} must not overlap itself")
            reach = st * (n - 1) + reach
    return t, _rows(t, order, device, name)


def _ints(t, shape, device, name):
    return None if t is None else _want(t, shape, torch.int32, device, name)


def _transform(table, interleaved, q_weight, k_weight, eps, d, device):
    n_pos = rot = 0
    if table is not None:
        if table.dim() != 2:
            raise ValueError("table must be [positions, rot]")
        n_pos, rot = table.shape
        _want(table, (n_pos, rot), torch.float32, device, "table")
        if n_pos < 1 or rot < 16 or rot > d or rot % 16:
            raise ValueError("the rotated part must be a multiple of 16 elements, at most d")
    if (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight go together")
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _want(w, (d,), torch.float32, device, name)
    return QKTransform(_at(table), n_pos, rot, int(bool(interleaved)), _at(q_weight),
                       _at(k_weight), float(eps))


def _cuda(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


# ------------------------------------------------------------------------------------------ rotary
def rope_frequencies(rot, base=10000.0, scaling=None, factor=1.0, original_len=None,
                     beta_fast=32.0, beta_slow=1.0):
    """(frequencies float64 [rot / 2] on the CPU, amplitude) of the rotation's pairs.

    scaling: None; "linear" (positions divided by `factor`); "ntk" (the base raised so that the
    slowest pair is stretched by `factor` and the fastest not at all); "yarn" (pairs that turn
    more than `beta_fast` times over `original_len` positions are kept, those that turn less than
    `beta_slow` times are divided by `factor`, a linear ramp between; cos and sin scaled by
    0.1 ln(factor) + 1)."""
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
    # the ramp is linear in the pair's index between the pairs that turn beta_fast and beta_slow times
    index = lambda t: (rot / 2) * math.log(original_len / (2 * math.pi * t)) / math.log(base)  # noqa: E731
    lo, hi = index(beta_fast), index(beta_slow)
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
    launch = _Launch(device, stream)
    with launch.guard, torch.cuda.stream(launch.stream):
        freq = inv_freq.to(device).contiguous()
        table = torch.empty((n_pos, rot), dtype=torch.float32, device=device)
        st = load_library().fa_rope_table(freq.data_ptr(), rot, n_pos, float(amplitude),
                                          table.data_ptr(), launch.handle)
    _check(st, "fa_rope_table")
    return table


def _qkv_shapes(q, k, name_q="q"):
    """(B, N, H, Hkv, d, input order, output order, output shape) of [B, N, H, d] or packed
    [total, H, d] queries and keys."""
    if q.dim() not in (3, 4) or k.dim() != q.dim():
        raise ValueError(f"{name_q} must be [B, N, H, d] or packed [total, H, d]")
    if k.shape[:-2] != q.shape[:-2] or k.shape[-1] != q.shape[-1]:
        raise ValueError("q and k must agree in tokens and head dimension")
    H, d, Hkv = q.shape[-2], q.shape[-1], k.shape[-2]
    if q.dim() == 3:
        return 1, q.shape[0], H, Hkv, d, "nh", "nh", lambda h: (q.shape[0], h, d)
    B, N = q.shape[:2]
    return B, N, H, Hkv, d, "bnh", "bhn", lambda h: (B, h, N, d)


def fa_qk_norm_rope_fwd(q, k, v=None, table=None, positions=None, interleaved=False,
                        q_weight=None, k_weight=None, eps=1e-6, q_out=None, k_out=None,
                        v_out=None, stream=None):
    """Norms and rotation of q and k, from the projection's layout to the attention's (see
    include/fa.h): [B, N, heads, d] views -> [B, heads, N, d], or packed [total, heads, d] views
    -> contiguous [total, heads, d].  Inputs (and given outputs) may be strided, such as slices
    of a fused projection; v, if given, is copied to the same layout.  table: fa_rope_table's,
    or None; positions: int32 [B, N] or [total], default each token's index n in its row.
    Returns (q, k, v or None)."""
    device = _cuda(q, "q")
    B, N, H, Hkv, d, order, out_order, shape = _qkv_shapes(q, k)
    t = _transform(table, interleaved, q_weight, k_weight, eps, d, device)
    _ints(positions, q.shape[:-2], device, "positions")
    if v is not None and tuple(v.shape) != tuple(k.shape):
        raise ValueError("v must have k's shape")
    if N == 0 or B == 0:
        return tuple(torch.empty(shape(h), dtype=_BF16, device=device) if x is not None else None
                     for x, h in ((q, H), (k, Hkv), (v, Hkv)))
    views = [_rows(q, order, device, "q"), _rows(k, order, device, "k"),
             _NO_VIEW if v is None else _rows(v, order, device, "v")]
    launch = _Launch(device, stream)
    q_out, vq = _own_rows(q_out, shape(H), out_order, device, "q_out")
    k_out, vk = _own_rows(k_out, shape(Hkv), out_order, device, "k_out")
    vv = _NO_VIEW
    if v is not None:
        v_out, vv = _own_rows(v_out, shape(Hkv), out_order, device, "v_out")
    else:
        v_out = None
    launch.keep(q_out, k_out, v_out)
    with launch.guard:
        st = load_library().fa_qk_norm_rope_fwd(*views, vq, vk, vv, _at(positions), B, N, H, Hkv,
                                                d, ctypes.byref(t), launch.handle)
    _check(st, "fa_qk_norm_rope_fwd")
    return q_out, k_out, v_out


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
    device = _cuda(dq, "dq")
    norm = q_weight is not None
    if dq.dim() == 4:
        B, H, N, d = dq.shape
        lead, order, out_order = (B, N), "bhn", "bnh"
        Hkv = dk.shape[1] if dk.dim() == 4 else 0
        want = (B, Hkv, N, d)
    elif dq.dim() == 3:
        B, (N, H, d) = 1, dq.shape
        lead, order, out_order = (N,), "nh", "nh"
        Hkv = dk.shape[1] if dk.dim() == 3 else 0
        want = (N, Hkv, d)
    else:
        raise ValueError("dq must be [B, H, N, d] or packed [total, H, d]")
    for x, name in ((dk, "dk"), (dv, "dv")):
        if x is not None and tuple(x.shape) != want:
            raise ValueError(f"{name} must agree with dq")
    t = _transform(table, interleaved, q_weight, k_weight, eps, d, device)
    _ints(positions, lead, device, "positions")
    for x, h, name in ((q, H, "q"), (k, Hkv, "k")):
        if norm and (x is None or tuple(x.shape) != (*lead, h, d)):
            raise ValueError(f"{name} (the forward's input) is needed with norms")
    launch = _Launch(device, stream)
    if dq_in is None and dk_in is None and dv_in is None:
        fused = torch.empty((*lead, H + (2 if dv is not None else 1) * Hkv, d), dtype=_BF16,
                            device=device)
        dq_in, dk_in = fused[..., :H, :], fused[..., H:H + Hkv, :]
        dv_in = fused[..., H + Hkv:, :] if dv is not None else None
        launch.keep(fused)
    empty = B == 0 or N == 0
    views = [_NO_VIEW] * 8
    if not empty:
        views[0] = _rows(dq, order, device, "dq")
        views[1] = _rows(dk, order, device, "dk")
        if norm:
            views[3] = _rows(q, out_order, device, "q")
            views[4] = _rows(k, out_order, device, "k")
        dq_in, views[5] = _own_rows(dq_in, (*lead, H, d), out_order, device, "dq_in")
        dk_in, views[6] = _own_rows(dk_in, (*lead, Hkv, d), out_order, device, "dk_in")
        launch.keep(dq_in, dk_in)
        if dv is not None:
            views[2] = _rows(dv, order, device, "dv")
            dv_in, views[7] = _own_rows(dv_in, (*lead, Hkv, d), out_order, device, "dv_in")
            launch.keep(dv_in)
    dwq = dwk = ws = None
    ws_bytes = 0
    if norm:
        dwq, dwk = torch.empty((2, d), dtype=torch.float32, device=device).unbind(0)
        ws, ws_bytes = _workspace(workspace, fa_qk_norm_rope_bwd_workspace_size(d), device)
        launch.keep(dwq, dwk, ws)
    with launch.guard:
        st = load_library().fa_qk_norm_rope_bwd(*views, _at(dwq), _at(dwk), _at(positions),
                                                max(B, 1), 0 if empty else N, H, Hkv, d,
                                                ctypes.byref(t), _at(ws), ws_bytes,
                                                launch.handle)
    _check(st, "fa_qk_norm_rope_bwd")
    return dq_in, dk_in, dv_in if dv is not None else None, dwq, dwk


# ------------------------------------------------------------------------------------- paged cache
def _cache(k_cache, v_cache, block_table, kv_lens, device):
    """(fa_paged_kv, B, Hkv, page size, d) after the checks of the cache's tensors."""
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages, Hkv, page_size, d]")
    pages, Hkv, page, d = k_cache.shape
    _want(k_cache, k_cache.shape, _BF16, device, "k_cache")
    _want(v_cache, k_cache.shape, _BF16, device, "v_cache")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    B, max_pages = block_table.shape
    _ints(block_table, (B, max_pages), device, "block_table")
    _ints(kv_lens, (B,), device, "kv_lens")
    return (PagedKV(k_cache.data_ptr(), v_cache.data_ptr(), pages, page, block_table.data_ptr(),
                    max_pages, kv_lens.data_ptr()), B, Hkv, page, d)


def _tokens(cu_seqlens, B, total, device):
    if cu_seqlens is None:
        if total != B:
            raise ValueError("without cu_seqlens there is one token per sequence")
    else:
        _ints(cu_seqlens, (B + 1,), device, "cu_seqlens")


def fa_kv_append(q, k, v, k_cache, v_cache, block_table, kv_lens, cu_seqlens=None,
                 pos_offset=None, table=None, interleaved=False, q_weight=None, k_weight=None,
                 eps=1e-6, q_out=None, stream=None):
    """Norms and rotation of the new tokens' q and k [total, heads, d] (strided views allowed),
    k and v written into the paged cache [pages, Hkv, page_size, d], q (or None) into a packed
    tensor, in one launch (see include/fa.h).  kv_lens counts the new tokens; cu_seqlens: their
    offsets, default one token per sequence; pos_offset: int32 [B] added to the rotation's
    positions.  Returns the transformed q (None without q)."""
    device = _cuda(k, "k")
    cache, B, Hkv, _, d = _cache(k_cache, v_cache, block_table, kv_lens, device)
    if k.dim() != 3 or tuple(k.shape[1:]) != (Hkv, d) or tuple(v.shape) != tuple(k.shape):
        raise ValueError("k and v must be [total, Hkv, d] with the cache's heads")
    total = k.shape[0]
    H = Hkv
    if q is not None:
        if q.dim() != 3 or q.shape[0] != total or q.shape[2] != d:
            raise ValueError("q must be [total, H, d]")
        H = q.shape[1]
    _tokens(cu_seqlens, B, total, device)
    _ints(pos_offset, (B,), device, "pos_offset")
    t = _transform(table, interleaved, q_weight, k_weight, eps, d, device)
    if total == 0:
        return None if q is None else torch.empty((0, H, d), dtype=_BF16, device=device)
    launch = _Launch(device, stream)
    vq = vo = _NO_VIEW
    if q is not None:
        vq = _rows(q, "nh", device, "q")
        q_out, vo = _own_rows(q_out, (total, H, d), "nh", device, "q_out")
        launch.keep(q_out)
    else:
        q_out = None
    with launch.guard:
        st = load_library().fa_kv_append(vq, _rows(k, "nh", device, "k"),
                                         _rows(v, "nh", device, "v"), vo, ctypes.byref(cache),
                                         _at(cu_seqlens), _at(pos_offset), B, total, H, Hkv, d,
                                         ctypes.byref(t), launch.handle)
    _check(st, "fa_kv_append")
    return q_out


def fa_fwd_paged_workspace_size(B, total, H, Hkv, d) -> int:
    return int(load_library().fa_fwd_paged_workspace_size(int(B), int(total), int(H), int(Hkv),
                                                          int(d)))


def fa_fwd_shared_prefix_workspace_size(B, groups, total, H, Hkv, d) -> int:
    return int(load_library().fa_fwd_shared_prefix_workspace_size(
        int(B), int(groups), int(total), int(H), int(Hkv), int(d)))


def _paged(q, k_cache, v_cache, block_table, kv_lens, prefix_of, cu_seqlens, max_q, max_kv, causal,
           scale, out, lse, workspace, stream, where):
    device = _cuda(q, "q")
    cache, B, Hkv, page, d = _cache(k_cache, v_cache, block_table, kv_lens, device)
    if q.dim() != 3 or q.shape[2] != d or q.shape[1] % Hkv:
        raise ValueError("q must be [total, H, d] with H a multiple of the cache's heads")
    total, H, _ = q.shape
    _want(q, q.shape, _BF16, device, "q")
    _tokens(cu_seqlens, B, total, device)
    prefix = prefix_of(device)
    if max_q is None:
        max_q = 1 if cu_seqlens is None else max(total, 1)
    if max_kv is None:
        max_kv = min(cache.max_pages * page, 0x7fffffff)
    launch = _Launch(device, stream)
    out = _out(out, q.shape, _BF16, device, "out")
    lse = _out(lse, (H, total), torch.float32, device, "lse")
    lib = load_library()
    if prefix is None:
        need = lib.fa_fwd_paged_workspace_size(B, total, H, Hkv, d)
    else:
        need = lib.fa_fwd_shared_prefix_workspace_size(B, prefix.groups, total, H, Hkv, d)
    ws, ws_bytes = _workspace(workspace, need, device)
    launch.keep(out, lse, ws)
    head = (q.data_ptr(), ctypes.byref(cache))
    tail = (out.data_ptr(), lse.data_ptr(), _at(cu_seqlens), B, int(max_q), int(max_kv), total, H,
            Hkv, d, int(bool(causal)), _scale(scale), ws.data_ptr(), ws_bytes, launch.handle)
    with launch.guard:
        st = (lib.fa_fwd_paged(*head, *tail) if prefix is None
              else lib.fa_fwd_shared_prefix(*head, ctypes.byref(prefix), *tail))
    _check(st, where)
    return out, lse


def fa_fwd_paged(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens=None, max_q=None,
                 max_kv=None, causal=False, scale=None, out=None, lse=None, workspace=None,
                 stream=None):
    """O [total, H, d] and LSE [H, total] of packed queries over the paged cache (see
    include/fa.h).  cu_seqlens: offsets of each sequence's query tokens, default one per
    sequence; causal aligns them to the end of the sequence.  max_q and max_kv bound the query
    tokens and keys of a sequence (defaults: total, and the block table's reach); close bounds
    let the launch fit the work."""
    return _paged(q, k_cache, v_cache, block_table, kv_lens, lambda device: None, cu_seqlens,
                  max_q, max_kv, causal, scale, out, lse, workspace, stream, "fa_fwd_paged")


def fa_fwd_shared_prefix(q, k_cache, v_cache, block_table, kv_lens, prefix_table, prefix_lens,
                         group_cu, cu_seqlens=None, max_q=None, max_kv=None, max_prefix=None,
                         causal=False, scale=None, out=None, lse=None, workspace=None,
                         stream=None):
    """fa_fwd_paged for sequences that share prefixes held in the same cache (see include/fa.h):
    sequences [group_cu[g], group_cu[g + 1]) begin with the prefix_lens[g] keys in pages
    prefix_table[g]; block_table and kv_lens are their own keys behind it."""
    def prefix_of(device):
        if prefix_table.dim() != 2:
            raise ValueError("prefix_table must be [groups, pages]")
        groups, pages = prefix_table.shape
        _ints(prefix_table, (groups, pages), device, "prefix_table")
        _ints(prefix_lens, (groups,), device, "prefix_lens")
        _ints(group_cu, (groups + 1,), device, "group_cu")
        reach = min(pages * k_cache.shape[2], 0x7fffffff)
        return Prefix(prefix_table.data_ptr(), pages, prefix_lens.data_ptr(),
                      group_cu.data_ptr(), groups, reach if max_prefix is None else int(max_prefix))

    return _paged(q, k_cache, v_cache, block_table, kv_lens, prefix_of, cu_seqlens, max_q, max_kv,
                  causal, scale, out, lse, workspace, stream, "fa_fwd_shared_prefix")
