"""Binding of the operators around attention: norms and rotary positions of queries and keys, the
paged key/value cache, and the attention that reads it (the calls of include/fa.h with the same
names).  As in binding.py only argument checks and marshalling happen here; a call is a few
microseconds of kernel in the smallest cases, so the checks are written to be short.

Calls launch on the tensors' device, on its current stream or on ``stream``; outputs and
workspaces allocated here for another stream than the current one are recorded on it.
"""

from __future__ import annotations

import math
import struct

import torch

from .binding import _check, _out, _scale, _workspace, load_library

_BF16 = torch.bfloat16
_F32 = torch.float32
_I32 = torch.int32
_current_stream = torch._C._cuda_getCurrentRawStream  # stream handle of a device index

# the structures of include/fa.h, in native alignment
_VIEW = struct.Struct("@Pqqq")          # fa_view: data, batch, token, head
_VIEWS2 = struct.Struct("@PqqqPqqq")
_VIEWS3 = struct.Struct("@PqqqPqqqPqqq")
_TRANSFORM = struct.Struct("@PiiiPPf4x")  # fa_qk_transform
_PAGED_KV = struct.Struct("@PPiiPiP")     # fa_paged_kv
_PREFIX = struct.Struct("@PiPPii")        # fa_prefix
_NO_VIEW = (0, 0, 0, 0)
_NO_TRANSFORM = _TRANSFORM.pack(0, 0, 0, 0, 0, 0, 0.0)


def _handle(device, stream):
    return _current_stream(device.index) if stream is None else stream.cuda_stream


def _keep(stream, device, *tensors):
    """Records fresh tensors on a given stream that is not the one they were allocated for."""
    if stream is not None and stream.cuda_stream != _current_stream(device.index):
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _launch(device, call, *args):
    """call(*args) with the tensors' device current."""
    if device.index == torch.cuda.current_device():
        return call(*args)
    with torch.cuda.device(device):
        return call(*args)


def _array(t, dtype, shape, device, name):
    """Address of a contiguous `dtype` tensor of `shape` on `device`; 0 for None."""
    if t is None:
        return 0
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape
            or t.device != device or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} "
                         f"on {device}")
    return t.data_ptr()


_DIMS = {"nh": (None, 0, 1), "bnh": (0, 1, 2), "bhn": (0, 2, 1)}  # batch, token, head


def _rows(t, order, device, name):
    """fa_view fields of a bf16 tensor whose dimensions are (batch, token, head) in `order`
    ("bnh", "bhn", or "nh" without a batch), then the head's contiguous elements."""
    ib, i_n, ih = _DIMS[order]
    if (not isinstance(t, torch.Tensor) or t.dtype is not _BF16 or t.device != device
            or t.dim() != len(order) + 1):
        raise ValueError(f"{name} must be a bfloat16 tensor on {device} of {len(order) + 1} "
                         "dimensions")
    st, ptr = t.stride(), t.data_ptr()
    b, n, h = 0 if ib is None else st[ib], st[i_n], st[ih]
    if (b | n | h) & 7:  # the stride of a dimension of one element does not matter
        sh = t.shape
        b = 0 if ib is None or sh[ib] == 1 else b
        n, h = (0 if sh[i_n] == 1 else n), (0 if sh[ih] == 1 else h)
    if (b | n | h) & 7 or ptr & 15 or st[-1] != 1:
        raise ValueError(f"{name} must have contiguous rows, 16-byte aligned, at strides that "
                         "are multiples of 8 elements")
    return ptr, b, n, h


def _own_rows(t, shape, order, device, name):
    """(tensor, fa_view fields) of an output: a new contiguous tensor, or the caller's, whose
    elements must be distinct (no expanded or overlapping dimensions)."""
    if t is None:
        t = torch.empty(shape, dtype=_BF16, device=device)
    else:
        if not isinstance(t, torch.Tensor) or t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}")
        reach = 1
        for st, n in sorted((t.stride(i), t.shape[i]) for i in range(t.dim()) if t.shape[i] > 1):
            if st < reach:
                raise ValueError(f"{name} must not overlap itself")
            reach = st * (n - 1) + reach
    return t, _rows(t, order, device, name)


def _transform(table, interleaved, q_weight, k_weight, eps, d, device):
    if table is None and q_weight is None and k_weight is None:
        return _NO_TRANSFORM
    n_pos = rot = at = 0
    if table is not None:
        if not isinstance(table, torch.Tensor) or table.dim() != 2:
            raise ValueError("table must be a tensor [positions, rot]")
        n_pos, rot = table.shape
        at = _array(table, _F32, table.shape, device, "table")
        if n_pos < 1 or rot < 16 or rot > d or rot % 16:
            raise ValueError("the rotated part must be a multiple of 16 elements, at most d")
    if (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight go together")
    return _TRANSFORM.pack(at, n_pos, rot, 1 if interleaved else 0,
                           _array(q_weight, _F32, (d,), device, "q_weight"),
                           _array(k_weight, _F32, (d,), device, "k_weight"), eps)


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
    # the ramp is linear in the pair's index, between the pairs that turn beta_fast and beta_slow
    # times over original_len positions
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
    with torch.cuda.device(device), torch.cuda.stream(stream):
        freq = inv_freq.to(device).contiguous()
        table = torch.empty((n_pos, rot), dtype=_F32, device=device)
        st = load_library().fa_rope_table(freq.data_ptr(), rot, n_pos, float(amplitude),
                                          table.data_ptr(), _handle(device, stream))
    _check(st, "fa_rope_table")
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
    device = _cuda(q, "q")
    shape, shape_k = q.shape, k.shape
    if len(shape) not in (3, 4) or shape_k[:-2] != shape[:-2] or shape_k[-1] != shape[-1]:
        raise ValueError("q and k must be [B, N, heads, d] or packed [total, heads, d], alike in "
                         "tokens and head dimension")
    if v is not None and v.shape != shape_k:
        raise ValueError("v must have k's shape")
    H, d, Hkv = shape[-2], shape[-1], shape_k[-2]
    if len(shape) == 3:
        B, N, order, out_order = 1, shape[0], "nh", "nh"
    else:
        B, N, order, out_order = shape[0], shape[1], "bnh", "bhn"
        shape, shape_k = (B, H, N, d), (B, Hkv, N, d)
    t = _transform(table, interleaved, q_weight, k_weight, eps, d, device)
    pos = _array(positions, _I32, q.shape[:-2], device, "positions")
    if B == 0 or N == 0:
        return tuple(None if x is None else torch.empty(s, dtype=_BF16, device=device)
                     for x, s in ((q, shape), (k, shape_k), (v, shape_k)))
    views = _VIEWS3.pack(*_rows(q, order, device, "q"), *_rows(k, order, device, "k"),
                         *(_NO_VIEW if v is None else _rows(v, order, device, "v")))
    q_out, vq = _own_rows(q_out, shape, out_order, device, "q_out")
    k_out, vk = _own_rows(k_out, shape_k, out_order, device, "k_out")
    if v is None:
        v_out, vv = None, _NO_VIEW
    else:
        v_out, vv = _own_rows(v_out, shape_k, out_order, device, "v_out")
    _keep(stream, device, q_out, k_out, v_out)
    _check(_launch(device, load_library().fa_qk_norm_rope_fwd, views, _VIEWS3.pack(*vq, *vk, *vv),
                   pos, B, N, H, Hkv, d, t, _handle(device, stream)), "fa_qk_norm_rope_fwd")
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
    if dk.shape != want or (dv is not None and dv.shape != want):
        raise ValueError("dk and dv must agree with dq")
    t = _transform(table, interleaved, q_weight, k_weight, eps, d, device)
    pos = _array(positions, _I32, lead, device, "positions")
    if norm and (q is None or k is None or q.shape != (*lead, H, d) or k.shape != (*lead, Hkv, d)):
        raise ValueError("q and k (the forward's inputs) are needed with norms")
    if dq_in is None and dk_in is None and dv_in is None:
        fused = torch.empty((*lead, H + (2 if dv is not None else 1) * Hkv, d), dtype=_BF16,
                            device=device)
        parts = fused.split([H, Hkv, Hkv] if dv is not None else [H, Hkv], dim=-2)
        dq_in, dk_in = parts[:2]
        dv_in = parts[2] if dv is not None else None
    empty = B == 0 or N == 0
    grad = out = x = None
    if not empty:
        dq_in, vq = _own_rows(dq_in, (*lead, H, d), out_order, device, "dq_in")
        dk_in, vk = _own_rows(dk_in, (*lead, Hkv, d), out_order, device, "dk_in")
        vv, gv = _NO_VIEW, _NO_VIEW
        if dv is not None:
            gv = _rows(dv, order, device, "dv")
            dv_in, vv = _own_rows(dv_in, (*lead, Hkv, d), out_order, device, "dv_in")
        grad = _VIEWS3.pack(*_rows(dq, order, device, "dq"), *_rows(dk, order, device, "dk"), *gv)
        out = _VIEWS3.pack(*vq, *vk, *vv)
        if norm:
            x = _VIEWS2.pack(*_rows(q, out_order, device, "q"), *_rows(k, out_order, device, "k"))
    dw = ws = None
    ws_at = ws_bytes = dw_at = 0
    if norm:
        dw = torch.empty((2, d), dtype=_F32, device=device)
        dw_at = dw.data_ptr()
        ws, ws_bytes = _workspace(workspace, fa_qk_norm_rope_bwd_workspace_size(d), device)
        ws_at = ws.data_ptr()
    _keep(stream, device, dq_in, dk_in, dv_in, dw, ws)
    _check(_launch(device, load_library().fa_qk_norm_rope_bwd, grad, x, out, dw_at,
                   dw_at + 4 * d if norm else 0, pos, max(B, 1), 0 if empty else N, H, Hkv, d, t,
                   ws_at, ws_bytes, _handle(device, stream)), "fa_qk_norm_rope_bwd")
    dwq, dwk = dw.unbind(0) if norm else (None, None)
    return dq_in, dk_in, dv_in if dv is not None else None, dwq, dwk


# ------------------------------------------------------------------------------------- paged cache
def _cache(k_cache, v_cache, block_table, kv_lens, device):
    """(fa_paged_kv, cache shape, block table's shape) after the checks of the cache's tensors."""
    if k_cache.dim() != 4 or block_table.dim() != 2:
        raise ValueError("k_cache must be [pages, Hkv, page_size, d], block_table [B, max_pages]")
    shape, of_table = k_cache.shape, block_table.shape
    return _PAGED_KV.pack(_array(k_cache, _BF16, shape, device, "k_cache"),
                          _array(v_cache, _BF16, shape, device, "v_cache"), shape[0], shape[2],
                          _array(block_table, _I32, of_table, device, "block_table"), of_table[1],
                          _array(kv_lens, _I32, of_table[:1], device, "kv_lens")), shape, of_table


def _tokens(cu_seqlens, B, total, device):
    if cu_seqlens is None:
        if total != B:
            raise ValueError("without cu_seqlens there is one token per sequence")
        return 0
    return _array(cu_seqlens, _I32, (B + 1,), device, "cu_seqlens")


def fa_kv_append(q, k, v, k_cache, v_cache, block_table, kv_lens, cu_seqlens=None,
                 pos_offset=None, table=None, interleaved=False, q_weight=None, k_weight=None,
                 eps=1e-6, q_out=None, stream=None):
    """Norms and rotation of the new tokens' q and k [total, heads, d] (strided views allowed),
    k and v written into the paged cache [pages, Hkv, page_size, d], q (or None) into a packed
    tensor, in one launch (see include/fa.h).  kv_lens counts the new tokens; cu_seqlens: their
    offsets, default one token per sequence; pos_offset: int32 [B] added to the rotation's
    positions.  Returns the transformed q (None without q)."""
    device = _cuda(k, "k")
    cache, (_, Hkv, _, d), (B, _) = _cache(k_cache, v_cache, block_table, kv_lens, device)
    if k.dim() != 3 or k.shape[1:] != (Hkv, d) or v.shape != k.shape:
        raise ValueError("k and v must be [total, Hkv, d] with the cache's heads")
    total, H = k.shape[0], Hkv
    if q is not None:
        if q.dim() != 3 or q.shape[0] != total or q.shape[2] != d:
            raise ValueError("q must be [total, H, d]")
        H = q.shape[1]
    cu = _tokens(cu_seqlens, B, total, device)
    offset = _array(pos_offset, _I32, (B,), device, "pos_offset")
    t = _transform(table, interleaved, q_weight, k_weight, eps, d, device)
    if total == 0:
        return None if q is None else torch.empty((0, H, d), dtype=_BF16, device=device)
    if q is None:
        q_out, vq, vo = None, _NO_VIEW, None
    else:
        vq = _rows(q, "nh", device, "q")
        q_out, vo = _own_rows(q_out, (total, H, d), "nh", device, "q_out")
        vo = _VIEW.pack(*vo)
        _keep(stream, device, q_out)
    views = _VIEWS3.pack(*vq, *_rows(k, "nh", device, "k"), *_rows(v, "nh", device, "v"))
    _check(_launch(device, load_library().fa_kv_append, views, vo, cache, cu, offset, B, total, H,
                   Hkv, d, t, _handle(device, stream)), "fa_kv_append")
    return q_out


def fa_fwd_paged_workspace_size(B, total, H, Hkv, d) -> int:
    return int(load_library().fa_fwd_paged_workspace_size(int(B), int(total), int(H), int(Hkv),
                                                          int(d)))


def fa_fwd_shared_prefix_workspace_size(B, groups, total, H, Hkv, d) -> int:
    return int(load_library().fa_fwd_shared_prefix_workspace_size(
        int(B), int(groups), int(total), int(H), int(Hkv), int(d)))


def _paged(q, k_cache, v_cache, block_table, kv_lens, prefix, groups, cu_seqlens, max_q, max_kv,
           causal, scale, out, lse, workspace, stream, device, where):
    cache, (_, Hkv, page, d), (B, pages) = _cache(k_cache, v_cache, block_table, kv_lens, device)
    if q.dim() != 3 or q.shape[2] != d or q.shape[1] % Hkv:
        raise ValueError("q must be [total, H, d] with H a multiple of the cache's heads")
    total, H, _ = q.shape
    at = _array(q, _BF16, q.shape, device, "q")
    cu = _tokens(cu_seqlens, B, total, device)
    if max_q is None:
        max_q = 1 if cu_seqlens is None else max(total, 1)
    if max_kv is None:
        max_kv = min(pages * page, 0x7fffffff)
    out = torch.empty_like(q) if out is None else _out(out, q.shape, _BF16, device, "out")
    lse = _out(lse, (H, total), _F32, device, "lse")
    lib = load_library()
    if prefix is None:
        need = lib.fa_fwd_paged_workspace_size(B, total, H, Hkv, d)
        call = lib.fa_fwd_paged
        head = (at, cache)
    else:
        need = lib.fa_fwd_shared_prefix_workspace_size(B, groups, total, H, Hkv, d)
        call = lib.fa_fwd_shared_prefix
        head = (at, cache, prefix)
    ws, ws_bytes = _workspace(workspace, need, device)
    _keep(stream, device, out, lse, ws)
    _check(_launch(device, call, *head, out.data_ptr(), lse.data_ptr(), cu, B, max_q, max_kv,
                   total, H, Hkv, d, 1 if causal else 0, _scale(scale), ws.data_ptr(), ws_bytes,
                   _handle(device, stream)), where)
    return out, lse


def fa_fwd_paged(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens=None, max_q=None,
                 max_kv=None, causal=False, scale=None, out=None, lse=None, workspace=None,
                 stream=None):
    """O [total, H, d] and LSE [H, total] of packed queries over the paged cache (see
    include/fa.h).  cu_seqlens: offsets of each sequence's query tokens, default one per
    sequence; causal aligns them to the end of the sequence.  max_q and max_kv bound the query
    tokens and keys of a sequence (defaults: total, and the block table's reach); close bounds
    let the launch fit the work."""
    return _paged(q, k_cache, v_cache, block_table, kv_lens, None, 0, cu_seqlens, max_q, max_kv,
                  causal, scale, out, lse, workspace, stream, _cuda(q, "q"), "fa_fwd_paged")


def fa_fwd_shared_prefix(q, k_cache, v_cache, block_table, kv_lens, prefix_table, prefix_lens,
                         group_cu, cu_seqlens=None, max_q=None, max_kv=None, max_prefix=None,
                         causal=False, scale=None, out=None, lse=None, workspace=None,
                         stream=None):
    """fa_fwd_paged for sequences that share prefixes held in the same cache (see include/fa.h):
    sequences [group_cu[g], group_cu[g + 1]) begin with the prefix_lens[g] keys in pages
    prefix_table[g]; block_table and kv_lens are their own keys behind it."""
    device = _cuda(q, "q")
    if prefix_table.dim() != 2:
        raise ValueError("prefix_table must be [groups, pages]")
    groups, pages = prefix_table.shape
    if max_prefix is None:
        max_prefix = min(pages * k_cache.shape[2], 0x7fffffff)
    prefix = _PREFIX.pack(_array(prefix_table, _I32, (groups, pages), device, "prefix_table"),
                          pages, _array(prefix_lens, _I32, (groups,), device, "prefix_lens"),
                          _array(group_cu, _I32, (groups + 1,), device, "group_cu"), groups,
                          max_prefix)
    return _paged(q, k_cache, v_cache, block_table, kv_lens, prefix, groups, cu_seqlens, max_q,
                  max_kv, causal, scale, out, lse, workspace, stream, device,
                  "fa_fwd_shared_prefix")
