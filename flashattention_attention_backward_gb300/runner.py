"""Convenience wrappers that allocate device memory with torch and call the
C ABI in stream order: forward (O, LSE), then preprocess -> attn_bwd ->
finalize, and the operators around them (rotary positions, layer norm,
dropout with a residual, a paged key/value cache). No arithmetic happens here; torch provides memory
and streams.

Streams: a call runs on `stream` (a torch stream, another object with a
`cuda_stream` handle, or a handle), by default the current one of its tensors'
device. What it allocates belongs to that stream, and its results may also be
used and dropped on the stream that was current at the call. Its inputs have to
be ready on `stream`, and stay alive until it has read them (hold them, or
`record_stream`), as with torch's own operations on a side stream.
"""
import torch

from . import (ATTN_BF16, ATTN_FP16, ATTN_FP32, ATTN_ROTARY_BASE, ATTN_ROTARY_LINEAR,
               ATTN_ROTARY_PLAIN, ATTN_ROTARY_RAMP, attn_bwd, attn_bwd_deterministic,
               attn_bwd_dq_partials_bytes, attn_bwd_dropout, attn_bwd_finalize,
               attn_bwd_finalize_partials, attn_bwd_finalize_rotary, attn_bwd_local,
               attn_bwd_preprocess, attn_bwd_sinks, attn_bwd_sum_partials, attn_cache_append,
               attn_cache_fwd, attn_cache_fwd_workspace_bytes, attn_dropout_add,
               attn_dropout_add_norm, attn_dropout_add_norm_bwd, attn_fwd, attn_fwd_dropout,
               attn_fwd_local, attn_fwd_ref, attn_fwd_ref_dropout, attn_fwd_ref_local,
               attn_fwd_ref_sinks, attn_fwd_sinks, attn_layer_norm,
               attn_layer_norm_bwd, attn_layer_norm_bwd_workspace_bytes, attn_rotary,
               attn_rotary_frequencies, check)

_DTYPES = {torch.bfloat16: ATTN_BF16, torch.float16: ATTN_FP16, torch.float32: ATTN_FP32}
_SCALINGS = {"plain": ATTN_ROTARY_PLAIN, "linear": ATTN_ROTARY_LINEAR, "base": ATTN_ROTARY_BASE,
             "ramp": ATTN_ROTARY_RAMP}


def _dims(q, k, *others):
    """(B, H, H_kv, N, d) of q [B,H,N,d] and k [B,H_kv,N,d], after checking
    what the C ABI assumes of its pointers: contiguous bf16 tensors on one
    CUDA device, with matching shapes (k, v alike; q, o, dO alike)."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be 4-D ([B, heads, N, d])")
    B, H, N, d = q.shape
    H_kv = k.shape[1]
    if k.shape != (B, H_kv, N, d):
        raise ValueError("k has shape %s, expected %s" % (tuple(k.shape), (B, H_kv, N, d)))
    for t in others:
        if t.shape not in (q.shape, k.shape):
            raise ValueError("tensor of shape %s matches neither q nor k" % (tuple(t.shape),))
    for t in (q, k) + others:
        if t.dtype != torch.bfloat16:
            raise ValueError("expected bfloat16 tensors, got %s" % t.dtype)
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous (row-major [B, heads, N, d])")
    for t in (q, k) + others:
        if t.device != q.device or t.device.type != "cuda":
            raise ValueError("all tensors must be on the same CUDA device")
    return B, H, H_kv, N, d


def _check_lse(lse, B, H, N, device):
    if lse.dtype != torch.float32 or not lse.is_contiguous() or tuple(lse.shape) != (B, H, N) \
            or lse.device != device:
        raise ValueError("lse must be a contiguous float32 [B, H, N] tensor on the inputs' device")


class _On:
    """The stream of a call on a device's tensors: current inside the context,
    as the device is. Memory allocated there comes from that stream's own
    blocks, so no work queued on another stream still reads what the call
    writes. Tensors handed back go through `made`."""

    def __init__(self, stream, device):
        current = torch.cuda.current_stream(device)
        self.stream, self.caller, self._context = current, None, None
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                handle = stream if isinstance(stream, int) else stream.cuda_stream
                stream = torch.cuda.ExternalStream(handle, device=device) if handle else \
                    torch.cuda.default_stream(device)
            if stream.device != device:
                raise ValueError("the stream is on %s, the tensors are on %s"
                                 % (stream.device, device))
            if stream != current:
                self.stream, self.caller = stream, current
                self._context = torch.cuda.stream(stream)
                return
        if torch.cuda.current_device() != device.index:
            self._context = torch.cuda.device(device)

    def __enter__(self):
        if self._context is not None:
            self._context.__enter__()
        return self

    def __exit__(self, *exc):
        if self._context is not None:
            self._context.__exit__(*exc)

    def made(self, *tensors):
        """Tells torch's allocator that the stream current at the call may use
        these tensors too: their memory is not handed out again before what is
        queued there when they are dropped has run."""
        self._record(self.caller, tensors)

    def given(self, *tensors):
        """The same of the call's stream and the caller's own tensors."""
        self._record(self.stream, tensors)

    def _record(self, stream, tensors):
        if self.caller is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)


def forward(q, k, v, scale, causal, softcap=0.0, stream=None, impl="tc", dropout=None,
            window=None, sinks=0):
    """O [B,H,N,d] bf16 and LSE [B,H,N] fp32: attn_fwd (tensor cores, impl
    "tc") or attn_fwd_ref (plain fp32, impl "ref"). dropout = (p_drop, seed)
    runs attn_fwd_dropout or attn_fwd_ref_dropout; window = (left, right) runs
    attn_fwd_local or attn_fwd_ref_local, with sinks = n (the first n keys stay
    visible to the left of the window) attn_fwd_sinks or attn_fwd_ref_sinks."""
    window, sinks = _check_sinks(sinks, window, dropout)
    B, H, H_kv, N, d = _dims(q, k, v)
    if v.shape != k.shape:
        raise ValueError("v must have the shape of k")
    args = (B, H, H_kv, N, d, scale, causal, softcap)
    if dropout is not None:
        fn = {"tc": attn_fwd_dropout, "ref": attn_fwd_ref_dropout}[impl]
        args += (dropout[0], dropout[1])
    elif sinks:
        fn = {"tc": attn_fwd_sinks, "ref": attn_fwd_ref_sinks}[impl]
        args += (window[0], window[1], sinks)
    elif window is not None:
        fn = {"tc": attn_fwd_local, "ref": attn_fwd_ref_local}[impl]
        args += (window[0], window[1])
    else:
        fn = {"tc": attn_fwd, "ref": attn_fwd_ref}[impl]
    with _On(stream, q.device) as on:
        o = torch.empty_like(q)
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
        check(fn(q, k, v, o, lse, *args, on.stream))
        on.made(o, lse)
    return o, lse


def _check_sinks(sinks, window, dropout):
    """(window, sinks) of a call: with sinks and no window, one without bounds."""
    if sinks < 0:
        raise ValueError("sinks must not be negative")
    if sinks and dropout is not None:
        raise ValueError("sinks have no dropout variant")
    if sinks and window is None:
        window = (-1, -1)
    return window if window is None else tuple(_bound(n) for n in window), _bound(sinks)


def _bound(n):
    """A count of keys as the C calls take it: an int keeps its low 32 bits on
    the way there, and every count from 2^30 on (past every position) hides
    and shows the same keys. Negative ones all mean no bound."""
    return max(-1, min(n, 1 << 30))


class BackwardBuffers:
    """Outputs and scratch of one backward problem, reusable across calls
    (calls that may run at the same time need their own). `stream`: the one that
    will use them, by default the current one; a call on another stream has to be
    ordered behind it first, as with any tensor made there."""

    def __init__(self, q, k, stream=None):
        dims = _dims(q, k)
        with _On(stream, q.device) as on:
            self._allocate(*dims, q.device)
            on.made(self.dq, self.dk, self.dv, self.dq_accum, self.dpsum)

    def _allocate(self, B, H, H_kv, N, d, dev):
        self.dq = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=dev)
        self.dk = torch.empty((B, H_kv, N, d), dtype=torch.bfloat16, device=dev)
        self.dv = torch.empty((B, H_kv, N, d), dtype=torch.bfloat16, device=dev)
        self.dq_accum = torch.empty((B, H, N, d), dtype=torch.float32, device=dev)
        self.dpsum = torch.empty((B, H, N), dtype=torch.float32, device=dev)
        self.dq_partials = None  # of the deterministic form, made by its first call
        return self


def backward(q, k, v, o, do, lse, scale, causal, softcap=0.0, stream=None, bufs=None,
             deterministic=False, dropout=None, window=None, rotary=None, positions=None,
             sinks=0):
    """dQ, dK, dV (bf16) via preprocess -> attn_bwd -> finalize, or, with
    deterministic=True, preprocess -> attn_bwd_deterministic ->
    finalize_partials (dQ identical bit for bit from run to run). window =
    (left, right) runs attn_bwd_local in place of attn_bwd, with sinks = n
    attn_bwd_sinks. rotary = the
    Rotary that q and k came from (with the same positions): dQ and dK are
    then the gradients of what went into it, each rounded once
    (attn_bwd_finalize_rotary in place of attn_bwd_finalize, and behind
    attn_bwd_sum_partials in the deterministic form)."""
    if sinks and deterministic:
        raise ValueError("sinks have no deterministic variant")
    window, sinks = _check_sinks(sinks, window, dropout)
    B, H, H_kv, N, d = _dims(q, k, v, o, do)
    if v.shape != k.shape or o.shape != q.shape or do.shape != q.shape:
        raise ValueError("v must have the shape of k, and o, dO that of q")
    _check_lse(lse, B, H, N, q.device)
    if rotary is not None:
        positions, pos_stride = _check_rotary(rotary, positions, B, N, d, q.device)
    elif positions is not None:
        raise ValueError("positions are those of a rotary")
    if dropout is None and window is not None and deterministic:
        raise ValueError("the local window has no deterministic variant")
    with _On(stream, q.device) as on:
        s, kept = on.stream, bufs is not None
        if not kept:
            bufs = object.__new__(BackwardBuffers)._allocate(B, H, H_kv, N, d, q.device)
            on.made(bufs.dq, bufs.dk, bufs.dv)
        shape = (B, H, H_kv, N, d, scale, causal, softcap, bufs.dpsum)
        if deterministic and dropout is None:
            _deterministic_dq_dk_dv(q, k, v, o, do, lse, bufs, kept, shape, s)
            if rotary is None:
                check(attn_bwd_finalize_partials(bufs.dq_partials, bufs.dq, scale, B, H, N, d,
                                                 causal, s))
                return bufs.dq, bufs.dk, bufs.dv
            check(attn_bwd_sum_partials(bufs.dq_partials, bufs.dq_accum, B, H, N, d, causal, s))
        else:
            check(attn_bwd_preprocess(o, do, bufs.dpsum, bufs.dq_accum, B, H, N, d, s))
            tensors = (q, k, v, o, do, lse, bufs.dq_accum, bufs.dk, bufs.dv)
            if dropout is not None:
                check(attn_bwd_dropout(*tensors, *shape, dropout[0], dropout[1], s))
            elif sinks:
                check(attn_bwd_sinks(*tensors, *shape, window[0], window[1], sinks, s))
            elif window is not None:
                check(attn_bwd_local(*tensors, *shape, window[0], window[1], s))
            else:
                check(attn_bwd(*tensors, *shape, s))
        if rotary is None:
            check(attn_bwd_finalize(bufs.dq_accum, bufs.dq, scale, B, H, N, d, s))
        else:
            check(attn_bwd_finalize_rotary(bufs.dq_accum, bufs.dq, bufs.dk, bufs.dk, scale,
                                           rotary.turns, positions, pos_stride, B, H, H_kv, N, d,
                                           rotary.rot, rotary.magnitude, rotary.interleaved, None,
                                           s))
        return bufs.dq, bufs.dk, bufs.dv


def _deterministic_dq_dk_dv(q, k, v, o, do, lse, bufs, kept, shape, s):
    """dQ's partial tiles, dK and dV; the partials' buffer grows with the problem
    (kept: it outlives the call)."""
    B, H, _, N, d, _, causal = shape[:7]
    nbytes = attn_bwd_dq_partials_bytes(B, H, N, d, causal)
    if nbytes < 0:
        check(int(nbytes))
    partials = getattr(bufs, "dq_partials", None)
    if partials is None or partials.numel() * 4 < nbytes:
        bufs.dq_partials = torch.empty(max(nbytes // 4, 4), dtype=torch.float32, device=q.device)
    if kept:  # a later call's larger one may replace it
        bufs.dq_partials.record_stream(s)
    check(attn_bwd_preprocess(o, do, bufs.dpsum, None, B, H, N, d, s))
    check(attn_bwd_deterministic(q, k, v, o, do, lse, bufs.dq_partials, bufs.dk, bufs.dv, *shape,
                                 s))


# ------------------------------------------------ around the attention call
def _check_cuda(device, **tensors):
    for name, t in tensors.items():
        if t is not None and (t.device != device or t.device.type != "cuda"):
            raise ValueError("%s must be on the same CUDA device as the other tensors" % name)


def _check_like(like, **tensors):
    """Contiguous tensors of like's shape and type."""
    for name, t in tensors.items():
        if t is None:
            continue
        if t.shape != like.shape or t.dtype != like.dtype:
            raise ValueError("%s must have the shape and dtype %s, %s" % (name, tuple(like.shape),
                                                                          like.dtype))
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)


class Rotary:
    """Rotary frequencies on a device: rot columns of each row turn, in pairs
    (i, i + rot / 2), or (2 i, 2 i + 1) with interleaved=True. scaling is
    "plain", "linear", "base" or "ramp" (attn_rotary_frequencies)."""

    def __init__(self, rot, device, base=10000.0, scaling="plain", factor=1.0, original_length=0,
                 low_turns=1.0, high_turns=32.0, interleaved=False):
        if scaling not in _SCALINGS:
            raise ValueError("scaling must be one of %s" % ", ".join(sorted(_SCALINGS)))
        rc, turns, self.magnitude = attn_rotary_frequencies(
            rot, base, _SCALINGS[scaling], factor, original_length, low_turns, high_turns)
        check(rc)
        self.rot, self.interleaved = int(rot), bool(interleaved)
        self.turns = torch.tensor(turns or [0], dtype=torch.int64, device=device)


def _check_rotary(plan, positions, B, N, d, device):
    """(positions, their batch stride) after checking them and the plan."""
    if plan.rot > d:
        raise ValueError("rot = %d exceeds the head dimension %d" % (plan.rot, d))
    _check_cuda(device, turns=plan.turns, positions=positions)
    if positions is None:
        return None, 0
    if positions.dtype != torch.int64 or tuple(positions.shape) not in ((N,), (B, N)):
        raise ValueError("positions must be an int64 tensor of shape [N] or [B, N]")
    if N > 1 and positions.stride(-1) != 1:
        raise ValueError("positions must be contiguous along N")
    return positions, positions.stride(0) if positions.dim() == 2 else 0


def rotary(q, k, plan, positions=None, adjoint=False, out=None, stream=None):
    """(q, k) rotated (attn_rotary), contiguous [B, heads, N, d]. q
    [B,H,N,d] and k [B,H_kv,N,d] (or None) may be strided as long as their
    rows are contiguous, e.g. parts of a packed [B, N, H + 2 H_kv, d]
    projection transposed. positions: int64 [N] or [B, N], default 0 .. N - 1.
    out = (q_out, k_out): written in place of new tensors (they may be strided
    too, and may be q and k)."""
    if q.dim() != 4 or (k is not None and k.dim() != 4):
        raise ValueError("q and k must be 4-D ([B, heads, N, d])")
    B, H, N, d = q.shape
    if k is not None and (k.shape[0], k.shape[2], k.shape[3]) != (B, N, d):
        raise ValueError("k has shape %s, expected [%d, heads, %d, %d]" % (tuple(k.shape), B, N, d))
    if q.dtype not in _DTYPES or (k is not None and k.dtype != q.dtype):
        raise ValueError("q and k must both be bfloat16, float16 or float32")
    given = (None, None) if out is None else out
    for x, y in ((q, given[0]), (k, given[1])):
        if x is None:
            continue
        if out is not None and (y is None or y.shape != x.shape or y.dtype != x.dtype):
            raise ValueError("out must have the shapes and dtype of q and k")
        if d > 1 and (x.stride(3) != 1 or (y is not None and y.stride(3) != 1)):
            raise ValueError("rows must be contiguous")
    _check_cuda(q.device, q=q, k=k, q_out=given[0], k_out=given[1])
    positions, pos_stride = _check_rotary(plan, positions, B, N, d, q.device)
    with _On(stream, q.device) as on:
        if out is None:
            out = (torch.empty(q.shape, dtype=q.dtype, device=q.device),
                   None if k is None else torch.empty(k.shape, dtype=k.dtype, device=k.device))
            on.made(*out)
        else:
            on.given(*out)
        parts = [q, q if k is None else k, out[0], out[0] if k is None else out[1]]
        strides = [v for t in parts for v in t.stride()[:3]]
        check(attn_rotary(q, k, out[0], out[1], plan.turns, positions, pos_stride, B, H,
                          0 if k is None else k.shape[1], N, d, plan.rot, plan.magnitude,
                          plan.interleaved, adjoint, _DTYPES[q.dtype], strides, on.stream))
    return out


def _check_cache(q, k_cache, v_cache, pages, starts, lengths, dtype):
    """(B, H_kv, d, page_size, max_pages, n_pages) of a batch over a cache."""
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must be 4-D of one shape "
                         "([pages, page size, heads, d])")
    n_pages, page_size, H_kv, d = k_cache.shape
    if dtype not in (torch.bfloat16, torch.float16) or k_cache.dtype != dtype or \
            v_cache.dtype != dtype:
        raise ValueError("the new tokens and the cache must all be bfloat16, or all float16")
    if d > 1 and (k_cache.stride(3) != 1 or v_cache.stride(3) != 1):
        raise ValueError("the cache's rows must be contiguous")
    if pages.dim() != 2 or lengths.shape != (pages.shape[0],) or \
            starts.shape != (pages.shape[0] + 1,):
        raise ValueError("pages must be [B, max_pages], lengths [B] and starts [B + 1]")
    for name, t in (("pages", pages), ("lengths", lengths), ("starts", starts)):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError("%s must be a contiguous int32 tensor" % name)
    if q is not None and (q.dim() != 3 or q.shape[2] != d):
        raise ValueError("expected rows [T, heads, %d]" % d)
    if q is not None and d > 1 and q.stride(2) != 1:
        raise ValueError("rows must be contiguous")
    if max(n_pages, page_size, pages.shape[1], 0 if q is None else q.shape[0]) >= 1 << 31:
        raise ValueError("sizes must stay below 2^31")
    _check_cuda(k_cache.device, k_cache=k_cache, v_cache=v_cache, pages=pages, starts=starts,
                lengths=lengths, q=q)
    return pages.shape[0], H_kv, d, page_size, pages.shape[1], n_pages


def cache_append(q, k, v, k_cache, v_cache, pages, starts, lengths, plan, out=None, stream=None):
    """The new tokens' keys (rotated by plan, a Rotary, to their positions) and
    values into a paged cache, and q rotated (attn_cache_append). q [T,H,d] (or
    None), k, v [T,H_kv,d], strided as long as rows are contiguous, e.g. parts
    of a packed [T, H + 2 H_kv, d] projection; k_cache, v_cache
    [pages, page size, H_kv, d] of any strides with contiguous rows; pages int32
    [B, max_pages], starts int32 [B + 1], lengths int32 [B]. out: written in
    place of a new tensor for q (may be q). Returns q rotated."""
    B, H_kv, d, page_size, max_pages, n_pages = _check_cache(
        q, k_cache, v_cache, pages, starts, lengths, k.dtype)
    for name, t in (("k", k), ("v", v)):
        if t.dim() != 3 or tuple(t.shape[1:]) != (H_kv, d) or t.shape[0] != k.shape[0] or \
                t.dtype != k.dtype:
            raise ValueError("%s must be [T, %d, %d] of k's dtype" % (name, H_kv, d))
        if d > 1 and t.stride(2) != 1:
            raise ValueError("rows must be contiguous")
    if k.shape[0] >= 1 << 31:
        raise ValueError("sizes must stay below 2^31")
    if q is not None and (q.shape[0] != k.shape[0] or q.dtype != k.dtype):
        raise ValueError("q must have k's rows and dtype")
    if out is not None:
        if q is None or out.shape != q.shape or out.dtype != q.dtype:
            raise ValueError("out must have the shape and dtype of q")
        if d > 1 and out.stride(2) != 1:
            raise ValueError("rows must be contiguous")
    if plan.rot > d:
        raise ValueError("rot = %d exceeds the head dimension %d" % (plan.rot, d))
    _check_cuda(k.device, k=k, v=v, k_cache=k_cache, out=out, turns=plan.turns)
    with _On(stream, k.device) as on:
        if out is not None:
            on.given(out)
        elif q is not None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            on.made(out)
        on.given(k_cache, v_cache)
        rows = [k if q is None else q, k, v, k if q is None else out]
        strides = [n for t in rows for n in t.stride()[:2]] + \
            [n for t in (k_cache, v_cache) for n in t.stride()[:3]]
        check(attn_cache_append(q, k, v, out, k_cache, v_cache, plan.turns, starts, lengths,
                                pages, k.shape[0], B, 0 if q is None else q.shape[1], H_kv, d,
                                plan.rot, plan.magnitude, plan.interleaved, page_size, max_pages,
                                n_pages, _DTYPES[k.dtype], strides, on.stream))
    return out


def cache_attention(q, k_cache, v_cache, pages, starts, lengths, scale, causal=True, softcap=0.0,
                    window_left=-1, sinks=0, out=None, workspace=None, stream=None):
    """(o, lse) of the new tokens' attention over a paged cache that holds their
    keys and values too (attn_cache_fwd): o [T,H,d] of q's type, lse [T,H] fp32.
    The cache, pages, starts and lengths are those of cache_append; window_left
    (negative: no bound) and sinks hide keys as the window and the sinks of
    forward do. out = (o, lse): written in place of new tensors, whose rows
    outside starts[0] .. starts[B] - 1 are undefined. workspace: a uint8 tensor of
    attn_cache_fwd_workspace_bytes, for one call at a time."""
    B, H_kv, d, page_size, max_pages, n_pages = _check_cache(
        q, k_cache, v_cache, pages, starts, lengths, q.dtype)
    T, H = q.shape[:2]
    if out is not None:
        if out[0].shape != q.shape or out[0].dtype != q.dtype or (d > 1 and
                                                                  out[0].stride(2) != 1):
            raise ValueError("out[0] must have the shape and dtype of q, and contiguous rows")
        if out[1].shape != (T, H) or out[1].dtype != torch.float32 or \
                not out[1].is_contiguous():
            raise ValueError("out[1] must be a contiguous float32 [%d, %d] tensor" % (T, H))
        _check_cuda(q.device, o=out[0], lse=out[1])
    nbytes = attn_cache_fwd_workspace_bytes(T, B, H, H_kv, d)
    if nbytes < 0:
        check(int(nbytes))
    if workspace is not None:
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or \
                workspace.numel() < nbytes:
            raise ValueError("workspace must be a contiguous uint8 tensor of %d bytes" % nbytes)
        _check_cuda(q.device, workspace=workspace)
    with _On(stream, q.device) as on:
        if out is None:
            out = (torch.empty(q.shape, dtype=q.dtype, device=q.device),
                   torch.empty((T, H), dtype=torch.float32, device=q.device))
            on.made(*out)
        else:
            on.given(*out)
        if workspace is None:
            workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
        else:
            on.given(workspace)
        strides = [n for t in (q, out[0]) for n in t.stride()[:2]] + \
            [n for t in (k_cache, v_cache) for n in t.stride()[:3]]
        check(attn_cache_fwd(q, k_cache, v_cache, out[0], out[1], starts, lengths, pages,
                             workspace, T, B, H, H_kv, d, page_size, max_pages, n_pages, scale,
                             causal, softcap, _bound(window_left), _bound(sinks), _DTYPES[q.dtype],
                             strides, on.stream))
    return out


def _norm_dims(x, gamma, beta):
    """(rows, C, dtype code, weight dtype code) of x [..., C]."""
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("expected a tensor [..., C] with C >= 1")
    if x.dtype not in _DTYPES:
        raise ValueError("expected a bfloat16, float16 or float32 tensor, got %s" % x.dtype)
    if not x.is_contiguous():
        raise ValueError("tensors must be contiguous")
    C = x.shape[-1]
    wd = None
    for name, w in (("gamma", gamma), ("beta", beta)):
        if w is None:
            continue
        if tuple(w.shape) != (C,) or not w.is_contiguous():
            raise ValueError("%s must be a contiguous [%d] tensor" % (name, C))
        if w.dtype not in _DTYPES or (wd is not None and w.dtype != wd):
            raise ValueError("gamma and beta must share one of the types bfloat16, float16, "
                             "float32")
        wd = w.dtype
    _check_cuda(x.device, x=x, gamma=gamma, beta=beta)
    return x.numel() // C, C, _DTYPES[x.dtype], _DTYPES[wd or x.dtype]


def _row_stats(x):
    return tuple(torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
                 for _ in range(2))


def layer_norm(x, gamma=None, beta=None, eps=1e-5, stream=None):
    """(y, mean, rstd) of x [..., C] (attn_layer_norm)."""
    rows, C, code, wcode = _norm_dims(x, gamma, beta)
    with _On(stream, x.device) as on:
        y = torch.empty_like(x)
        mean, rstd = _row_stats(x)
        check(attn_layer_norm(x, gamma, beta, y, mean, rstd, rows, C, eps, code, wcode,
                              on.stream))
        on.made(y, mean, rstd)
    return y, mean, rstd


def _check_stats(x, mean, rstd):
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t.dtype != torch.float32 or t.shape != x.shape[:-1] or not t.is_contiguous():
            raise ValueError("%s must be a contiguous float32 %s tensor"
                             % (name, list(x.shape[:-1])))
    _check_cuda(x.device, mean=mean, rstd=rstd)


def _weight_grads(x, gamma, want, rows, C, wdtype):
    """(dgamma, dbeta, workspace): None where not wanted."""
    if not want:
        return None, None, None
    nbytes = attn_layer_norm_bwd_workspace_bytes(rows, C)
    if nbytes < 0:
        check(int(nbytes))
    dt = gamma.dtype if gamma is not None else wdtype
    grads = [torch.empty(C, dtype=dt, device=x.device) for _ in range(2)]
    return grads[0], grads[1], torch.empty(nbytes // 4, dtype=torch.float32, device=x.device)


def layer_norm_backward(dy, x, gamma, mean, rstd, weight_grads=True, stream=None):
    """(dx, dgamma, dbeta) of layer_norm (attn_layer_norm_bwd); dgamma and
    dbeta have gamma's type (x's if gamma is None), or are None with
    weight_grads=False."""
    rows, C, code, wcode = _norm_dims(x, gamma, None)
    _check_like(x, dy=dy)
    _check_cuda(x.device, dy=dy)
    _check_stats(x, mean, rstd)
    with _On(stream, x.device) as on:
        dx = torch.empty_like(x)
        dgamma, dbeta, workspace = _weight_grads(x, gamma, weight_grads, rows, C, x.dtype)
        check(attn_layer_norm_bwd(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, workspace, rows, C,
                                  code, wcode, on.stream))
        on.made(dx, dgamma, dbeta)
    return dx, dgamma, dbeta


def dropout_add(x, residual=None, dropout=(0.0, 0), stream=None):
    """residual + dropout(x) (attn_dropout_add), dropout = (p_drop, seed); the
    adjoint is the call on dy without a residual."""
    if x.dtype not in _DTYPES:
        raise ValueError("expected a bfloat16, float16 or float32 tensor, got %s" % x.dtype)
    _check_like(x, x=x, residual=residual)
    _check_cuda(x.device, x=x, residual=residual)
    with _On(stream, x.device) as on:
        y = torch.empty_like(x)
        check(attn_dropout_add(x, residual, y, x.numel(), dropout[0], dropout[1],
                               _DTYPES[x.dtype], on.stream))
        on.made(y)
    return y


def dropout_add_norm(x, residual, gamma=None, beta=None, eps=1e-5, dropout=(0.0, 0), stream=None):
    """(z, y, mean, rstd): z = residual + dropout(x), y its layer norm
    (attn_dropout_add_norm)."""
    rows, C, code, wcode = _norm_dims(x, gamma, beta)
    _check_like(x, residual=residual)
    _check_cuda(x.device, residual=residual)
    with _On(stream, x.device) as on:
        z, y = torch.empty_like(x), torch.empty_like(x)
        mean, rstd = _row_stats(x)
        check(attn_dropout_add_norm(x, residual, gamma, beta, z, y, mean, rstd, rows, C, eps,
                                    dropout[0], dropout[1], code, wcode, on.stream))
        on.made(z, y, mean, rstd)
    return z, y, mean, rstd


def dropout_add_norm_backward(dy, dz, z, gamma, mean, rstd, dropout=(0.0, 0), weight_grads=True,
                              stream=None):
    """(dx, dresidual, dgamma, dbeta) of dropout_add_norm
    (attn_dropout_add_norm_bwd); dz is the gradient that reaches z by its
    other uses, or None. Without dropout dx is dresidual."""
    rows, C, code, wcode = _norm_dims(z, gamma, None)
    _check_like(z, dy=dy, dz=dz)
    _check_cuda(z.device, dy=dy, dz=dz)
    _check_stats(z, mean, rstd)
    with _On(stream, z.device) as on:
        dres = torch.empty_like(z)
        dx = torch.empty_like(z) if dropout[0] != 0 else None
        dgamma, dbeta, workspace = _weight_grads(z, gamma, weight_grads, rows, C, z.dtype)
        check(attn_dropout_add_norm_bwd(dy, dz, z, gamma, mean, rstd, dx, dres, dgamma, dbeta,
                                        workspace, rows, C, dropout[0], dropout[1], code, wcode,
                                        on.stream))
        on.made(dx, dres, dgamma, dbeta)
    return (dres if dx is None else dx), dres, dgamma, dbeta
