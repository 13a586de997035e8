"""The paged key/value cache in 4 bits: quantizing new tokens into it, reading
it back, and attention over it (the binding of fp4q_kv_* of include/fp4q.h).

A cache is four uint8 planes of pages, [pages, kv_heads, page_size, bytes] in
any memory order (a cache kept [pages, page_size, kv_heads, bytes] is passed
as its .transpose(1, 2)): packed E2M1 codes, head_dim / 2 bytes a row, and
block scales, head_dim / 16 E4M3 bytes for "nvfp4" or head_dim / 32 E8M0 bytes
for "mxfp4".  NVFP4 keys and values each have one fp32 tensor scale g, fixed
before the first token is written (quantize_nvfp4 of a calibration tensor
returns one as global_scale).
"""
import torch

from . import _lib

__all__ = ["KvCache", "kv_cache", "kv_cache_write", "kv_cache_read", "kv_cache_attention",
           "kv_cache_attention_workspace_bytes"]

_FORMATS = {"nvfp4": (_lib.FP4Q_NVFP4, 16), "mxfp4": (_lib.FP4Q_MXFP4, 32)}
_DTYPES = {torch.float32: _lib.FP4Q_F32, torch.bfloat16: _lib.FP4Q_BF16}
_ROTATIONS = {None: _lib.FP4Q_ROT_NONE, "none": _lib.FP4Q_ROT_NONE, "fwht128": _lib.FP4Q_ROT_FWHT128}


class KvCache:
    """A cache over planes that the caller owns.  Checked once, here; the
    calls below take it as it is."""

    def __init__(self, format, k_codes, k_scales, v_codes, v_scales, k_global=None, v_global=None):
        if format not in _FORMATS:
            raise ValueError("fp4q: a cache's format is 'nvfp4' or 'mxfp4', got %r" % (format,))
        code, block = _FORMATS[format]
        planes = (("k_codes", k_codes), ("k_scales", k_scales), ("v_codes", v_codes), ("v_scales", v_scales))
        for what, t in planes:
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise ValueError("fp4q: %s must be a GPU tensor" % what)
            if t.dtype != torch.uint8 or t.dim() != 4:
                raise ValueError("fp4q: %s must be uint8 [pages, kv_heads, page_size, bytes]" % what)
            if t.device != k_codes.device:
                raise ValueError("fp4q: the planes of a cache must be on one device")
            if t.shape[3] > 1 and t.stride(3) != 1:
                raise ValueError("fp4q: rows of %s must be contiguous (stride(3) == 1)" % what)
        pages, heads, page, half = k_codes.shape
        scales = (pages, heads, page, half * 2 // block)
        if half * 2 % 32 or v_codes.shape != k_codes.shape or tuple(k_scales.shape) != scales \
                or v_scales.shape != k_scales.shape:
            raise ValueError("fp4q: inconsistent cache planes: codes %s and %s, scales %s and %s" %
                             tuple(tuple(t.shape) for t in (k_codes, v_codes, k_scales, v_scales)))
        if k_codes.stride() != v_codes.stride() or k_scales.stride() != v_scales.stride():
            raise ValueError("fp4q: key and value planes must have the same strides")
        if format == "nvfp4":
            for what, t in (("k_global", k_global), ("v_global", v_global)):
                if not isinstance(t, torch.Tensor) or t.device != k_codes.device or t.dtype != torch.float32 \
                        or t.numel() != 1:
                    raise ValueError("fp4q: %s must be one float32 on the cache's device" % what)
        else:
            k_global = v_global = None
        self.format, self.head_dim, self.kv_heads, self.page_size, self.num_pages = format, half * 2, heads, page, pages
        self.device = k_codes.device
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.k_global, self.v_global = k_global, v_global
        # (the planes are kept here, so that the addresses stay theirs)
        a = _lib.KvCacheArgs()
        a.format, a.kv_heads, a.head_dim, a.page_size, a.num_pages = code, heads, half * 2, page, pages
        for what, t in planes:
            setattr(a, what, t.data_ptr())
        if k_global is not None:
            a.k_global, a.v_global = k_global.data_ptr(), v_global.data_ptr()
        a.code_stride[:] = k_codes.stride()[:3]
        a.scale_stride[:] = k_scales.stride()[:3]
        self._args = a
        self._index = k_codes.get_device()


def kv_cache(num_pages, page_size, kv_heads, head_dim, *, format="nvfp4", k_global=1.0, v_global=1.0, device="cuda"):
    """A zeroed cache, [pages, kv_heads, page_size, bytes] dense.  k_global,
    v_global: the NVFP4 tensor scales, floats or one-element float32 tensors."""
    if format not in _FORMATS:
        raise ValueError("fp4q: a cache's format is 'nvfp4' or 'mxfp4', got %r" % (format,))
    if head_dim % 32:
        raise ValueError("fp4q: head_dim must be a multiple of 32, got %d" % head_dim)
    block = _FORMATS[format][1]
    widths = (head_dim // 2, head_dim // block) * 2
    planes = [torch.zeros((num_pages, kv_heads, page_size, w), dtype=torch.uint8, device=device) for w in widths]
    if format == "mxfp4":
        return KvCache(format, *planes)
    scales = [g if isinstance(g, torch.Tensor) else torch.full((1,), float(g), dtype=torch.float32, device=device)
              for g in (k_global, v_global)]
    return KvCache(format, *planes, *scales)


# The raw handle of a device's current stream; what torch.cuda.current_stream()
# wraps into an object, which takes as long as a small kernel.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(cache, function, *args):
    """function(*args) with the cache's device as the current one."""
    if torch.cuda.current_device() == cache._index:
        return function(*args)
    with torch.cuda.device(cache._index):
        return function(*args)


def _rotation(rotation):
    try:
        return _ROTATIONS[rotation]
    except (KeyError, TypeError):
        raise ValueError("fp4q: a cache's rotation is None or 'fwht128', got %r" % (rotation,)) from None


def _rows(t, what, cache, heads):
    """Checks a [tokens, heads, head_dim] tensor of fp32 or bf16 on the cache's
    device; its shape, strides and dtype code."""
    if not isinstance(t, torch.Tensor) or t.get_device() != cache._index:
        raise ValueError("fp4q: %s must be a tensor on the cache's device" % what)
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError("fp4q: %s must be float32 or bfloat16, got %s" % (what, t.dtype))
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[2] != cache.head_dim or (heads and shape[1] != heads):
        raise ValueError("fp4q: %s must be [tokens, %s, %d], got %s" % (what, heads or "heads", cache.head_dim, tuple(shape)))
    if stride[2] != 1:
        raise ValueError("fp4q: rows of %s must be contiguous (stride(2) == 1)" % what)
    return shape, stride, code


def _index(t, what, cache, dtype, dims):
    if not isinstance(t, torch.Tensor) or t.get_device() != cache._index or t.dtype != dtype or t.dim() != dims:
        raise ValueError("fp4q: %s must be a %d-D %s tensor on the cache's device" % (what, dims, dtype))
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError("fp4q: %s must be contiguous along its last dimension" % what)
    return t.shape


def _int32(x):
    """x as far as 32 bits go (ctypes would keep its low bits); what is negative
    stays so."""
    return max(-1, min(int(x), 2 ** 31 - 1))


def _table(page_table, cache):
    """Sequences, pages a sequence and the row stride of a page table."""
    seqs, cols = _index(page_table, "page_table", cache, torch.int32, 2)
    return seqs, cols, max(page_table.stride(0), cols) if seqs <= 1 else page_table.stride(0)


def kv_cache_write(cache, k, v, slots, *, rotation=None):
    """Quantize new tokens' keys and values, [tokens, kv_heads, head_dim] fp32
    or bf16 (any 16-byte aligned token and head strides, e.g. slices of a
    projection), into the cache.

    slots: int64 [tokens], page * page_size + offset of each token; a token
    whose slot lies outside the cache (a negative one, say) is skipped, and no
    two tokens of a call share a slot.  rotation "fwht128" stores the keys in
    the basis of the normalised Hadamard transform of each 128 elements
    (head_dim a multiple of 128); pass the same to kv_cache_attention and
    kv_cache_read.  The bytes are those of quantize_nvfp4 / quantize_mxfp4."""
    shape, ks, code = _rows(k, "k", cache, cache.kv_heads)
    v_shape, vs, v_code = _rows(v, "v", cache, cache.kv_heads)
    if shape != v_shape or code != v_code:
        raise ValueError("fp4q: k and v must have the same shape and dtype")
    if _index(slots, "slots", cache, torch.int64, 1)[0] != shape[0]:
        raise ValueError("fp4q: slots must have one entry a token")
    a = _lib.KvWriteArgs(shape[0], k.data_ptr(), v.data_ptr(), ks[:2], vs[:2], slots.data_ptr(), code,
                         _rotation(rotation))
    status = _call(cache, _lib.load().fp4q_kv_write, cache._args, a, _raw_stream(cache._index))
    if status:
        _lib.check(status, "fp4q_kv_write")


def kv_cache_read(cache, page_table, cu, *, total, starts=None, rotation=None, out_dtype=torch.bfloat16, out=None):
    """The values that the cache holds of runs of tokens: (k, v), each [total,
    kv_heads, head_dim] in out_dtype.

    page_table: int32 [seqs, pages]; cu: int32 [seqs + 1], output rows cu[b]
    to cu[b + 1] - 1 are tokens starts[b] (0 without starts, int32 [seqs])
    onwards of sequence b; total: rows of the output.  Keys written with a
    rotation come back in their original basis when it is given here.  out: a
    pair of buffers to write, either of them None to leave it out."""
    seqs, cols, stride = _table(page_table, cache)
    if _index(cu, "cu", cache, torch.int32, 1)[0] != seqs + 1:
        raise ValueError("fp4q: cu must have one entry more than page_table has rows")
    if starts is not None and _index(starts, "starts", cache, torch.int32, 1)[0] != seqs:
        raise ValueError("fp4q: starts must have one entry a sequence")
    code = _DTYPES.get(out_dtype)
    if code is None:
        raise TypeError("fp4q: out_dtype must be float32 or bfloat16, got %s" % out_dtype)
    shape = (int(total), cache.kv_heads, cache.head_dim)
    if out is None:
        out = (torch.empty(shape, dtype=out_dtype, device=cache.device),
               torch.empty(shape, dtype=out_dtype, device=cache.device))
    else:
        for t in out:
            if t is not None and (t.get_device() != cache._index or t.dtype != out_dtype or tuple(t.shape) != shape
                                  or not t.is_contiguous()):
                raise ValueError("fp4q: out must be contiguous %s tensors of shape %s" % (out_dtype, shape))
    k_out, v_out = (None if t is None else t.data_ptr() for t in out)
    a = _lib.KvReadArgs(page_table.data_ptr(), stride, cols, seqs, cu.data_ptr(),
                        None if starts is None else starts.data_ptr(), shape[0], k_out, v_out, code,
                        _rotation(rotation))
    status = _call(cache, _lib.load().fp4q_kv_read, cache._args, a, _raw_stream(cache._index))
    if status:
        _lib.check(status, "fp4q_kv_read")
    return out


# One zeroed workspace per (device, stream), grown as calls need it: calls on
# one stream are ordered, and a call leaves its counters zero.  Smaller ones
# are kept too, since captured calls go on using them.
_workspaces = {}
_outgrown = []


def _grow_workspace(cache, a, stream):
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError("fp4q: the workspace of this stream is missing or too small; pass workspace= or make one "
                           "call of this size on the stream before capturing it")
    need = _lib.load().fp4q_kv_attention_workspace_bytes(cache._args, a)
    old = _workspaces.get((cache._index, stream))
    if old is not None:
        _outgrown.append(old)
    ws = _workspaces[(cache._index, stream)] = torch.zeros(need, dtype=torch.uint8, device=cache.device)
    return ws


def kv_cache_attention_workspace_bytes(q, cache, page_table, *, max_q=1, window=0):
    """Bytes of the workspace= that kv_cache_attention takes for these
    arguments (max_q 1 where it is called without cu_q)."""
    shape, qs, code = _rows(q, "q", cache, 0)
    seqs, cols, stride = _table(page_table, cache)
    # (shapes decide; the tensors that are not at hand stand in for each other)
    at = page_table.data_ptr() or cache.k_codes.data_ptr()
    a = _lib.KvAttentionArgs(q.data_ptr(), qs[:2], q.data_ptr(), None, at, at, at, stride, shape[0], cols, seqs,
                             _int32(max_q), shape[1], code, 1, _int32(window), _lib.FP4Q_ROT_NONE, 1.0)
    return _lib.load().fp4q_kv_attention_workspace_bytes(cache._args, a)


def kv_cache_attention(q, cache, page_table, seq_lens, *, cu_q=None, max_q=None, scale=None, causal=True, window=0,
                       rotation=None, out=None, return_lse=False, workspace=None):
    """softmax(scale q k^T) v over the cache: q [total, q_heads, head_dim],
    fp32 or bf16, q_heads a multiple of the cache's heads (consecutive query
    heads share one); head_dim 64, 96, 128 or 256.

    page_table: int32 [seqs, pages]; seq_lens: int32 [seqs], the tokens in the
    cache, new ones among them.  Without cu_q each sequence has one query;
    with cu_q (int32 [seqs + 1]) sequence b's are rows cu_q[b] to
    cu_q[b + 1] - 1, at most max_q (default: all rows) in any; rows from
    cu_q[seqs] on, and those of a sequence past max_q, are zeros.  causal: query
    i of m sees token j <= n - m + i of the n; window > 0: only the last
    `window` of them.  scale: 1 / sqrt(head_dim) by default.  rotation: as the
    keys were written.

    Returns out [total, q_heads, head_dim] in q's dtype, or (out, lse) with
    the fp32 log-sum-exps [total, q_heads].  A query that sees no token gives
    zeros and -inf.  Nothing waits for the GPU: lengths and tables are read
    there, so a captured call may be replayed with others in place.  Calls on
    one stream share a workspace that is kept for it; workspace: another one
    (a zeroed GPU tensor of kv_cache_attention_workspace_bytes bytes, for calls
    on other streams at the same time, replays of captured ones among them)."""
    shape, qs, code = _rows(q, "q", cache, 0)
    seqs, cols, stride = _table(page_table, cache)
    total, q_heads = shape[0], shape[1]
    if _index(seq_lens, "seq_lens", cache, torch.int32, 1)[0] != seqs:
        raise ValueError("fp4q: seq_lens must have one entry a sequence")
    cu = None
    if cu_q is None:
        if total != seqs:
            raise ValueError("fp4q: without cu_q, q must have one row a sequence")
        max_q = 1
    else:
        if _index(cu_q, "cu_q", cache, torch.int32, 1)[0] != seqs + 1:
            raise ValueError("fp4q: cu_q must have one entry more than there are sequences")
        cu = cu_q.data_ptr()
        max_q = total if max_q is None else _int32(max_q)
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=cache.device)
    elif out.get_device() != cache._index or out.dtype != q.dtype or out.shape != shape or not out.is_contiguous():
        raise ValueError("fp4q: out must be a contiguous %s tensor of shape %s" % (q.dtype, tuple(shape)))
    lse = torch.empty((total, q_heads), dtype=torch.float32, device=cache.device) if return_lse else None
    a = _lib.KvAttentionArgs(q.data_ptr(), qs[:2], out.data_ptr(), lse.data_ptr() if return_lse else None, cu,
                             seq_lens.data_ptr(), page_table.data_ptr(), stride, total, cols, seqs, max_q, q_heads,
                             code, 1 if causal else 0, _int32(window), _rotation(rotation),
                             cache.head_dim ** -0.5 if scale is None else float(scale))
    run, stream = _lib.load().fp4q_kv_attention, _raw_stream(cache._index)
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.get_device() != cache._index \
                or not workspace.is_contiguous():
            raise ValueError("fp4q: the workspace must be a contiguous tensor on the cache's device")
        status = _call(cache, run, cache._args, a, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                       stream)
    else:
        ws, status = _workspaces.get((cache._index, stream)), _lib.FP4Q_ERR_WORKSPACE
        if ws is not None:
            status = _call(cache, run, cache._args, a, ws.data_ptr(), ws.numel(), stream)
        if status == _lib.FP4Q_ERR_WORKSPACE:
            ws = _grow_workspace(cache, a, stream)
            status = _call(cache, run, cache._args, a, ws.data_ptr(), ws.numel(), stream)
    if status:
        _lib.check(status, "fp4q_kv_attention")
    return (out, lse) if return_lse else out
