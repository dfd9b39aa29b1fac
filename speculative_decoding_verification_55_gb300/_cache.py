"""ctypes binding of the paged-cache calls of include/spec_verify.h under the same names.

Argument marshalling only, as in _binding: torch tensors supply device memory and the stream.
"""
from __future__ import annotations

import ctypes
import math
import threading

from ._binding import SV_DTYPE_BF16, SV_DTYPE_F16, SV_OK, SpecVerifyError, _on, _stream_handle, lib


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("slot_stride", ctypes.c_int64),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class PagedCache:
    """A batch's paged key-value cache (sv_paged_cache): k and v [num_pages, heads, page_size, D] in
    bfloat16 or float16 with D contiguous and any order of the other dimensions in memory (pass
    ``x.transpose(1, 2)`` for pages of [page_size, heads, D]), page_table [B, max_pages] int32 and,
    for the calls on attention weights, weight [num_pages, heads, page_size] float32. Holds the
    tensors; their contents may change between calls."""

    def __init__(self, k, v, page_table, weight=None):
        import torch
        if k.dim() != 4 or k.shape != v.shape:
            raise ValueError(f"k and v must be [num_pages, heads, page_size, D] of one shape, got "
                             f"{tuple(k.shape)} and {tuple(v.shape)}")
        if k.dtype not in (torch.bfloat16, torch.float16) or v.dtype != k.dtype:
            raise TypeError(f"k and v must both be bfloat16 or float16, got {k.dtype} and {v.dtype}")
        P, H, S, D = k.shape
        if page_table.dim() != 2 or page_table.dtype != torch.int32 or not page_table.is_contiguous():
            raise ValueError("page_table must be a contiguous [B, max_pages] int32 tensor")
        if weight is not None and (tuple(weight.shape) != (P, H, S) or weight.dtype != torch.float32
                                   or not weight.is_contiguous()):
            raise ValueError(f"weight must be a contiguous {(P, H, S)} float32 tensor")
        for name, t in (("v", v), ("page_table", page_table), ("weight", weight)):
            if t is not None and t.device != k.device:
                raise ValueError(f"{name} must be on {k.device}, got {t.device}")
        # The stride of a dimension of one element says nothing.
        steps = [[st if n > 1 else D for n, st in zip(t.shape[:3], t.stride()[:3])] for t in (k, v)]
        if D > 1 and (k.stride(3) != 1 or v.stride(3) != 1):
            raise ValueError("the D elements of an entry must be contiguous")
        if steps[0] != steps[1]:
            raise ValueError(f"k and v must have the same strides, got {k.stride()} and {v.stride()}")
        self.k, self.v, self.page_table, self.weight = k, v, page_table, weight
        self.B, self.heads, self.head_dim, self.dtype, self.device = page_table.shape[0], H, D, k.dtype, k.device
        self.struct = _CacheStruct(
            k.data_ptr(), v.data_ptr(), None if weight is None else weight.data_ptr(),
            page_table.data_ptr(), steps[0][0], steps[0][1], steps[0][2], P, S, page_table.shape[1],
            H, D, SV_DTYPE_BF16 if k.dtype == torch.bfloat16 else SV_DTYPE_F16)
        self.ref = ctypes.addressof(self.struct)
        self.workspace_need = {}


def _tokens(x, name, cache, N=None):
    """Checks a round's [B, N, heads, D] tensor; returns (N, heads, strides over rows and tokens)."""
    shape = x.shape
    if len(shape) != 4 or shape[0] != cache.B or shape[3] != cache.head_dim \
            or (N is not None and shape[1] != N):
        raise ValueError(f"{name} must be [{cache.B}, {'N' if N is None else N}, heads, "
                         f"{cache.head_dim}], got {tuple(shape)}")
    if x.dtype is not cache.dtype:
        raise TypeError(f"{name} must be {cache.dtype}, got {x.dtype}")
    if x.device != cache.device:
        raise ValueError(f"{name} must be on {cache.device}, got {x.device}")
    B, n, heads, D = shape
    s = x.stride()
    if s[3] != 1 or (heads > 1 and s[2] != D):
        raise ValueError(f"the heads of a token of {name} must be contiguous")
    return n, heads, (s[0] if B > 1 else heads * D * n), (s[1] if n > 1 else heads * D)


def _small(t, name, dtype, shape, device):
    """Address of a contiguous tensor of this type, shape and device (None -> NULL)."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {shape}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    return t.data_ptr()


def _raw_stream(stream, device):
    import torch
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    return _stream_handle(stream, device)


def _on_gpu(device):
    if device.type != "cuda":
        raise ValueError(f"the cache must be on a CUDA device, got {device}")


def _call(f, cache, stream, *args):
    """Calls f(*args, stream) with the cache's device current and raises on a nonzero status."""
    import torch
    dev = cache.device
    _on_gpu(dev)
    if torch._C._cuda_getDevice() == dev.index:
        st = f(*args, _raw_stream(stream, dev))
    else:
        with _on(dev):
            st = f(*args, _raw_stream(stream, dev))
    if st != SV_OK:
        raise SpecVerifyError(st, f.__name__)


def spec_verify_paged_attention_workspace_size(N: int, Hq: int, cache: PagedCache) -> int:
    return int(lib().spec_verify_paged_attention_workspace_size(N, Hq, cache.ref))


def spec_verify_kv_append(k_new, v_new, cache, prefix_len, num_new=None, path=None, out_len=None,
                          stream=None) -> None:
    """Calls the C ABI spec_verify_kv_append on torch tensors: token d (or path[:, d]) of k_new and
    v_new [B, N, heads, D] becomes entry prefix_len + d. Raises SpecVerifyError on a nonzero status."""
    import torch
    dev, B = cache.device, cache.B
    N, heads, rs, ts = _tokens(k_new, "k_new", cache)
    if _tokens(v_new, "v_new", cache, N) != (N, heads, rs, ts) or heads != cache.heads:
        raise ValueError(f"k_new and v_new must have {cache.heads} heads and the same strides")
    i32 = torch.int32
    _call(lib().spec_verify_kv_append, cache, stream, k_new.data_ptr(), v_new.data_ptr(), rs, ts, cache.ref,
          _small(prefix_len, "prefix_len", i32, (B,), dev), _small(num_new, "num_new", i32, (B,), dev),
          _small(path, "path", i32, (B, N), dev), _small(out_len, "out_len", i32, (B,), dev), B, N)


def _attention(q, cache, prefix_len, num_queries, tree_parents, N, Hq, rs, ts, out, out_lse, workspace,
               workspace_bytes, scale, stream):
    import torch
    dev, B, i32 = cache.device, cache.B, torch.int32
    _call(lib().spec_verify_paged_attention, cache, stream, q.data_ptr(), rs, ts, cache.ref,
          _small(prefix_len, "prefix_len", i32, (B,), dev), _small(num_queries, "num_queries", i32, (B,), dev),
          _small(tree_parents, "tree_parents", i32, (B, N), dev),
          1.0 / math.sqrt(cache.head_dim) if scale is None else scale, out, out_lse, B, N, Hq, workspace,
          workspace_bytes)


def spec_verify_paged_attention(q, cache, prefix_len, num_queries, tree_parents, out, out_lse,
                                workspace, scale=None, stream=None) -> None:
    """Calls the C ABI spec_verify_paged_attention on torch tensors: q [B, N, Hq, D] (heads of a token
    together), scale 1 / sqrt(D) unless given. Raises SpecVerifyError on a nonzero status."""
    import torch
    dev, B = cache.device, cache.B
    N, Hq, rs, ts = _tokens(q, "q", cache)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {dev}")
    _attention(q, cache, prefix_len, num_queries, tree_parents, N, Hq, rs, ts,
               _small(out, "out", cache.dtype, (B, N, Hq, cache.head_dim), dev),
               _small(out_lse, "out_lse", torch.float32, (B, N, Hq), dev), workspace.data_ptr(),
               workspace.nbytes, scale, stream)


def spec_verify_kv_weights(q, lse, cache, prefix_len, num_kept=None, path=None, scale=None,
                           stream=None) -> None:
    """Calls the C ABI spec_verify_kv_weights on torch tensors: cache.weight gains what the kept tokens
    of q [B, N, Hq, D] gave to each entry (lse: spec_verify_paged_attention's out_lse). Raises
    SpecVerifyError on a nonzero status."""
    import torch
    dev, B = cache.device, cache.B
    N, Hq, rs, ts = _tokens(q, "q", cache)
    i32 = torch.int32
    _call(lib().spec_verify_kv_weights, cache, stream, q.data_ptr(), rs, ts,
          _small(lse, "lse", torch.float32, (B, N, Hq), dev), cache.ref,
          _small(prefix_len, "prefix_len", i32, (B,), dev), _small(num_kept, "num_kept", i32, (B,), dev),
          _small(path, "path", i32, (B, N), dev),
          1.0 / math.sqrt(cache.head_dim) if scale is None else scale, B, N, Hq)


def spec_verify_kv_evict(cache, length, budget, recent, out_len, stream=None) -> None:
    """Calls the C ABI spec_verify_kv_evict on torch tensors: rows with more than budget entries keep
    the last ``recent`` and, per head, the others of the largest cache.weight. Raises SpecVerifyError on
    a nonzero status."""
    import torch
    dev, B = cache.device, cache.B
    _call(lib().spec_verify_kv_evict, cache, stream, cache.ref, _small(length, "length", torch.int32, (B,), dev),
          budget, recent, _small(out_len, "out_len", torch.int32, (B,), dev), B)


def spec_verify_shared_attention_workspace_size(B: int, N: int, Hq: int, groups: int, cache: PagedCache) -> int:
    return int(lib().spec_verify_shared_attention_workspace_size(B, N, Hq, groups, cache.ref))


def _starts(group_start, device):
    """(address, number of groups) of group_start [groups + 1]."""
    import torch
    if group_start.dim() != 1 or group_start.shape[0] < 2:
        raise ValueError(f"group_start must be [groups + 1], got {tuple(group_start.shape)}")
    return _small(group_start, "group_start", torch.int32, group_start.shape, device), group_start.shape[0] - 1


def _shared_attention(q, cache, prefix_len, shared_len, start, groups, num_queries, tree_parents, N, Hq, rs, ts, out,
                      out_lse, workspace, workspace_bytes, scale, stream):
    import torch
    dev, B, i32 = cache.device, cache.B, torch.int32
    if B > 1 and N > 1 and rs != N * ts:
        raise ValueError(f"the rows of q must follow one another: strides {q.stride()}")
    _call(lib().spec_verify_shared_attention, cache, stream, q.data_ptr(), rs, ts, cache.ref,
          _small(prefix_len, "prefix_len", i32, (B,), dev), _small(shared_len, "shared_len", i32, (B,), dev), start, groups,
          _small(num_queries, "num_queries", i32, (B,), dev), _small(tree_parents, "tree_parents", i32, (B, N), dev),
          1.0 / math.sqrt(cache.head_dim) if scale is None else scale, out, out_lse, B, N, Hq, workspace,
          workspace_bytes)


def spec_verify_shared_attention(q, cache, prefix_len, shared_len, group_start, num_queries, tree_parents, out, out_lse,
                                 workspace, scale=None, stream=None) -> None:
    """Calls the C ABI spec_verify_shared_attention on torch tensors: spec_verify_paged_attention of rows
    group_start[g] .. group_start[g + 1] - 1 whose first shared_len entries are the same pages. The rows of q [B, N, Hq,
    D] follow one another. Raises SpecVerifyError on a nonzero status."""
    import torch
    dev, B = cache.device, cache.B
    N, Hq, rs, ts = _tokens(q, "q", cache)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {dev}")
    _shared_attention(q, cache, prefix_len, shared_len, *_starts(group_start, dev), num_queries, tree_parents, N, Hq, rs, ts,
                      _small(out, "out", cache.dtype, (B, N, Hq, cache.head_dim), dev),
                      _small(out_lse, "out_lse", torch.float32, (B, N, Hq), dev), workspace.data_ptr(),
                      workspace.nbytes, scale, stream)


_attend_ws = {}
# A call makes two or three launches on its stream's workspace: another thread's must not come in between.
_attend_lock = threading.Lock()


def _attend_workspace(N, Hq, cache, groups=0):
    """A workspace cached per (device, current stream) and grown on demand. A call that is being captured
    gets one of its own: replays of two graphs may overlap."""
    import torch
    need = cache.workspace_need.get((N, Hq, groups))
    if need is None:
        need = spec_verify_shared_attention_workspace_size(cache.B, N, Hq, groups, cache) if groups \
            else spec_verify_paged_attention_workspace_size(N, Hq, cache)
        cache.workspace_need[N, Hq, groups] = need
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(need, dtype=torch.uint8, device=cache.device)
    key = (cache.device, _raw_stream(None, cache.device))
    ws = _attend_ws.get(key)
    if ws is None or ws.nbytes < need:
        ws = _attend_ws[key] = torch.empty(need, dtype=torch.uint8, device=cache.device)
    return ws


def attend(q, cache, prefix_len, num_queries=None, tree_parents=None, scale=None, stream=None):
    """Allocates the outputs, runs spec_verify_paged_attention and returns (out [B, N, Hq, D],
    lse [B, N, Hq]), both of the given stream (the current one unless given). Host threads may call it at once."""
    import torch
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), cache.device)
        with torch.cuda.stream(stream):
            return attend(q, cache, prefix_len, num_queries, tree_parents, scale)
    N, Hq, rs, ts = _tokens(q, "q", cache)
    _on_gpu(cache.device)
    out = torch.empty((cache.B, N, Hq, cache.head_dim), dtype=q.dtype, device=cache.device)
    lse = torch.empty((cache.B, N, Hq), dtype=torch.float32, device=cache.device)
    with _attend_lock:
        ws = _attend_workspace(N, Hq, cache)
        _attention(q, cache, prefix_len, num_queries, tree_parents, N, Hq, rs, ts, out.data_ptr(), lse.data_ptr(),
                   ws.data_ptr(), ws.nbytes, scale, None)
    return out, lse


def attend_shared(q, cache, prefix_len, shared_len, group_start, num_queries=None, tree_parents=None, scale=None, stream=None):
    """attend of a batch whose rows share the fronts of their contexts, each front read once for many of its rows' queries:
    rows group_start[g] .. group_start[g + 1] - 1 have their first shared_len[b] entries, whole pages, in common. Returns
    (out, lse) as attend does."""
    import torch
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), cache.device)
        with torch.cuda.stream(stream):
            return attend_shared(q, cache, prefix_len, shared_len, group_start, num_queries, tree_parents, scale)
    N, Hq, rs, ts = _tokens(q, "q", cache)
    _on_gpu(cache.device)
    start, groups = _starts(group_start, cache.device)
    out = torch.empty((cache.B, N, Hq, cache.head_dim), dtype=q.dtype, device=cache.device)
    lse = torch.empty((cache.B, N, Hq), dtype=torch.float32, device=cache.device)
    with _attend_lock:
        ws = _attend_workspace(N, Hq, cache, groups)
        _shared_attention(q, cache, prefix_len, shared_len, start, groups, num_queries, tree_parents, N, Hq, rs, ts,
                          out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.nbytes, scale, None)
    return out, lse
