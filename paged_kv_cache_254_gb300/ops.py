"""Python entry points with the C ABI's names: torch tensors in, kernels run.

PyTorch supplies device memory and streams only.  Each function checks that
its tensors sit on one CUDA device with the expected dtype and layout, then
calls the matching ``pa_*`` function of libpa.so on the current stream.
"""

from __future__ import annotations

import ctypes
import threading

import torch

from . import _lib

_DTYPES = {torch.float16: _lib.PA_FP16, torch.bfloat16: _lib.PA_BF16}


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(device, stream=None) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _need_cuda(name, t, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def make_shape(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, max_blocks_per_seq,
               dtype) -> _lib.PaShape:
    return _lib.PaShape(int(num_seqs), int(num_q_heads), int(num_kv_heads), int(head_dim), int(block_size),
                        int(num_blocks), int(max_blocks_per_seq), _DTYPES[dtype])


def _pool_shape(k_pool, num_seqs=0, num_q_heads=1, max_blocks=1) -> _lib.PaShape:
    NB, Hkv, B, d = k_pool.shape
    return make_shape(num_seqs, num_q_heads, Hkv, d, B, NB, max_blocks, k_pool.dtype)


def pa_decode_workspace_bytes(q, k_pool, block_tables) -> int:
    N, Hq, _ = q.shape
    shape = _pool_shape(k_pool, N, Hq, block_tables.shape[1])
    with torch.cuda.device(q.device):
        return int(_lib.load().pa_decode_workspace_bytes(ctypes.byref(shape)))


_ws_lock = threading.Lock()
_ws_cache = {}


def workspace_for(q, k_pool, block_tables, stream=None) -> torch.Tensor:
    """A pa_decode workspace kept per (device, stream) and grown on demand, for
    callers that pass one; pa_decode clears its counter region itself, so the
    buffer is reused as is.  Every caller on the stream gets the same one:
    threads that share a stream need their own, or none (see _lend)."""
    need = pa_decode_workspace_bytes(q, k_pool, block_tables)
    if need == 0:
        return torch.empty(0, dtype=torch.uint8, device=q.device)
    s = stream if stream is not None else torch.cuda.current_stream(q.device)
    key = (q.device.index, s.cuda_stream)
    with _ws_lock:
        ws = _ws_cache.get(key)
        if ws is None or ws.numel() < need:
            ws = torch.zeros(max(need, 1 << 20), dtype=torch.uint8, device=q.device)
            _ws_cache[key] = ws
        return ws


# Workspaces of calls that are given none, by (device index, stream handle).
_sp_cache = {}


def _lend(given, index, handle, need, call, stream=None):
    """call(workspace) with the one given, or with one of ``need`` bytes that
    is this call's alone until it returns.

    A call is several launches that hand their intermediate state over in the
    workspace, and other threads may queue work on the same stream between
    them.  So the stream's workspace leaves ``_sp_cache`` for the call (dict.pop
    is one step under the interpreter lock); a call that finds none allocates,
    and the larger one is kept.  Everything stays in the stream's order, so a
    workspace that is dropped or used again meets no work of its last call.
    A captured call's belongs to its graph: the stream's may be replaced by a
    larger one, and another graph may run beside this one.  ``stream`` is the
    call's, where the memory has to belong, if that is not the current one."""
    if given is not None:
        return call(given)
    key = (index, handle)
    with torch.cuda.stream(stream):                      # None: where we are
        capturing = torch.cuda.is_current_stream_capturing()
        ws = None if capturing else _sp_cache.pop(key, None)
        if ws is None or ws.numel() < need:
            size = need if capturing else max(need, 1 << 20)
            ws = torch.empty(size, dtype=torch.uint8, device=f"cuda:{index}")
    if capturing:
        return call(ws)
    try:
        return call(ws)
    finally:
        other = _sp_cache.get(key)
        if other is None or other.numel() < ws.numel():
            _sp_cache[key] = ws


def new_error_word(device) -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device)


def pa_decode(q, k_pool, v_pool, block_tables, context_lens, scale, out=None, workspace=None, err=None,
              stream=None):
    """out[N, Hq, d] = paged decode attention of q over the pools (see include/pa.h)."""
    _need_cuda("q", q)
    _need_cuda("k_pool", k_pool, q.dtype)
    _need_cuda("v_pool", v_pool, q.dtype)
    _need_cuda("block_tables", block_tables, torch.int32)
    _need_cuda("context_lens", context_lens, torch.int32)
    if q.dtype not in _DTYPES:
        raise TypeError("q must be float16 or bfloat16")
    if k_pool.shape != v_pool.shape or k_pool.dim() != 4 or q.dim() != 3:
        raise ValueError("q [N, Hq, d], k_pool and v_pool [NB, Hkv, B, d]")
    N, Hq, d = q.shape
    if k_pool.shape[3] != d or block_tables.dim() != 2 or block_tables.shape[0] != N or context_lens.shape != (N,):
        raise ValueError("shape mismatch between q, pools, block_tables and context_lens")
    if out is None:
        out = torch.empty_like(q)
    else:
        _need_cuda("out", out, q.dtype)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if workspace is not None:
        _need_cuda("workspace", workspace)
    if err is not None:
        _need_cuda("err", err, torch.int32)
    shape = _pool_shape(k_pool, N, Hq, block_tables.shape[1])
    lib = _lib.load()
    with torch.cuda.device(q.device):
        need = 0 if workspace is not None else int(lib.pa_decode_workspace_bytes(ctypes.byref(shape)))
        s = _stream(q.device, stream)
        st = _lend(workspace, q.device.index, s.value or 0, need,
                   lambda ws: lib.pa_decode(ctypes.byref(shape), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_tables),
                                            _ptr(context_lens), ctypes.c_float(scale), _ptr(out), _ptr(ws),
                                            ctypes.c_size_t(ws.numel() * ws.element_size()), _ptr(err), s), stream)
    _lib.check(st, "pa_decode")
    return out


def pa_append_kv(k_new, v_new, slot_mapping, k_pool, v_pool, err=None, stream=None):
    """Write k_new/v_new [T, Hkv, d] into the pools at slot_mapping [T] (int64; < 0 skips)."""
    _need_cuda("k_pool", k_pool)
    _need_cuda("v_pool", v_pool, k_pool.dtype)
    _need_cuda("k_new", k_new, k_pool.dtype)
    _need_cuda("v_new", v_new, k_pool.dtype)
    _need_cuda("slot_mapping", slot_mapping, torch.int64)
    T = slot_mapping.shape[0]
    if k_new.shape != (T,) + tuple(k_pool.shape[1:2]) + tuple(k_pool.shape[3:]) or v_new.shape != k_new.shape:
        raise ValueError("k_new, v_new must be [T, Hkv, d]")
    if err is not None:
        _need_cuda("err", err, torch.int32)
    shape = _pool_shape(k_pool)
    with torch.cuda.device(k_pool.device):
        st = _lib.load().pa_append_kv(ctypes.byref(shape), ctypes.c_int32(T), _ptr(k_new), _ptr(v_new),
                                      _ptr(slot_mapping), _ptr(k_pool), _ptr(v_pool), _ptr(err),
                                      _stream(k_pool.device, stream))
    _lib.check(st, "pa_append_kv")


def pa_copy_blocks(src_dst_pairs, k_pool, v_pool, err=None, stream=None):
    """Copy whole blocks src -> dst for each row of src_dst_pairs [n, 2] (int32)."""
    _need_cuda("k_pool", k_pool)
    _need_cuda("v_pool", v_pool, k_pool.dtype)
    _need_cuda("src_dst_pairs", src_dst_pairs, torch.int32)
    if src_dst_pairs.dim() != 2 or src_dst_pairs.shape[1] != 2:
        raise ValueError("src_dst_pairs must be [n, 2]")
    if err is not None:
        _need_cuda("err", err, torch.int32)
    shape = _pool_shape(k_pool)
    with torch.cuda.device(k_pool.device):
        st = _lib.load().pa_copy_blocks(ctypes.byref(shape), _ptr(src_dst_pairs),
                                        ctypes.c_int32(src_dst_pairs.shape[0]), _ptr(k_pool), _ptr(v_pool),
                                        _ptr(err), _stream(k_pool.device, stream))
    _lib.check(st, "pa_copy_blocks")


def pa_set_decode_stall_ns(wait_ns: int) -> None:
    """Fault injection for tests (see include/pa.h): with wait_ns > 0 every
    later decode launch, and every launch of pa_decode_multi_bs8's chunk
    kernel, makes each worker's first stage wait on a barrier that nothing
    completes, for at most wait_ns, so the kernel's timeout path
    runs; 0 turns it off."""
    _lib.check(_lib.load().pa_set_decode_stall_ns(ctypes.c_uint64(int(wait_ns))), "pa_set_decode_stall_ns")


def pa_read_error(err, stream=None) -> int:
    """Synchronise the stream and return the status the error word maps to."""
    _need_cuda("err", err, torch.int32)
    with torch.cuda.device(err.device):
        return int(_lib.load().pa_read_error(_ptr(err), _stream(err.device, stream)))


def pa_decode_shared_prefix(q, k_pool, v_pool, block_tables, context_lens, group_starts, group_prefix_blocks,
                            scale, out=None, workspace=None, err=None, stream=None):
    """Prefix-aware decode (see include/pa.h): group_starts [G + 1] and
    group_prefix_blocks [G] are int32 CUDA tensors describing sequences that
    share their leading blocks."""
    _need_cuda("q", q)
    _need_cuda("k_pool", k_pool, q.dtype)
    _need_cuda("v_pool", v_pool, q.dtype)
    _need_cuda("block_tables", block_tables, torch.int32)
    _need_cuda("context_lens", context_lens, torch.int32)
    _need_cuda("group_starts", group_starts, torch.int32)
    _need_cuda("group_prefix_blocks", group_prefix_blocks, torch.int32)
    n_groups = group_prefix_blocks.shape[0]
    if group_starts.shape != (n_groups + 1,):
        raise ValueError("group_starts must have one more entry than group_prefix_blocks")
    N, Hq, d = q.shape
    if k_pool.shape != v_pool.shape or k_pool.shape[3] != d or block_tables.shape[0] != N:
        raise ValueError("shape mismatch between q, pools and block_tables")
    if out is None:
        out = torch.empty_like(q)
    else:
        _need_cuda("out", out, q.dtype)
    shape = _pool_shape(k_pool, N, Hq, block_tables.shape[1])
    lib = _lib.load()
    with torch.cuda.device(q.device):
        need = int(lib.pa_decode_shared_prefix_workspace_bytes(ctypes.byref(shape)))
        if workspace is not None:
            _need_cuda("workspace", workspace)
        if err is not None:
            _need_cuda("err", err, torch.int32)
        s = _stream(q.device, stream)
        st = _lend(workspace, q.device.index, s.value or 0, need,
                   lambda ws: lib.pa_decode_shared_prefix(
                       ctypes.byref(shape), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_tables), _ptr(context_lens),
                       ctypes.c_int32(n_groups), _ptr(group_starts), _ptr(group_prefix_blocks), ctypes.c_float(scale),
                       _ptr(out), _ptr(ws), ctypes.c_size_t(ws.numel() * ws.element_size()), _ptr(err), s), stream)
    _lib.check(st, "pa_decode_shared_prefix")
    return out


def pa_decode_multi(q, k_pool, v_pool, block_tables, context_lens, q_start, scale, max_q_len=None,
                    out=None, workspace=None, err=None, stream=None):
    """Multi-token query paged attention (see include/pa.h): q [T, Hq, d]
    holds each sequence's chunk of new tokens at rows q_start[b] ..
    q_start[b + 1] - 1 (q_start: int32 CUDA tensor [N + 1]); token i of a
    chunk attends causally to keys t <= ctx - q_len + i.  max_q_len defaults
    to the largest chunk (read from q_start on the host)."""
    _need_cuda("q", q)
    _need_cuda("k_pool", k_pool, q.dtype)
    _need_cuda("v_pool", v_pool, q.dtype)
    _need_cuda("block_tables", block_tables, torch.int32)
    _need_cuda("context_lens", context_lens, torch.int32)
    _need_cuda("q_start", q_start, torch.int32)
    T, Hq, d = q.shape
    N = block_tables.shape[0]
    if q_start.shape != (N + 1,) or context_lens.shape != (N,):
        raise ValueError("q_start must have N + 1 entries and context_lens N")
    if k_pool.shape != v_pool.shape or k_pool.shape[3] != d:
        raise ValueError("shape mismatch between q and the pools")
    if max_q_len is None:
        qs = q_start.cpu()
        max_q_len = max(1, int((qs[1:] - qs[:-1]).max().item())) if N > 0 else 1
    if out is None:
        out = torch.empty_like(q)
    else:
        _need_cuda("out", out, q.dtype)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    shape = _pool_shape(k_pool, N, Hq, block_tables.shape[1])
    lib = _lib.load()
    with torch.cuda.device(q.device):
        need = int(lib.pa_decode_multi_workspace_bytes(ctypes.byref(shape), ctypes.c_int32(max_q_len)))
        if need == 0 and workspace is None:
            # an invalid shape or chunk bound: let the call report which
            workspace = torch.empty(0, dtype=torch.uint8, device=q.device)
        elif workspace is not None:
            _need_cuda("workspace", workspace)
        if err is not None:
            _need_cuda("err", err, torch.int32)
        s = _stream(q.device, stream)
        st = _lend(workspace, q.device.index, s.value or 0, need,
                   lambda ws: lib.pa_decode_multi(
                       ctypes.byref(shape), ctypes.c_int32(max_q_len), ctypes.c_int32(T), _ptr(q), _ptr(q_start),
                       _ptr(k_pool), _ptr(v_pool), _ptr(block_tables), _ptr(context_lens), ctypes.c_float(scale),
                       _ptr(out), _ptr(ws), ctypes.c_size_t(ws.numel() * ws.element_size()), _ptr(err), s), stream)
    _lib.check(st, "pa_decode_multi")
    return out


# --------------------------------------------------------------------------- drafted trees, rotary positions
# These calls run beside kernels of a few microseconds, so calls in order go
# through a compiled twin of their host side (csrc/fast_calls.cpp), which
# declines whatever is not plainly right; the checks below then say what is
# wrong, or do what is rare (a first workspace, another device, a capture).
_raw_stream = torch._C._cuda_getCurrentRawStream


def _arg(name, t, dtype, device):
    """``t`` is a contiguous tensor of ``dtype`` on CUDA device ``device``."""
    if isinstance(t, torch.Tensor) and t.get_device() == device and t.dtype is dtype and t.is_contiguous():
        return
    _need_cuda(name, t, dtype)
    raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")


def _index(name, t) -> int:
    """The CUDA device of the argument that the others have to share."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    return t.get_device()


def _call(fn, device, *args):
    """Call a library function with CUDA device ``device`` current."""
    if torch.cuda.current_device() == device:
        return fn(*args)
    with torch.cuda.device(device):
        return fn(*args)


def _addr(t):
    return None if t is None else t.data_ptr()


def _on_stream(stream, fn, *args):
    """fn(*args) with ``stream`` current, so that what it allocates belongs to
    the stream, and its arguments' memory is not reused before the stream has
    passed the call."""
    for t in args:
        if isinstance(t, torch.Tensor) and t.is_cuda and t.device != stream.device:
            raise ValueError(f"the stream is on {stream.device}, a tensor on {t.device}")
    with torch.cuda.stream(stream):
        result = fn(*args)
    for t in args:
        if isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(stream)
    return result


def _largest_chunk(q_start) -> int:
    """The longest chunk, read on the host (q_start may yet be of any shape)."""
    sizes = q_start.detach().flatten().cpu().diff()
    return max(1, int(sizes.max().item())) if sizes.numel() else 1


_fast = None


def _load_fast():
    global _fast
    _fast = _lib.load_fast()
    return _fast


_tree_bytes = {}


def _tree_workspace_bytes(dev, shape, max_nodes):
    # the size of a valid shape's workspace depends on these and the device's SM count alone
    key = (dev, max_nodes, shape.num_seqs, shape.num_q_heads, shape.num_kv_heads, shape.head_dim, shape.block_size,
           shape.dtype)
    need = _tree_bytes.get(key)
    if need is None:
        need = int(_call(_lib.load().pa_decode_tree_workspace_bytes, dev, shape, max_nodes))
        if need:                         # 0: something about the shape is invalid, which the call reports
            _tree_bytes[key] = need
    return need


def pa_decode_tree(q, k_pool, v_pool, block_tables, context_lens, q_start, tree_masks, scale, max_nodes=None,
                   out=None, workspace=None, err=None, stream=None):
    """Attention of drafted trees over the cache (see include/pa.h): q
    [T, Hq, d] holds each sequence's nodes at rows q_start[b] .. q_start[b + 1]
    - 1 (q_start: int32 [N + 1]); bit j of tree_masks [T] (int64, see
    ``tree_masks()``) lets a row see node j of its own tree, next to every key
    cached before the tree.  max_nodes (1..64) defaults to the largest tree
    (read from q_start on the host)."""
    if stream is not None:
        return _on_stream(stream, pa_decode_tree, q, k_pool, v_pool, block_tables, context_lens, q_start,
                          tree_masks, scale, max_nodes, out, workspace, err)
    if max_nodes is None and isinstance(q_start, torch.Tensor):
        max_nodes = _largest_chunk(q_start)
    args = (q, k_pool, v_pool, block_tables, context_lens, q_start, tree_masks, scale, max_nodes, out, workspace, err)
    done = (_fast or _load_fast()).decode_tree(_sp_cache, *args)
    return _decode_tree(*args) if done is NotImplemented else done


def _decode_tree(q, k_pool, v_pool, block_tables, context_lens, q_start, tree_masks, scale, max_nodes, out,
                 workspace, err):
    """pa_decode_tree by way of every check."""
    dev = _index("q", q)
    if not 1 <= max_nodes <= 64:
        raise ValueError("max_nodes must be 1..64")
    dt = q.dtype
    if dt not in _DTYPES:
        raise TypeError("q must be float16 or bfloat16")
    _arg("q", q, dt, dev)
    _arg("k_pool", k_pool, dt, dev)
    _arg("v_pool", v_pool, dt, dev)
    _arg("block_tables", block_tables, torch.int32, dev)
    _arg("context_lens", context_lens, torch.int32, dev)
    _arg("q_start", q_start, torch.int32, dev)
    _arg("tree_masks", tree_masks, torch.int64, dev)
    if q.dim() != 3 or k_pool.dim() != 4 or block_tables.dim() != 2:
        raise ValueError("q [T, Hq, d], k_pool and v_pool [NB, Hkv, B, d], block_tables [N, MB]")
    T, Hq, d = q.shape
    N, MB = block_tables.shape
    pool = k_pool.shape
    if q_start.shape != (N + 1,) or context_lens.shape != (N,) or tree_masks.shape != (T,):
        raise ValueError("q_start must have N + 1 entries, context_lens N and tree_masks T")
    if pool != v_pool.shape or pool[3] != d:
        raise ValueError("shape mismatch between q and the pools")
    if out is None:
        out = torch.empty_like(q)
    else:
        _arg("out", out, dt, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if err is not None:
        _arg("err", err, torch.int32, dev)
    shape = _lib.PaShape(N, Hq, pool[1], d, pool[2], pool[0], MB, _DTYPES[dt])
    need = 0
    if workspace is not None:
        _arg("workspace", workspace, workspace.dtype, dev)
    else:
        need = _tree_workspace_bytes(dev, shape, max_nodes)
        if need == 0:
            workspace = torch.empty(0, dtype=torch.uint8, device=q.device)
    handle = _raw_stream(dev)
    st = _lend(workspace, dev, handle, need,
               lambda ws: _call(_lib.load().pa_decode_tree, dev, shape, max_nodes, T, q.data_ptr(), q_start.data_ptr(),
                                tree_masks.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), block_tables.data_ptr(),
                                context_lens.data_ptr(), scale, out.data_ptr(), ws.data_ptr(), ws.nbytes, _addr(err),
                                handle))
    if st:
        _lib.check(st, "pa_decode_tree")
    return out


def pa_tree_verify(tree_masks, draft_tokens, target_tokens, q_start, context_lens, max_nodes=None, path=None,
                   err=None, stream=None):
    """The drafted path that the target model's tokens agree with (see
    include/pa.h).  Returns (path int32 [N, max_nodes], num_accepted int32 [N],
    next_tokens int64 [N], new_context_lens int32 [N])."""
    if stream is not None:
        return _on_stream(stream, pa_tree_verify, tree_masks, draft_tokens, target_tokens, q_start, context_lens,
                          max_nodes, path, err)
    if max_nodes is None and isinstance(q_start, torch.Tensor):
        max_nodes = _largest_chunk(q_start)
    args = (tree_masks, draft_tokens, target_tokens, q_start, context_lens, max_nodes, path, err)
    done = (_fast or _load_fast()).tree_verify(*args)
    return _tree_verify(*args) if done is NotImplemented else done


def _tree_verify(tree_masks, draft_tokens, target_tokens, q_start, context_lens, max_nodes, path, err):
    """pa_tree_verify by way of every check."""
    dev = _index("tree_masks", tree_masks)
    if not 1 <= max_nodes <= 64:
        raise ValueError("max_nodes must be 1..64")
    _arg("tree_masks", tree_masks, torch.int64, dev)
    _arg("draft_tokens", draft_tokens, torch.int64, dev)
    _arg("target_tokens", target_tokens, torch.int64, dev)
    _arg("q_start", q_start, torch.int32, dev)
    _arg("context_lens", context_lens, torch.int32, dev)
    if tree_masks.dim() != 1 or context_lens.dim() != 1:
        raise ValueError("tree_masks [T], context_lens [N]")
    T, N = tree_masks.shape[0], context_lens.shape[0]
    if draft_tokens.shape != (T,) or target_tokens.shape != (T,) or q_start.shape != (N + 1,):
        raise ValueError("draft_tokens and target_tokens must have tree_masks' shape, q_start N + 1 entries")
    if path is None:
        path = torch.empty((N, max_nodes), dtype=torch.int32, device=context_lens.device)
    else:
        _arg("path", path, torch.int32, dev)
        if path.shape != (N, max_nodes):
            raise ValueError("path must be [N, max_nodes]")
    if err is not None:
        _arg("err", err, torch.int32, dev)
    accepted, lens = torch.empty_like(context_lens), torch.empty_like(context_lens)
    following = torch.empty(N, dtype=torch.int64, device=context_lens.device)
    st = _call(_lib.load().pa_tree_verify, dev, N, max_nodes, T, q_start.data_ptr(), tree_masks.data_ptr(),
               draft_tokens.data_ptr(), target_tokens.data_ptr(), context_lens.data_ptr(), path.data_ptr(),
               accepted.data_ptr(), following.data_ptr(), lens.data_ptr(), _addr(err), _raw_stream(dev))
    if st:
        _lib.check(st, "pa_tree_verify")
    return path, accepted, following, lens


def pa_keep_kv(path, q_start, context_lens, block_tables, k_pool, v_pool, err=None, stream=None):
    """Move the accepted tokens' K and V rows to consecutive positions behind
    each sequence's context (see include/pa.h); path int32 [N, max_nodes] and
    the context lengths are those of the tree."""
    if stream is not None:
        return _on_stream(stream, pa_keep_kv, path, q_start, context_lens, block_tables, k_pool, v_pool, err)
    args = (path, q_start, context_lens, block_tables, k_pool, v_pool, err)
    if (_fast or _load_fast()).keep_kv(*args) is NotImplemented:
        _keep_kv(*args)


def _keep_kv(path, q_start, context_lens, block_tables, k_pool, v_pool, err):
    """pa_keep_kv by way of every check."""
    dev = _index("k_pool", k_pool)
    dt = k_pool.dtype
    if dt not in _DTYPES:
        raise TypeError("the pools must be float16 or bfloat16")
    _arg("k_pool", k_pool, dt, dev)
    _arg("v_pool", v_pool, dt, dev)
    _arg("path", path, torch.int32, dev)
    _arg("q_start", q_start, torch.int32, dev)
    _arg("context_lens", context_lens, torch.int32, dev)
    _arg("block_tables", block_tables, torch.int32, dev)
    pool = k_pool.shape
    if path.dim() != 2 or block_tables.dim() != 2 or len(pool) != 4 or pool != v_pool.shape:
        raise ValueError("path [N, max_nodes], block_tables [N, MB], k_pool and v_pool [NB, Hkv, B, d]")
    N, P = path.shape
    if q_start.shape != (N + 1,) or context_lens.shape != (N,) or block_tables.shape[0] != N:
        raise ValueError("q_start must have N + 1 entries, context_lens and block_tables N")
    if err is not None:
        _arg("err", err, torch.int32, dev)
    shape = _lib.PaShape(N, 1, pool[1], pool[3], pool[2], pool[0], block_tables.shape[1], _DTYPES[dt])
    st = _call(_lib.load().pa_keep_kv, dev, shape, P, path.data_ptr(), q_start.data_ptr(), block_tables.data_ptr(),
               context_lens.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), _addr(err), _raw_stream(dev))
    if st:
        _lib.check(st, "pa_keep_kv")


def _token_rows(name, t, dtype, shape, device):
    """Elements between the tokens of ``t`` [T, H, d], whose heads are
    contiguous within a token."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    T, H, d = shape
    st, sh, sd = t.stride()
    if T == 0:
        return H * d                                    # nothing is read
    if sd != 1 or (sh != d and H > 1):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    if T == 1:
        return H * d                                    # a single token's own stride is never used
    if st < H * d:
        raise ValueError(f"{name}: tokens must not overlap")
    return st


def pa_rope_append_kv(q, k_new, v_new, positions, slot_mapping, k_pool, v_pool, inv_freq, interleaved=False,
                      rope_scale=1.0, q_weight=None, k_weight=None, eps=1e-6, out=None, err=None, stream=None):
    """Norm (with q_weight / k_weight) and rotate queries and keys, write keys
    and values into the pools at slot_mapping, and return the queries
    [T, Hq, d] (see include/pa.h).  q, k_new, v_new [T, heads, d] may be views
    of one projection's output; inv_freq [rotary_dim / 2] fp32 as from
    ``rope_inv_freq()``, or None for no rotation; out may be q."""
    if stream is not None:
        return _on_stream(stream, pa_rope_append_kv, q, k_new, v_new, positions, slot_mapping, k_pool, v_pool,
                          inv_freq, interleaved, rope_scale, q_weight, k_weight, eps, out, err)
    args = (q, k_new, v_new, positions, slot_mapping, k_pool, v_pool, inv_freq, interleaved, rope_scale, q_weight,
            k_weight, eps, out, err)
    done = (_fast or _load_fast()).rope_append_kv(*args)
    return _rope_append_kv(*args) if done is NotImplemented else done


def _rope_append_kv(q, k_new, v_new, positions, slot_mapping, k_pool, v_pool, inv_freq, interleaved, rope_scale,
                    q_weight, k_weight, eps, out, err):
    """pa_rope_append_kv by way of every check."""
    dev = _index("k_pool", k_pool)
    dt = k_pool.dtype
    if dt not in _DTYPES:
        raise TypeError("the pools must be float16 or bfloat16")
    _arg("k_pool", k_pool, dt, dev)
    _arg("v_pool", v_pool, dt, dev)
    pool = k_pool.shape
    if len(pool) != 4 or pool != v_pool.shape:
        raise ValueError("k_pool and v_pool must be [NB, Hkv, B, d]")
    NB, Hkv, B, d = pool
    if not isinstance(q, torch.Tensor) or q.dim() != 3 or q.shape[2] != d:
        raise ValueError("q must be a tensor [T, Hq, d] with the pools' d")
    T, Hq, _ = q.shape
    qs = _token_rows("q", q, dt, (T, Hq, d), dev)
    ks = _token_rows("k_new", k_new, dt, (T, Hkv, d), dev)
    vs = _token_rows("v_new", v_new, dt, (T, Hkv, d), dev)
    _arg("positions", positions, torch.int32, dev)
    _arg("slot_mapping", slot_mapping, torch.int64, dev)
    if positions.shape != (T,) or slot_mapping.shape != (T,):
        raise ValueError("positions and slot_mapping must be [T]")
    rotary = 0
    if inv_freq is not None:
        _arg("inv_freq", inv_freq, torch.float32, dev)
        if inv_freq.dim() != 1 or 2 * inv_freq.shape[0] > d:
            raise ValueError("inv_freq must be [rotary_dim / 2] with rotary_dim <= d")
        rotary = 2 * inv_freq.shape[0]
    if q_weight is not None:
        _arg("q_weight", q_weight, dt, dev)
        if q_weight.shape != (d,):
            raise ValueError("q_weight must be [d]")
    if k_weight is not None:
        _arg("k_weight", k_weight, dt, dev)
        if k_weight.shape != (d,):
            raise ValueError("k_weight must be [d]")
    if out is None:
        out = torch.empty_like(q) if q.is_contiguous() else torch.empty((T, Hq, d), dtype=dt, device=q.device)
    else:
        _arg("out", out, dt, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if err is not None:
        _arg("err", err, torch.int32, dev)
    shape = _lib.PaShape(0, Hq, Hkv, d, B, NB, 1, _DTYPES[dt])
    rope = _lib.PaRope(_addr(inv_freq) if rotary else None, rotary, 1 if interleaved else 0, rope_scale, eps,
                       _addr(q_weight), _addr(k_weight))
    st = _call(_lib.load().pa_rope_append_kv, dev, shape, rope, T, q.data_ptr(), qs, k_new.data_ptr(), ks,
               v_new.data_ptr(), vs, positions.data_ptr(), slot_mapping.data_ptr(), out.data_ptr(),
               k_pool.data_ptr(), v_pool.data_ptr(), _addr(err), _raw_stream(dev))
    if st:
        _lib.check(st, "pa_rope_append_kv")
    return out


KV_FORMATS = {"e4m3": _lib.PA_FP8_E4M3, "e5m2": _lib.PA_FP8_E5M2}


def _need_pool8(kv_pool):
    _need_cuda("kv_pool", kv_pool, torch.uint8)
    if kv_pool.dim() != 5 or kv_pool.shape[2] != 2:
        raise ValueError("kv_pool must be uint8 [NB, Hkv, 2, B, d] (the V half stored dims-first)")
    return kv_pool.shape[0], kv_pool.shape[1], kv_pool.shape[3], kv_pool.shape[4]


def pa_decode_fp8(q, kv_pool, block_tables, context_lens, scale, k_scale, v_scale, kv_format="e4m3", out=None,
                  workspace=None, err=None, stream=None):
    """Decode over the 8-bit cache (see include/pa.h)."""
    _need_cuda("q", q)
    _need_cuda("block_tables", block_tables, torch.int32)
    _need_cuda("context_lens", context_lens, torch.int32)
    NB, Hkv, B, d = _need_pool8(kv_pool)
    N, Hq, dq = q.shape
    if dq != d or block_tables.shape[0] != N:
        raise ValueError("q [N, Hq, d] and kv_pool [NB, Hkv, 2, B, d] disagree")
    out = torch.empty_like(q) if out is None else out
    fmt = KV_FORMATS[kv_format]
    shape = make_shape(N, Hq, Hkv, d, B, NB, block_tables.shape[1], q.dtype)
    lib = _lib.load()
    with torch.cuda.device(q.device):
        need = 0 if workspace is not None else int(lib.pa_decode_fp8_workspace_bytes(ctypes.byref(shape), fmt))
        s = _stream(q.device, stream)
        st = _lend(workspace, q.device.index, s.value or 0, max(need, 1),
                   lambda ws: lib.pa_decode_fp8(ctypes.byref(shape), fmt, _ptr(q), _ptr(kv_pool), _ptr(block_tables),
                                                _ptr(context_lens), ctypes.c_float(scale), ctypes.c_float(k_scale),
                                                ctypes.c_float(v_scale), _ptr(out), _ptr(ws),
                                                ctypes.c_size_t(ws.numel() * ws.element_size()), _ptr(err), s), stream)
    _lib.check(st, "pa_decode_fp8")
    return out


def pa_append_kv_fp8(k_new, v_new, slot_mapping, kv_pool, k_scale, v_scale, kv_format="e4m3", err=None,
                     stream=None):
    """Quantize k_new / v_new [T, Hkv, d] (fp16/bf16) into the 8-bit pool."""
    _need_cuda("k_new", k_new)
    _need_cuda("v_new", v_new, k_new.dtype)
    _need_cuda("slot_mapping", slot_mapping, torch.int64)
    NB, Hkv, B, d = _need_pool8(kv_pool)
    T = slot_mapping.shape[0]
    shape = make_shape(0, 1, Hkv, d, B, NB, 1, k_new.dtype)
    with torch.cuda.device(kv_pool.device):
        st = _lib.load().pa_append_kv_fp8(ctypes.byref(shape), KV_FORMATS[kv_format], ctypes.c_int32(T),
                                          _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(kv_pool),
                                          ctypes.c_float(k_scale), ctypes.c_float(v_scale), _ptr(err),
                                          _stream(kv_pool.device, stream))
    _lib.check(st, "pa_append_kv_fp8")


def pa_copy_blocks_fp8(src_dst_pairs, kv_pool, kv_format="e4m3", err=None, stream=None):
    """Copy-on-write copies of whole blocks of the 8-bit pool."""
    _need_cuda("src_dst_pairs", src_dst_pairs, torch.int32)
    NB, Hkv, B, d = _need_pool8(kv_pool)
    shape = _lib.PaShape(0, 1, Hkv, d, B, NB, 1, KV_FORMATS[kv_format])
    with torch.cuda.device(kv_pool.device):
        st = _lib.load().pa_copy_blocks_fp8(ctypes.byref(shape), _ptr(src_dst_pairs),
                                            ctypes.c_int32(src_dst_pairs.shape[0]), _ptr(kv_pool), _ptr(err),
                                            _stream(kv_pool.device, stream))
    _lib.check(st, "pa_copy_blocks_fp8")


# --------------------------------------------------------------------------- 4-bit cache
def int4_pool(num_blocks, num_kv_heads, block_size, head_dim=128, device="cuda"):
    """A zeroed 4-bit pool.  Its tensor shape [NB, Hkv, B, d + 8] only sizes
    the bytes of each (block, head) piece (B * d code nibbles + 8 * B scale
    bytes); the piece layout itself is the one include/pa.h describes."""
    return torch.zeros((num_blocks, num_kv_heads, block_size, head_dim + 8), dtype=torch.uint8, device=device)


def _need_pool4(kv_pool):
    _need_cuda("kv_pool", kv_pool, torch.uint8)
    if kv_pool.dim() != 4:
        raise ValueError("kv_pool must be uint8 [NB, Hkv, B, d + 8] (see int4_pool)")
    return kv_pool.shape[0], kv_pool.shape[1], kv_pool.shape[2], kv_pool.shape[3] - 8


def pa_decode_int4(q, kv_pool, block_tables, context_lens, scale, out=None, workspace=None, err=None,
                   stream=None):
    """Decode over the 4-bit cache (see include/pa.h)."""
    _need_cuda("q", q)
    _need_cuda("block_tables", block_tables, torch.int32)
    _need_cuda("context_lens", context_lens, torch.int32)
    NB, Hkv, B, d = _need_pool4(kv_pool)
    N, Hq, dq = q.shape
    if dq != d or block_tables.shape[0] != N:
        raise ValueError("q [N, Hq, d] and kv_pool [NB, Hkv, B, d + 8] disagree")
    out = torch.empty_like(q) if out is None else out
    shape = make_shape(N, Hq, Hkv, d, B, NB, block_tables.shape[1], q.dtype)
    lib = _lib.load()
    with torch.cuda.device(q.device):
        need = 0 if workspace is not None else int(lib.pa_decode_int4_workspace_bytes(ctypes.byref(shape)))
        s = _stream(q.device, stream)
        st = _lend(workspace, q.device.index, s.value or 0, max(need, 1),
                   lambda ws: lib.pa_decode_int4(ctypes.byref(shape), _ptr(q), _ptr(kv_pool), _ptr(block_tables),
                                                 _ptr(context_lens), ctypes.c_float(scale), _ptr(out), _ptr(ws),
                                                 ctypes.c_size_t(ws.numel() * ws.element_size()), _ptr(err), s), stream)
    _lib.check(st, "pa_decode_int4")
    return out


def pa_append_kv_int4(k_new, v_new, slot_mapping, kv_pool, err=None, stream=None):
    """Quantize k_new / v_new [T, Hkv, d] (fp16/bf16) into the 4-bit pool."""
    _need_cuda("k_new", k_new)
    _need_cuda("v_new", v_new, k_new.dtype)
    _need_cuda("slot_mapping", slot_mapping, torch.int64)
    NB, Hkv, B, d = _need_pool4(kv_pool)
    T = slot_mapping.shape[0]
    shape = make_shape(0, 1, Hkv, d, B, NB, 1, k_new.dtype)
    with torch.cuda.device(kv_pool.device):
        st = _lib.load().pa_append_kv_int4(ctypes.byref(shape), ctypes.c_int32(T), _ptr(k_new), _ptr(v_new),
                                           _ptr(slot_mapping), _ptr(kv_pool), _ptr(err),
                                           _stream(kv_pool.device, stream))
    _lib.check(st, "pa_append_kv_int4")


def pa_copy_blocks_int4(src_dst_pairs, kv_pool, dtype=torch.bfloat16, err=None, stream=None):
    """Copy-on-write copies of whole blocks of the 4-bit pool."""
    _need_cuda("src_dst_pairs", src_dst_pairs, torch.int32)
    NB, Hkv, B, d = _need_pool4(kv_pool)
    shape = make_shape(0, 1, Hkv, d, B, NB, 1, dtype)
    with torch.cuda.device(kv_pool.device):
        st = _lib.load().pa_copy_blocks_int4(ctypes.byref(shape), _ptr(src_dst_pairs),
                                             ctypes.c_int32(src_dst_pairs.shape[0]), _ptr(kv_pool), _ptr(err),
                                             _stream(kv_pool.device, stream))
    _lib.check(st, "pa_copy_blocks_int4")


# --------------------------------------------------------------------------- 8-bit cache, a scale per block and head
BS8_HEAD = 32


def bs8_pool(num_blocks, num_kv_heads, block_size, head_dim=128, device="cuda"):
    """An empty block-scaled 8-bit pool: zeros, uint8 [NB, Hkv, 32 + 2 * B * d]
    (two scales, then the codes of B keys and B values; see include/pa.h)."""
    return torch.zeros((num_blocks, num_kv_heads, BS8_HEAD + 2 * block_size * head_dim), dtype=torch.uint8,
                       device=device)


def bs8_scales(kv_pool):
    """The pool's scales as a view, fp32 [NB, Hkv, 2]: keys', values'."""
    return kv_pool[..., :8].view(torch.float32)


def _bs8_format(kv_format) -> int:
    if kv_format not in KV_FORMATS:
        raise ValueError(f"kv_format must be one of {sorted(KV_FORMATS)}, got {kv_format!r}")
    return KV_FORMATS[kv_format]


def _bound(n):
    # (no chunk reaches 2^31 tokens; ctypes would cut the number to its low 32 bits)
    return n if n is None else min(n, 2 ** 31 - 1)


def _bs8_shape(kv_pool, head_dim, dtype, dev) -> _lib.PaShape:
    """Shape of a pool of pieces for head_dim; the block size follows from their bytes."""
    if dtype not in _DTYPES:
        raise TypeError(f"queries and values must be float16 or bfloat16, got {dtype}")
    _arg("kv_pool", kv_pool, torch.uint8, dev)
    if kv_pool.dim() != 3 or head_dim < 1 or (kv_pool.shape[2] - BS8_HEAD) % (2 * head_dim):
        raise ValueError("kv_pool must be uint8 [NB, Hkv, 32 + 2 * B * d] (see bs8_pool)")
    NB, Hkv, P = kv_pool.shape
    return _lib.PaShape(0, Hkv, Hkv, head_dim, (P - BS8_HEAD) // (2 * head_dim), NB, 1, _DTYPES[dtype])


def pa_append_kv_bs8(k_new, v_new, block_tables, context_lens, q_start, kv_pool, kv_format="e4m3", max_new=None,
                     err=None, stream=None):
    """Quantise new tokens into the block-scaled pool (see include/pa.h): rows
    q_start[b] .. q_start[b + 1] - 1 of k_new and v_new [T, Hkv, d] are sequence
    b's last cached tokens, counted in context_lens.  k_new, v_new may be views
    of one projection's output.  max_new defaults to the largest number of new
    tokens (read from q_start on the host)."""
    if stream is not None:
        return _on_stream(stream, pa_append_kv_bs8, k_new, v_new, block_tables, context_lens, q_start, kv_pool,
                          kv_format, max_new, err)
    if max_new is None and isinstance(q_start, torch.Tensor):
        max_new = _largest_chunk(q_start)
    max_new = _bound(max_new)
    args = (k_new, v_new, block_tables, context_lens, q_start, kv_pool, _bs8_format(kv_format), max_new, err)
    if (_fast or _load_fast()).append_kv_bs8(*args) is NotImplemented:
        _append_kv_bs8(*args)


def _append_kv_bs8(k_new, v_new, block_tables, context_lens, q_start, kv_pool, fmt, max_new, err):
    """pa_append_kv_bs8 by way of every check."""
    dev = _index("kv_pool", kv_pool)
    if not isinstance(k_new, torch.Tensor) or k_new.dim() != 3:
        raise ValueError("k_new must be a tensor [T, Hkv, d]")
    T, Hkv, d = k_new.shape
    shape = _bs8_shape(kv_pool, d, k_new.dtype, dev)
    if shape.num_kv_heads != Hkv:
        raise ValueError(f"k_new has {Hkv} heads, kv_pool {shape.num_kv_heads}")
    ks = _token_rows("k_new", k_new, k_new.dtype, (T, Hkv, d), dev)
    vs = _token_rows("v_new", v_new, k_new.dtype, (T, Hkv, d), dev)
    _arg("block_tables", block_tables, torch.int32, dev)
    _arg("context_lens", context_lens, torch.int32, dev)
    _arg("q_start", q_start, torch.int32, dev)
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be [N, MB]")
    N, MB = block_tables.shape
    if q_start.shape != (N + 1,) or context_lens.shape != (N,):
        raise ValueError("q_start must have N + 1 entries, context_lens N")
    if err is not None:
        _arg("err", err, torch.int32, dev)
    shape.num_seqs, shape.max_blocks_per_seq = N, MB
    st = _call(_lib.load().pa_append_kv_bs8, dev, shape, fmt, max_new, T, k_new.data_ptr(), ks, v_new.data_ptr(), vs,
               q_start.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(), kv_pool.data_ptr(), _addr(err),
               _raw_stream(dev))
    if st:
        _lib.check(st, "pa_append_kv_bs8")


_bs8_bytes = {}


def _bs8_workspace_bytes(dev, shape, fmt, max_q):
    # (max_q 0: pa_decode_bs8) the size of a valid shape's workspace depends on these and the device's SM count alone
    key = (dev, fmt, max_q, shape.num_seqs, shape.num_q_heads, shape.num_kv_heads, shape.head_dim, shape.block_size,
           shape.dtype)
    need = _bs8_bytes.get(key)
    if need is None:
        lib = _lib.load()
        need = int(_call(lib.pa_decode_multi_bs8_workspace_bytes, dev, shape, fmt, max_q) if max_q else
                   _call(lib.pa_decode_bs8_workspace_bytes, dev, shape, fmt))
        if need:                         # 0: something about the shape is invalid, which the call reports
            _bs8_bytes[key] = need
    return need


def _bs8_attention(call, q, kv_pool, block_tables, context_lens, fmt, out, workspace, err, max_q, run):
    """The checks and the workspace that both attention calls share;
    run(lib, shape, out, ws, err, handle) makes the call."""
    dev = _index("q", q)
    dt = q.dtype
    _arg("q", q, dt, dev)
    if q.dim() != 3:
        raise ValueError("q must be [rows, Hq, d]")
    shape = _bs8_shape(kv_pool, q.shape[2], dt, dev)
    _arg("block_tables", block_tables, torch.int32, dev)
    _arg("context_lens", context_lens, torch.int32, dev)
    if block_tables.dim() != 2 or context_lens.shape != (block_tables.shape[0],):
        raise ValueError("block_tables must be [N, MB], context_lens [N]")
    if out is None:
        out = torch.empty_like(q)
    else:
        _arg("out", out, dt, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if err is not None:
        _arg("err", err, torch.int32, dev)
    shape.num_q_heads = q.shape[1]
    shape.num_seqs, shape.max_blocks_per_seq = block_tables.shape
    need = 0
    if workspace is not None:
        _arg("workspace", workspace, workspace.dtype, dev)
    else:
        need = _bs8_workspace_bytes(dev, shape, fmt, max_q)
        if need == 0:
            workspace = torch.empty(0, dtype=torch.uint8, device=q.device)
    handle = _raw_stream(dev)
    st = _lend(workspace, dev, handle, need, lambda ws: run(_lib.load(), dev, shape, out, ws, handle))
    if st:
        _lib.check(st, call)
    return out


def pa_decode_bs8(q, kv_pool, block_tables, context_lens, scale, kv_format="e4m3", out=None, workspace=None, err=None,
                  stream=None):
    """Decode over the block-scaled 8-bit cache (see include/pa.h): out [N, Hq, d]
    in q's type, for q [N, Hq, d]."""
    if stream is not None:
        return _on_stream(stream, pa_decode_bs8, q, kv_pool, block_tables, context_lens, scale, kv_format, out,
                          workspace, err)
    args = (q, kv_pool, block_tables, context_lens, scale, _bs8_format(kv_format), out, workspace, err)
    done = (_fast or _load_fast()).decode_bs8(_sp_cache, *args)
    return _decode_bs8(*args) if done is NotImplemented else done


def _decode_bs8(q, kv_pool, block_tables, context_lens, scale, fmt, out, workspace, err):
    """pa_decode_bs8 by way of every check."""
    def run(lib, dev, shape, out, ws, handle):
        if q.shape[0] != shape.num_seqs:
            raise ValueError("q and block_tables must have N rows")
        return _call(lib.pa_decode_bs8, dev, shape, fmt, q.data_ptr(), kv_pool.data_ptr(), block_tables.data_ptr(),
                     context_lens.data_ptr(), scale, out.data_ptr(), ws.data_ptr(), ws.nbytes, _addr(err), handle)
    return _bs8_attention("pa_decode_bs8", q, kv_pool, block_tables, context_lens, fmt, out, workspace, err, 0, run)


def pa_decode_multi_bs8(q, kv_pool, block_tables, context_lens, q_start, scale, kv_format="e4m3", max_q_len=None,
                        out=None, workspace=None, err=None, stream=None):
    """Causal attention of a chunk of new tokens per sequence over the
    block-scaled 8-bit cache (see include/pa.h): q [T, Hq, d] holds each
    sequence's last cached tokens at rows q_start[b] .. q_start[b + 1] - 1
    (q_start: int32 [N + 1]), few or thousands.  max_q_len defaults to the
    largest chunk (read from q_start on the host)."""
    if stream is not None:
        return _on_stream(stream, pa_decode_multi_bs8, q, kv_pool, block_tables, context_lens, q_start, scale,
                          kv_format, max_q_len, out, workspace, err)
    if max_q_len is None and isinstance(q_start, torch.Tensor):
        max_q_len = _largest_chunk(q_start)
    max_q_len = _bound(max_q_len)
    args = (q, kv_pool, block_tables, context_lens, q_start, scale, _bs8_format(kv_format), max_q_len, out, workspace,
            err)
    done = (_fast or _load_fast()).decode_multi_bs8(_sp_cache, *args)
    return _decode_multi_bs8(*args) if done is NotImplemented else done


def _decode_multi_bs8(q, kv_pool, block_tables, context_lens, q_start, scale, fmt, max_q_len, out, workspace, err):
    """pa_decode_multi_bs8 by way of every check."""
    _arg("q_start", q_start, torch.int32, _index("q", q))
    if max_q_len < 1:
        raise ValueError("max_q_len must be at least 1")

    def run(lib, dev, shape, out, ws, handle):
        if q_start.shape != (shape.num_seqs + 1,):
            raise ValueError("q_start must have N + 1 entries")
        return _call(lib.pa_decode_multi_bs8, dev, shape, fmt, max_q_len, q.shape[0], q.data_ptr(), q_start.data_ptr(),
                     kv_pool.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(), scale, out.data_ptr(),
                     ws.data_ptr(), ws.nbytes, _addr(err), handle)
    return _bs8_attention("pa_decode_multi_bs8", q, kv_pool, block_tables, context_lens, fmt, out, workspace, err,
                          max_q_len, run)


def pa_copy_blocks_bs8(src_dst_pairs, kv_pool, err=None, stream=None):
    """Copy-on-write copies of whole blocks, scales included, of the
    block-scaled pool."""
    if stream is not None:
        return _on_stream(stream, pa_copy_blocks_bs8, src_dst_pairs, kv_pool, err)
    dev = _index("kv_pool", kv_pool)
    n = kv_pool.shape[-1] - BS8_HEAD
    # blocks of 16 or 32 tokens: the bytes are the same for either, and for either head_dim
    d = n // 32 if n // 32 in (64, 128) else n // 64
    shape = _bs8_shape(kv_pool, max(d, 1), torch.bfloat16, dev)
    _arg("src_dst_pairs", src_dst_pairs, torch.int32, dev)
    if src_dst_pairs.dim() != 2 or src_dst_pairs.shape[1] != 2:
        raise ValueError("src_dst_pairs must be [n, 2]")
    if err is not None:
        _arg("err", err, torch.int32, dev)
    st = _call(_lib.load().pa_copy_blocks_bs8, dev, shape, src_dst_pairs.data_ptr(), src_dst_pairs.shape[0],
               kv_pool.data_ptr(), _addr(err), _raw_stream(dev))
    if st:
        _lib.check(st, "pa_copy_blocks_bs8")


def _convert_bs8(call, src_dst_pairs, k_pool, v_pool, kv_pool, fmt, err):
    """pa_pack_blocks_bs8 and pa_unpack_blocks_bs8 by way of every check."""
    dev = _index("kv_pool", kv_pool)
    if not isinstance(k_pool, torch.Tensor) or k_pool.dim() != 4:
        raise ValueError("k_pool must be a tensor [NB, Hkv, B, d]")
    _arg("k_pool", k_pool, k_pool.dtype, dev)
    _arg("v_pool", v_pool, k_pool.dtype, dev)
    NB, Hkv, B, d = k_pool.shape
    shape = _bs8_shape(kv_pool, d, k_pool.dtype, dev)
    if v_pool.shape != k_pool.shape or (shape.num_kv_heads, shape.block_size) != (Hkv, B):
        raise ValueError("k_pool, v_pool [NB, Hkv, B, d] and kv_pool [NB, Hkv, 32 + 2 * B * d] disagree")
    _arg("src_dst_pairs", src_dst_pairs, torch.int32, dev)
    if src_dst_pairs.dim() != 2 or src_dst_pairs.shape[1] != 2:
        raise ValueError("src_dst_pairs must be [n, 2]")
    if err is not None:
        _arg("err", err, torch.int32, dev)
    pools = (k_pool, v_pool, kv_pool) if call == "pa_pack_blocks_bs8" else (kv_pool, k_pool, v_pool)
    st = _call(getattr(_lib.load(), call), dev, shape, fmt, NB, src_dst_pairs.data_ptr(), src_dst_pairs.shape[0],
               *(p.data_ptr() for p in pools), _addr(err), _raw_stream(dev))
    if st:
        _lib.check(st, call)


def pa_pack_blocks_bs8(src_dst_pairs, k_pool, v_pool, kv_pool, kv_format="e4m3", err=None, stream=None):
    """Quantise whole blocks src of a 16-bit cache (k_pool, v_pool [NB, Hkv, B, d])
    into blocks dst of the block-scaled pool, for each row of src_dst_pairs [n, 2]
    (int32)."""
    if stream is not None:
        return _on_stream(stream, pa_pack_blocks_bs8, src_dst_pairs, k_pool, v_pool, kv_pool, kv_format, err)
    args = (src_dst_pairs, k_pool, v_pool, kv_pool, _bs8_format(kv_format), err)
    if (_fast or _load_fast()).pack_blocks_bs8(*args) is NotImplemented:
        _convert_bs8("pa_pack_blocks_bs8", *args)


def pa_unpack_blocks_bs8(src_dst_pairs, kv_pool, k_pool, v_pool, kv_format="e4m3", err=None, stream=None):
    """Blocks src of the block-scaled pool back into blocks dst of a 16-bit cache,
    for each row of src_dst_pairs [n, 2] (int32)."""
    if stream is not None:
        return _on_stream(stream, pa_unpack_blocks_bs8, src_dst_pairs, kv_pool, k_pool, v_pool, kv_format, err)
    args = (src_dst_pairs, kv_pool, k_pool, v_pool, _bs8_format(kv_format), err)
    if (_fast or _load_fast()).unpack_blocks_bs8(*args) is NotImplemented:
        _convert_bs8("pa_unpack_blocks_bs8", src_dst_pairs, k_pool, v_pool, kv_pool, *args[-2:])
