"""Python binding of librkv.so (rolling-window chunk attention for B200).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels. Tensors are torch CUDA tensors (bf16, contiguous); PyTorch provides
device memory and streams. The C ABI is declared in include/rkv.h; the names
here are the C names without the ``rkv_`` prefix.

The library must be built (``python rolling_kv_chunked_b200/build.py``); if it
is missing, importing this package raises.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librkv.so")

OK = 0
ERR_ARG = 1
ERR_ORDER = 2
ERR_CAPACITY = 3
ERR_UNSUPPORTED = 4
ERR_CUDA = 5
ERR_TIMEOUT = 6
ERR_STATE = 7
ERR_PAGE = 8

ROPE_ABSOLUTE = 0
ROPE_RELATIVE = 1
ROPE_RELATIVE_SLOTS = 2

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run `python rolling_kv_chunked_b200/build.py`")

_lib = ctypes.CDLL(LIB_PATH)

_c_int, _c_ll, _c_dbl, _vp = ctypes.c_int, ctypes.c_longlong, ctypes.c_double, ctypes.c_void_p
_int_p = ctypes.POINTER(ctypes.c_int)


class FlowEpilogue(ctypes.Structure):
    """Mirror of ``rkv_flow_epilogue``."""
    _fields_ = [("xt", _vp), ("eps", _vp), ("sigma", _c_dbl), ("sigma_next", _c_dbl),
                ("x0_out", _vp), ("xt_next_out", _vp)]


class HeadCopy(ctypes.Structure):
    """Mirror of ``rkv_head_copy``: n_tok tokens x n_heads head vectors, strides in elements."""
    _fields_ = [("src", _vp), ("dst", _vp), ("src_tok_stride", _c_ll), ("src_head_stride", _c_ll),
                ("dst_tok_stride", _c_ll), ("dst_head_stride", _c_ll), ("n_tok", _c_int)]


class _PagePool(ctypes.Structure):
    """Mirror of ``rkv_page_pool``."""
    _fields_ = [("k", _vp), ("v", _vp), ("page_stride", _c_ll), ("n_pages", _c_int), ("kv_heads", _c_int),
                ("page_tokens", _c_int)]


class _PagedBatch(ctypes.Structure):
    """Mirror of ``rkv_paged_batch``."""
    _fields_ = [("page_table", _vp), ("kv_len", _vp), ("q_start", _vp), ("status", _vp), ("table_stride", _c_int),
                ("n_seqs", _c_int), ("max_q", _c_int), ("max_kv", _c_int)]


_pool_p, _batch_p = ctypes.POINTER(_PagePool), ctypes.POINTER(_PagedBatch)

_SIGS = {
    "rkv_create": ([_c_int] * 7 + [ctypes.POINTER(_vp)], _c_int),
    "rkv_set_rope_grid": ([_vp, _c_int, _c_int, _c_dbl, _c_int, _c_int, _c_int], _c_int),
    "rkv_write_chunk": ([_vp, _c_int, _vp, _vp, _c_int, _c_int, _vp], _c_int),
    "rkv_chunk_attention": ([_vp, _c_int, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _vp], _c_int),
    "rkv_chunk_attention_flow": ([_vp, _c_int, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int,
                                  ctypes.POINTER(FlowEpilogue), _vp], _c_int),
    "rkv_chunk_attention_cfg_flow": ([_vp, _c_int, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int,
                                      ctypes.POINTER(FlowEpilogue), _vp, _c_dbl, _vp], _c_int),
    "rkv_set_text_kv": ([_vp, _c_int, _vp, _vp, _c_int, _vp], _c_int),
    "rkv_cross_attention": ([_vp, _c_int, _vp, _vp, _c_int, _vp], _c_int),
    "rkv_rope_apply": ([_vp, _vp, _c_int, _c_int, _c_int, _vp], _c_int),
    "rkv_flow_x0_renoise": ([_vp, _vp, _vp, _c_dbl, _c_dbl, _vp, _vp, _c_ll, _vp], _c_int),
    "rkv_flow_cfg_x0_renoise": ([_vp, _vp, _vp, _vp, _c_dbl, _c_dbl, _c_dbl, _vp, _vp, _c_ll, _vp], _c_int),
    "rkv_slot_frames": ([_vp, _c_int, _int_p], _c_int),
    "rkv_frames_committed": ([_vp, _c_int, _int_p], _c_int),
    "rkv_cache_ptrs": ([_vp, _c_int, ctypes.POINTER(_vp), ctypes.POINTER(_vp)], _c_int),
    "rkv_reset": ([_vp], _c_int),
    "rkv_destroy": ([_vp], _c_int),
    "rkv_status_string": ([_c_int], ctypes.c_char_p),
    "rkv_poll_device_status": ([_vp, _vp], _c_int),
    "rkv_set_wait_limit": ([_vp, _c_ll], _c_int),
    "rkv_chunk_attention_noalloc": ([_vp, _vp, _vp, _vp] + [_c_int] * 8 + [_int_p, _c_int, _vp], _c_int),
    "rkv_timing_begin": ([_vp, _c_int], _c_int),
    "rkv_timing_end": ([_vp, ctypes.POINTER(ctypes.c_float), _c_int, _int_p], _c_int),
    "rkv_plan_window": ([_c_int, _c_int, _c_int, _c_int, _c_int, _int_p, _c_int, _int_p], _c_int),
    "rkv_copy_heads": ([ctypes.POINTER(HeadCopy), _c_int, _c_int, _vp], _c_int),
    "rkv_paged_write": ([_pool_p, _batch_p, _vp, _vp, _c_int, _c_ll, _c_ll, _vp], _c_int),
    "rkv_paged_attention": ([_pool_p, _batch_p, _vp, _c_int, _c_int, _c_ll, _vp, _c_ll, _c_int, _vp, _vp, _c_ll,
                             _vp, _c_ll, _vp], _c_int),
    "rkv_paged_workspace": ([_pool_p, _batch_p, _c_int, _c_int, _c_int, ctypes.POINTER(_c_ll)], _c_int),
    "rkv_paged_evict": ([_pool_p, _batch_p, _vp, _c_ll, _c_int, _c_int, _c_int, _vp, _vp, _vp], _c_int),
    "rkv_paged_poll_status": ([_vp, _vp], _c_int),
}
for _name, (_args, _res) in _SIGS.items():
    try:
        _fn = getattr(_lib, _name)
    except AttributeError as _e:
        raise ImportError(f"{LIB_PATH} does not export {_name}; rebuild it") from _e
    _fn.argtypes = _args
    _fn.restype = _res

EXPORTED = tuple(_SIGS)


class RkvError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} (code {code})")


def status_string(code: int) -> str:
    return _lib.rkv_status_string(code).decode()


def _check(code: int, where: str) -> None:
    if code != OK:
        raise RkvError(code, where)


def _ptr(t):
    """Device pointer of a torch tensor (or an int / None)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def plan_window(window_frames: int, sink_frames: int, frames_committed: int, n_frames: int, start_frame: int):
    """Host-only: the key segments chunk [start_frame, start_frame+n_frames) attends to."""
    buf = (ctypes.c_int * 16)()
    n = ctypes.c_int(0)
    _check(_lib.rkv_plan_window(window_frames, sink_frames, frames_committed, n_frames, start_frame,
                                buf, 4, ctypes.byref(n)), "rkv_plan_window")
    return [tuple(buf[4 * i:4 * i + 4]) for i in range(n.value)]


def flow_x0_renoise(xt, v, eps, sigma: float, sigma_next: float, x0_out, xt_next_out=None, stream=None) -> None:
    """x0 = xt - sigma v; xt_next = (1 - sigma') x0 + sigma' eps (sigma' < 0: last step)."""
    _check(_lib.rkv_flow_x0_renoise(_ptr(xt), _ptr(v), _ptr(eps), float(sigma), float(sigma_next),
                                    _ptr(x0_out), _ptr(xt_next_out), xt.numel(), _stream(stream)),
           "rkv_flow_x0_renoise")


def copy_heads(runs, n_heads: int, stream=None) -> None:
    """Strided head-vector copies. ``runs``: (src_ptr, dst_ptr, src_tok_stride, src_head_stride,
    dst_tok_stride, dst_head_stride, n_tok) tuples, pointers as ints, strides in elements."""
    arr = (HeadCopy * max(1, len(runs)))()
    for i, r in enumerate(runs):
        arr[i] = HeadCopy(*r)
    _check(_lib.rkv_copy_heads(arr, len(runs), int(n_heads), _stream(stream)), "rkv_copy_heads")


def flow_cfg_x0_renoise(xt, v_cond, v_uncond, eps, cfg_scale: float, sigma: float, sigma_next: float, x0_out,
                        xt_next_out=None, stream=None) -> None:
    """v = v_uncond + cfg_scale (v_cond - v_uncond), then the x0 / renoise step of flow_x0_renoise."""
    _check(_lib.rkv_flow_cfg_x0_renoise(_ptr(xt), _ptr(v_cond), _ptr(v_uncond), _ptr(eps), float(cfg_scale),
                                        float(sigma), float(sigma_next), _ptr(x0_out), _ptr(xt_next_out),
                                        xt.numel(), _stream(stream)), "rkv_flow_cfg_x0_renoise")


# ---------------------------------------------------------------------- paged caches
def _torch():
    import torch
    return torch


def _refuse(where: str):
    raise RkvError(ERR_ARG, where)


def _int32(x, where: str) -> int:
    """x as the library takes it; refused where a C int would keep the low 32 bits."""
    if not -(1 << 31) <= x < 1 << 31:
        _refuse(where)
    return x


def _dense(t, dtype, shape, index, where: str):
    """Pointer of a contiguous tensor of this type and shape (None: any extent) on GPU ``index``; refused otherwise."""
    if t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        _refuse(where)
    have = t.shape
    if have != shape and (len(have) != len(shape) or any(w is not None and n != w for n, w in zip(have, shape))):
        _refuse(where)
    return t.data_ptr()


def _rows(t, heads, rows, pool, where: str):
    """(pointer, rows, heads, row stride) of a [rows, heads, 128] bf16 tensor whose rows may lie apart."""
    if t.dtype is not pool.bf16 or t.dim() != 3 or t.get_device() != pool.index:
        _refuse(where)
    n, h, d = t.shape
    row, head, one = t.stride()
    if (d != 128 or one != 1 or (head != 128 and h != 1) or (heads is not None and h != heads)
            or (rows is not None and n != rows)):
        _refuse(where)
    return t.data_ptr(), n, h, row if n > 1 else h * 128


def _pair(pool, batch, where: str) -> None:
    """Pool and batch fit: the same GPU, and page lists whose columns reach max_kv. (The library sees the lists' stride
    only, and a column slice's stride counts columns that are not its own.)"""
    if pool.index != batch.index or batch.width * pool.page_tokens < batch.max_kv:
        _refuse(where)


def _launch(fn, where: str, pool, stream, *args) -> None:
    """Call with the tensors' device current and, unless a stream is given, on its current stream."""
    torch, index = pool.torch, pool.index
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if torch._C._cuda_getDevice() == index:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, stream)
    if rc != OK:
        _check(rc, where)


class PagePool:
    """One layer's pages: k and v, each [n_pages, kv_heads, page_tokens, 128] bf16, contiguous but for
    the distance between pages, which is the same in both (two halves of one tensor will do)."""

    def __init__(self, k, v):
        where = "PagePool"
        torch = _torch()
        if (k.dtype is not torch.bfloat16 or v.dtype is not torch.bfloat16 or not k.is_cuda or k.device != v.device
                or k.dim() != 4 or k.shape != v.shape or k.shape[3] != 128):
            _refuse(where)
        n, h, p, _ = k.shape
        for t in (k, v):
            if t.stride(3) != 1 or (p > 1 and t.stride(2) != 128) or (h > 1 and t.stride(1) != p * 128):
                _refuse(where)
        if n > 1 and k.stride(0) != v.stride(0):
            _refuse(where)
        self.k, self.v, self.device, self.kv_heads, self.page_tokens = k, v, k.device, h, p
        self.torch, self.index, self.bf16 = torch, k.device.index, torch.bfloat16
        self._c = _PagePool(k.data_ptr(), v.data_ptr(), k.stride(0) if n > 1 else h * p * 128, n, h, p)
        self._ref = ctypes.byref(self._c)


class PagedBatch:
    """The streams of one step: page_table [n_seqs, pages] int32, kv_len [n_seqs] int32, q_start
    [n_seqs + 1] int32 (None for eviction only), all on the GPU, and host bounds of chunk rows and
    cached tokens per stream (page_table has columns for max_kv tokens). ``status``: one zeroed int32
    on the GPU that collects errors (``poll``); without it they are not reported. Layers can share one."""

    def __init__(self, page_table, kv_len, q_start, max_q: int, max_kv: int, status=None):
        where = "PagedBatch"
        i32 = _torch().int32
        if page_table.dtype is not i32 or not page_table.is_cuda or page_table.dim() != 2:
            _refuse(where)
        n, width = page_table.shape
        dev = page_table.device
        stride = page_table.stride(0) if n > 1 else width
        if (width > 1 and page_table.stride(1) != 1) or stride < width:
            _refuse(where)
        for t, shape in ((kv_len, (n,)), (q_start, (n + 1,)), (status, (1,))):
            if t is not None:
                _dense(t, i32, shape, dev.index, where)
        self.page_table, self.kv_len, self.q_start, self.status = page_table, kv_len, q_start, status
        self.device, self.index, self.n_seqs, self.width, self.max_kv = dev, dev.index, n, width, max_kv
        self._c = _PagedBatch(_ptr(page_table), _ptr(kv_len), _ptr(q_start), _ptr(status),
                              _int32(stride, where), n, _int32(max_q, where), _int32(max_kv, where))
        self._ref = ctypes.byref(self._c)

    def poll(self, stream=None) -> int:
        """Synchronise the stream and return (and clear) the status: OK, ERR_PAGE or ERR_TIMEOUT."""
        if self.status is None:
            _refuse("rkv_paged_poll_status")
        with _torch().cuda.device(self.device):
            return _lib.rkv_paged_poll_status(_ptr(self.status), _stream(stream))


def paged_write(pool: PagePool, batch: PagedBatch, k, v, stream=None) -> None:
    """The chunk's K and V, [rows, kv_heads, 128] bf16, into the pages."""
    where = "rkv_paged_write"
    _pair(pool, batch, where)
    kp, rows, _, ks = _rows(k, pool.kv_heads, None, pool, where)
    vp, _, _, vs = _rows(v, pool.kv_heads, rows, pool, where)
    _launch(_lib.rkv_paged_write, where, pool, stream, pool._ref, batch._ref, kp, vp, rows, ks, vs)


def paged_workspace_bytes(pool: PagePool, batch: PagedBatch, rows: int, q_heads: int, weight: bool = False) -> int:
    """Bytes of workspace that ``paged_attention`` needs for a chunk tensor of ``rows`` rows."""
    where = "rkv_paged_workspace"
    _pair(pool, batch, where)
    n = _c_ll(0)
    _check(_lib.rkv_paged_workspace(pool._ref, batch._ref, _int32(q_heads, where), _int32(rows, where),
                                    int(bool(weight)), ctypes.byref(n)), where)
    return n.value


def paged_attention(pool: PagePool, batch: PagedBatch, q, out, causal: bool = True, lse=None, weight=None,
                    workspace=None, stream=None) -> None:
    """out = softmax(q K^T / sqrt(128)) V over each stream's pages; q, out [rows, q_heads, 128] bf16, lse
    [rows, q_heads] fp32 (optional), weight [n_seqs, kv_heads, tokens] fp32 (optional): the attention weight
    of every key, added up. ``workspace``: a uint8 tensor of ``paged_workspace_bytes`` (allocated on the
    call's stream if None)."""
    where = "rkv_paged_attention"
    index, torch = pool.index, pool.torch
    _pair(pool, batch, where)
    qp, rows, heads, qs = _rows(q, None, None, pool, where)
    op, _, _, os_ = _rows(out, heads, rows, pool, where)
    zp = wp = None
    width = 0
    if lse is not None:
        zp = _dense(lse, torch.float32, (rows, heads), index, where)
    if weight is not None:
        wp = _dense(weight, torch.float32, (batch.n_seqs, pool.kv_heads, None), index, where)
        width = weight.shape[2]
        if width < batch.max_kv:
            _refuse(where)  # here too: a tensor without elements has no address to refuse
    if workspace is None:
        size = paged_workspace_bytes(pool, batch, rows, heads, weight is not None)
        if stream is None:
            stream = torch.cuda.current_stream(index)
        elif isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, pool.device) if stream else torch.cuda.default_stream(index)
        with torch.cuda.stream(stream):
            workspace = torch.empty(size, dtype=torch.uint8, device=pool.device)
    sp = _dense(workspace, torch.uint8, (None,), index, where)
    _launch(_lib.rkv_paged_attention, where, pool, stream, pool._ref, batch._ref, qp, heads, rows, qs, op, os_,
            1 if causal else 0, zp, wp, width, sp, workspace.shape[0])


def paged_evict(pool: PagePool, batch: PagedBatch, weight, keep: int, sinks: int, recent: int, kept, kv_len_out,
                stream=None) -> None:
    """Trim every (stream, KV head) to its first ``sinks``, last ``recent`` and heaviest other tokens, ``keep``
    in all, in their order. weight [n_seqs, kv_heads, tokens] fp32, kept [n_seqs, kv_heads, keep] int32 and
    kv_len_out [n_seqs] int32 (both written)."""
    where = "rkv_paged_evict"
    index, n, torch = pool.index, batch.n_seqs, pool.torch
    _pair(pool, batch, where)
    wp = _dense(weight, torch.float32, (n, pool.kv_heads, None), index, where)
    kp = _dense(kept, torch.int32, (n, pool.kv_heads, keep), index, where)
    lp = _dense(kv_len_out, torch.int32, (n,), index, where)
    _launch(_lib.rkv_paged_evict, where, pool, stream, pool._ref, batch._ref, wp, weight.shape[2],
            _int32(keep, where), _int32(sinks, where), _int32(recent, where), kp, lp)


class RollingKV:
    """One rkv handle: per-layer rolling caches plus the RoPE configuration."""

    def __init__(self, layers: int, H: int, d: int, tokens_per_frame: int, window_frames: int,
                 sink_frames: int, rope_mode: int):
        h = _vp()
        _check(_lib.rkv_create(layers, H, d, tokens_per_frame, window_frames, sink_frames, rope_mode,
                               ctypes.byref(h)), "rkv_create")
        self._h = h
        self.layers, self.H, self.d, self.T = layers, H, d, tokens_per_frame
        self.window_frames, self.sink_frames, self.rope_mode = window_frames, sink_frames, rope_mode

    # ------------------------------------------------------------------ config
    def set_rope_grid(self, grid_h: int, grid_w: int, theta: float = 1.0e4, pairs=(22, 21, 21)) -> None:
        _check(_lib.rkv_set_rope_grid(self._h, grid_h, grid_w, float(theta), *pairs), "rkv_set_rope_grid")

    def set_wait_limit(self, nanoseconds: int) -> None:
        _check(_lib.rkv_set_wait_limit(self._h, int(nanoseconds)), "rkv_set_wait_limit")

    # ------------------------------------------------------------------ hot path
    def write_chunk(self, layer: int, k, v, n_frames: int, start_frame: int, stream=None) -> None:
        _check(_lib.rkv_write_chunk(self._h, layer, _ptr(k), _ptr(v), n_frames, start_frame, _stream(stream)),
               "rkv_write_chunk")

    def chunk_attention(self, layer: int, q, k, v, out, n_frames: int, start_frame: int, commit: bool,
                        stream=None, flow: dict | None = None) -> None:
        """out = attention of the chunk's queries; ``flow`` = dict(xt, eps, sigma, sigma_next, x0_out,
        xt_next_out) fuses the x0/renoise epilogue into the output store. With ``v_cond`` and
        ``cfg_scale`` in ``flow`` this call is the unconditional branch of a guided step: the epilogue
        uses v = out + cfg_scale (v_cond - out)."""
        if flow is None:
            rc = _lib.rkv_chunk_attention(self._h, layer, _ptr(q), _ptr(k), _ptr(v), _ptr(out), n_frames,
                                          start_frame, int(bool(commit)), _stream(stream))
            _check(rc, "rkv_chunk_attention")
            return
        epi = FlowEpilogue(_ptr(flow["xt"]), _ptr(flow.get("eps")), float(flow["sigma"]),
                           float(flow["sigma_next"]), _ptr(flow["x0_out"]), _ptr(flow.get("xt_next_out")))
        if flow.get("v_cond") is not None:
            rc = _lib.rkv_chunk_attention_cfg_flow(self._h, layer, _ptr(q), _ptr(k), _ptr(v), _ptr(out), n_frames,
                                                   start_frame, int(bool(commit)), ctypes.byref(epi),
                                                   _ptr(flow["v_cond"]), float(flow["cfg_scale"]), _stream(stream))
            _check(rc, "rkv_chunk_attention_cfg_flow")
            return
        rc = _lib.rkv_chunk_attention_flow(self._h, layer, _ptr(q), _ptr(k), _ptr(v), _ptr(out), n_frames,
                                           start_frame, int(bool(commit)), ctypes.byref(epi), _stream(stream))
        _check(rc, "rkv_chunk_attention_flow")

    def set_text_kv(self, layer: int, k_text, v_text, stream=None) -> None:
        """Cache the text context's K and V ([n_text, H, d] each) for cross-attention."""
        _check(_lib.rkv_set_text_kv(self._h, layer, _ptr(k_text), _ptr(v_text), k_text.shape[0], _stream(stream)),
               "rkv_set_text_kv")

    def cross_attention(self, layer: int, q, out, stream=None) -> None:
        """out = softmax(q K_text^T / sqrt(d)) V_text over the cached text tokens; q, out [n, H, d]."""
        _check(_lib.rkv_cross_attention(self._h, layer, _ptr(q), _ptr(out), q.shape[0], _stream(stream)),
               "rkv_cross_attention")

    def rope_apply(self, x, n_frames: int, start_frame: int, window_end_frame: int = 0, stream=None) -> None:
        _check(_lib.rkv_rope_apply(self._h, _ptr(x), n_frames, start_frame, window_end_frame, _stream(stream)),
               "rkv_rope_apply")

    # ------------------------------------------------------------------ state
    def slot_frames(self, layer: int):
        buf = (ctypes.c_int * self.window_frames)()
        _check(_lib.rkv_slot_frames(self._h, layer, buf), "rkv_slot_frames")
        return list(buf)

    def frames_committed(self, layer: int) -> int:
        n = ctypes.c_int(0)
        _check(_lib.rkv_frames_committed(self._h, layer, ctypes.byref(n)), "rkv_frames_committed")
        return n.value

    def cache_ptrs(self, layer: int):
        k, v = _vp(), _vp()
        _check(_lib.rkv_cache_ptrs(self._h, layer, ctypes.byref(k), ctypes.byref(v)), "rkv_cache_ptrs")
        return k.value, v.value

    def timing_begin(self, max_launches: int) -> None:
        """Record CUDA events around each attention kernel launch (instrumentation only)."""
        _check(_lib.rkv_timing_begin(self._h, int(max_launches)), "rkv_timing_begin")

    def timing_end(self, max_launches: int = 4096):
        """Synchronise and return the recorded attention launch durations in ms."""
        buf = (ctypes.c_float * max_launches)()
        n = ctypes.c_int(0)
        _check(_lib.rkv_timing_end(self._h, buf, max_launches, ctypes.byref(n)), "rkv_timing_end")
        return list(buf[:n.value])

    def poll_device_status(self, stream=None) -> int:
        """Synchronise the stream and return (and clear) the device status: OK or ERR_TIMEOUT."""
        return _lib.rkv_poll_device_status(self._h, _stream(stream))

    def reset(self) -> None:
        _check(_lib.rkv_reset(self._h), "rkv_reset")

    def close(self) -> None:
        if getattr(self, "_h", None):
            _lib.rkv_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
