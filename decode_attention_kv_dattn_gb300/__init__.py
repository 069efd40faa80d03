"""Python binding of the dattn C ABI (include/dattn.h).

Argument marshalling only: tensors are passed to the library as raw device
pointers (torch is used for device memory and streams), and every step of the
computation runs in the library's CUDA kernels. There is no CPU fallback:
importing this package fails if libdattn.so has not been built (run
`python -c "import __graft_entry__ as g; g.build()"` or
`python decode_attention_kv_dattn_gb300/build.py`).
"""
import ctypes
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libdattn.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"dattn CUDA library not built: {LIB_PATH} is missing "
                      "(build it with decode_attention_kv_dattn_gb300/build.py)")

lib = ctypes.CDLL(LIB_PATH)

# ---------------------------------------------------------------- C types

OK, EINVAL, EXCEEDS, ECUDA, EINDEX, ETIMEOUT, EUNSUPPORTED, ELENGTH, ERANGE = range(9)
CACHE_RING, CACHE_PAGED, CACHE_STATE = 0, 1, 2
KV_BF16, KV_E4M3 = 0, 1
_I32, _BF16 = torch.int32, torch.bfloat16

_vp = ctypes.c_void_p
_int = ctypes.c_int


class LayerConfig(ctypes.Structure):
    _fields_ = [("cache_kind", _int), ("ring_slots", _int), ("page_size", _int),
                ("rotary_dim", _int), ("rope_theta", ctypes.c_double),
                ("q_norm_weight", _vp), ("k_norm_weight", _vp), ("norm_eps", ctypes.c_double),
                ("kv_format", _int), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float),
                ("log_decay", _vp)]


def _host_f32(x, n, what):
    """A contiguous host array of n fp32 values (numpy, a CPU tensor or a list), or None."""
    if x is None:
        return None
    if isinstance(x, torch.Tensor) and x.is_cuda:
        raise TypeError(f"{what}: a host array")
    x = np.ascontiguousarray(x, dtype=np.float32)
    if x.shape != (n,):
        raise ValueError(f"{what}: shape {x.shape}, expected ({n},)")
    return x


def _host_bf16(w, D, what):
    """QK-norm weights as a contiguous host array of D bf16 bit patterns
    (numpy uint16, or a CPU bfloat16 tensor), or None."""
    if w is None:
        return None
    if isinstance(w, torch.Tensor):
        if w.is_cuda or w.dtype != torch.bfloat16:
            raise TypeError(f"{what}: a CPU bfloat16 tensor or a uint16 numpy array")
        w = w.contiguous().view(torch.int16).numpy().view(np.uint16)
    w = np.ascontiguousarray(w, dtype=np.uint16)
    if w.shape != (D,):
        raise ValueError(f"{what}: shape {w.shape}, expected ({D},)")
    return w


class Config(ctypes.Structure):
    _fields_ = [("num_q_heads", _int), ("num_kv_heads", _int), ("head_dim", _int),
                ("max_streams", _int), ("max_context", _int), ("max_verify_rows", _int),
                ("num_layers", _int), ("layers", ctypes.POINTER(LayerConfig)),
                ("max_selected_pages", _int)]


class Cache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("n_rows", _int), ("ring_head", _vp),
                ("ring_count", _vp), ("stream_rows", _vp), ("block_table", _vp),
                ("bt_stride", _int), ("seq_len", _vp)]


class DecodeArgs(ctypes.Structure):
    _fields_ = [("num_streams", _int), ("q", _vp), ("k_new", _vp), ("v_new", _vp), ("gate", _vp),
                ("pos", _vp), ("out", _vp), ("max_seq_len", _int), ("write_back", _int)]


class PageSelection(ctypes.Structure):
    _fields_ = [("summary", _vp), ("num_pages", _int), ("keep_first", _int), ("keep_last", _int),
                ("selected", _vp)]


class VerifyArgs(ctypes.Structure):
    _fields_ = [("num_streams", _int), ("rows", _int), ("q", _vp), ("k", _vp), ("v", _vp),
                ("parent", _vp), ("gate", _vp), ("out", _vp), ("max_prefix_len", _int),
                ("write_back", _int), ("pos", _vp)]


lib.dattn_create.argtypes = [ctypes.POINTER(Config), _int, ctypes.POINTER(_vp)]
lib.dattn_create.restype = _int
lib.dattn_append_kv.argtypes = [_vp, _int, ctypes.POINTER(Cache), _int, _int, _vp, _vp, _vp,
                                _vp, _vp, _int, _vp]
lib.dattn_append_kv.restype = _int
lib.dattn_decode.argtypes = [_vp, _int, ctypes.POINTER(Cache), ctypes.POINTER(DecodeArgs), _vp]
lib.dattn_decode.restype = _int
lib.dattn_sparse_decode.argtypes = [_vp, _int, ctypes.POINTER(Cache), ctypes.POINTER(DecodeArgs),
                                    ctypes.POINTER(PageSelection), _vp]
lib.dattn_sparse_decode.restype = _int
lib.dattn_summarize.argtypes = [_vp, _int, ctypes.POINTER(Cache), _vp, _int, _int, _vp, _vp, _vp]
lib.dattn_summarize.restype = _int
lib.dattn_verify.argtypes = [_vp, _int, ctypes.POINTER(Cache), ctypes.POINTER(VerifyArgs), _vp]
lib.dattn_verify.restype = _int
lib.dattn_commit.argtypes = [_vp, _int, ctypes.POINTER(Cache), _int, _int, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
lib.dattn_commit.restype = _int
lib.dattn_prefill.argtypes = [_vp, _int, ctypes.POINTER(Cache), _int, _int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
lib.dattn_prefill.restype = _int
lib.dattn_get_error.argtypes = [_vp, _vp]
lib.dattn_get_error.restype = _int
lib.dattn_error_string.argtypes = [_int]
lib.dattn_error_string.restype = ctypes.c_char_p
lib.dattn_destroy.argtypes = [_vp]
lib.dattn_destroy.restype = None
lib.dattn_decode_noalloc.argtypes = [ctypes.POINTER(Config), _int, ctypes.POINTER(Cache),
                                     ctypes.POINTER(DecodeArgs), _vp]
lib.dattn_decode_noalloc.restype = _int
lib.dattn_debug_config.argtypes = [_vp, _int, ctypes.c_uint]
lib.dattn_debug_config.restype = _int
DEBUG_WITHHOLD_Q, DEBUG_WITHHOLD_KV = 1, 2

EXPORTS = ("dattn_create", "dattn_append_kv", "dattn_decode", "dattn_verify", "dattn_commit", "dattn_prefill",
           "dattn_get_error", "dattn_error_string", "dattn_destroy", "dattn_decode_noalloc",
           "dattn_debug_config", "dattn_sparse_decode", "dattn_summarize")


class DattnError(RuntimeError):
    def __init__(self, code, what):
        self.code = code
        super().__init__(f"{what}: {error_string(code)} (status {code})")


def error_string(code: int) -> str:
    return lib.dattn_error_string(code).decode()


def _check(code, what):
    if code != OK:
        raise DattnError(code, what)


def _ptr(t):
    if t is None:
        return None
    try:
        if t.is_cuda and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch tensor")
    if not t.is_cuda:
        raise ValueError("dattn takes device tensors")
    raise ValueError("dattn takes contiguous tensors")


# The current stream of a device as an integer. (torch.cuda.current_stream builds
# a Stream object on every call: 3.0 us of the 10 us that a call took on the
# host, against 0.1 us.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_ptr(stream, device=None):
    """A stream's handle; None: the current stream of `device` (of the current one if not given)."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None or device is None:
        return torch.cuda.current_stream(device).cuda_stream
    return _raw_stream(device)


# ---------------------------------------------------------------- cache descriptors

def ring_cache(k, v, ring_head, ring_count, stream_rows=None) -> Cache:
    """k, v: [rows, Hkv, R, D] bf16; ring_head, ring_count (, stream_rows): [B] int32.
    The descriptor holds the tensors it points to, so they live as long as it does."""
    c = Cache(_ptr(k), _ptr(v), k.shape[0], _ptr(ring_head), _ptr(ring_count),
              _ptr(stream_rows), None, 0, None)
    c._tensors = (k, v, ring_head, ring_count, stream_rows)
    return c


def paged_cache(k, v, block_table, seq_len) -> Cache:
    """k, v: [pages, Hkv, P, D] bf16; block_table [B, max_pages] int32; seq_len [B] int32.
    The descriptor holds the tensors it points to, so they live as long as it does."""
    c = Cache(_ptr(k), _ptr(v), k.shape[0], None, None, None, _ptr(block_table),
              block_table.shape[1], _ptr(seq_len))
    c._tensors = (k, v, block_table, seq_len)
    return c


def state_cache(state, stream_rows=None) -> Cache:
    """state: [rows, Hkv, D, D] fp32 of a state layer; stream_rows: [B] int32 or None.
    The descriptor holds the tensors it points to, so they live as long as it does."""
    if state.dtype != torch.float32:
        raise TypeError("a state layer's cache is fp32")
    if state.dim() != 4 or state.shape[2] != state.shape[3]:
        raise ValueError(f"state: shape {tuple(state.shape)}, expected (rows, Hkv, D, D)")
    if stream_rows is not None and stream_rows.dtype != torch.int32:
        raise TypeError("stream_rows: int32")
    c = Cache(_ptr(state), None, state.shape[0], None, None, _ptr(stream_rows), None, 0, None)
    c._tensors = (state, stream_rows)
    # what a handle compares on every call: heads and dims, and the streams it has rows for
    c._state = list(state.shape[1:3])
    c._streams = None if stream_rows is None else stream_rows.numel()
    return c


# ---------------------------------------------------------------- handle

class Handle:
    """A dattn handle: per-layer RoPE tables and the split-K workspace."""

    def __init__(self, num_q_heads, num_kv_heads, head_dim, layers, max_streams,
                 max_context=0, max_verify_rows=0, device=None, max_selected_pages=0):
        if device is not None and not isinstance(device, int):
            device = torch.device(device)
            if device.type != "cuda":
                raise ValueError(f"a handle is on a CUDA device, not {device}")
            device = device.index  # (None: the current one)
        self.device = device = torch.cuda.current_device() if device is None else device
        # QK-norm weights (layer keys "q_norm", "k_norm", "norm_eps") and state
        # layers' decays ("log_decay" [Hkv]): host arrays the config points at,
        # kept alive with it (dattn_create copies them; decode_noalloc reads the
        # weights on every call)
        self._norm_keep = []
        cfgs = []
        for l in layers:
            qn = _host_bf16(l.get("q_norm"), head_dim, "q_norm")
            kn = _host_bf16(l.get("k_norm"), head_dim, "k_norm")
            ld = _host_f32(l.get("log_decay"), num_kv_heads, "log_decay")
            self._norm_keep += [qn, kn, ld]
            cfgs.append(LayerConfig(l["kind"], l.get("ring_slots", 0), l.get("page_size", 0),
                                    l.get("rotary_dim", 0), float(l.get("rope_theta", 0.0)),
                                    None if qn is None else qn.ctypes.data,
                                    None if kn is None else kn.ctypes.data,
                                    float(l.get("norm_eps", 0.0)), int(l.get("kv_format", KV_BF16)),
                                    float(l.get("k_scale", 1.0)), float(l.get("v_scale", 1.0)),
                                    None if ld is None else ld.ctypes.data))
        self._layers = (LayerConfig * len(layers))(*cfgs)
        # (for the checks of every call: plain Python values; a structure's field or a
        # tensor's sliced shape takes longer than the whole check)
        self._kinds = {i: l["kind"] for i, l in enumerate(layers)}
        self._heads = [num_kv_heads, head_dim]
        self.config = Config(num_q_heads, num_kv_heads, head_dim, max_streams, max_context,
                             max_verify_rows, len(layers), self._layers, max_selected_pages)
        h = _vp()
        _check(lib.dattn_create(ctypes.byref(self.config), device, ctypes.byref(h)), "dattn_create")
        self._h = h

    @property
    def ptr(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            lib.dattn_destroy(self._h)
            self._h = _vp()

    __del__ = close

    def _check_state(self, cache, streams):
        """A state layer's call has states of this handle's heads, and a row for each stream."""
        if not hasattr(cache, "_tensors"):
            return  # (a descriptor of the caller's own)
        if getattr(cache, "_state", None) != self._heads:
            raise ValueError(f"a state layer's cache: {cache._tensors[0].dtype} {tuple(cache._tensors[0].shape)}, expected "
                             f"state_cache of (rows, {self._heads[0]}, {self._heads[1]}, {self._heads[1]})")
        if cache._streams is not None and cache._streams < streams:
            raise ValueError(f"stream_rows: {cache._streams} rows for {streams} streams")

    def _check_summary(self, cache, summary):
        """A paged layer's summaries: one for each page and KV head."""
        if summary.dtype is not _BF16:
            raise TypeError(f"summary: {summary.dtype}, expected bf16")
        pages, *heads = summary.shape
        if pages < cache.n_rows or heads != self._heads:
            raise ValueError(f"summary: shape {tuple(summary.shape)}, expected ({cache.n_rows} pages, {self._heads[0]}, "
                             f"{self._heads[1]})")

    def append_kv(self, layer, cache: Cache, k, v, start_index, count, start_pos=None,
                  rotate=True, stream=None):
        """k, v: [B, T, Hkv, D] bf16; start_index, count (, start_pos): [B] int32."""
        B, T = k.shape[0], k.shape[1]
        _check(lib.dattn_append_kv(self._h, layer, ctypes.byref(cache), B, T, _ptr(start_index),
                                   _ptr(start_pos), _ptr(count), _ptr(k), _ptr(v), int(rotate),
                                   _stream_ptr(stream, self.device)), "dattn_append_kv")

    def decode(self, layer, cache: Cache, q, k_new, v_new, pos, out, gate=None, max_seq_len=0,
               write_back=True, stream=None):
        """q [B, Hq, D], k_new/v_new [B, Hkv, D] bf16; pos [B] int32; out [B, Hq, D] fp32;
        gate [B, Hq] bf16 or None."""
        B = q.shape[0]
        if self._kinds.get(layer) == CACHE_STATE:
            self._check_state(cache, B)
        args = DecodeArgs(B, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(gate), _ptr(pos),
                          _ptr(out), int(max_seq_len), int(write_back))
        _check(lib.dattn_decode(self._h, layer, ctypes.byref(cache), ctypes.byref(args),
                                _stream_ptr(stream, self.device)), "dattn_decode")

    def sparse_decode(self, layer, cache: Cache, summary, q, k_new, v_new, pos, out, num_pages, keep_first=1,
                      keep_last=1, gate=None, max_seq_len=0, write_back=True, selected=None, stream=None):
        """decode over the num_pages pages of each stream and KV head that score highest
        (the first keep_first and the newest keep_last are always read): summary
        [pages, Hkv, D] bf16 as `summarize` keeps it; selected [B, Hkv, num_pages] int32
        receives the pages (ascending, then -1) if given. The handle needs
        max_selected_pages >= num_pages."""
        if summary is not None and self._kinds.get(layer) == CACHE_PAGED:
            self._check_summary(cache, summary)
        args = DecodeArgs(q.shape[0], _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(gate), _ptr(pos),
                          _ptr(out), int(max_seq_len), int(write_back))
        if selected is not None and (selected.dtype != torch.int32 or selected.numel() !=
                                     q.shape[0] * self.config.num_kv_heads * num_pages):
            raise ValueError("selected: int32 [B, Hkv, num_pages]")
        sel = PageSelection(_ptr(summary), int(num_pages), int(keep_first), int(keep_last), _ptr(selected))
        _check(lib.dattn_sparse_decode(self._h, layer, ctypes.byref(cache), ctypes.byref(args), ctypes.byref(sel),
                                       _stream_ptr(stream, self.device)), "dattn_sparse_decode")

    def summarize(self, layer, cache: Cache, summary, start_index, count, max_tokens, stream=None):
        """Summaries (bf16 means of the stored keys, [pages, Hkv, D]) of the pages that the
        new tokens [start_index, start_index + count) of each row completed; start_index,
        count: [B] int32, count <= max_tokens."""
        if summary is not None and self._kinds.get(layer) == CACHE_PAGED:
            self._check_summary(cache, summary)
        B = start_index.shape[0]
        if start_index.dtype is not _I32 or count.dtype is not _I32 or count.numel() != B:
            raise ValueError("start_index, count: int32 [B]")
        _check(lib.dattn_summarize(self._h, layer, ctypes.byref(cache), _ptr(summary), B, int(max_tokens),
                                   _ptr(start_index), _ptr(count), _stream_ptr(stream, self.device)), "dattn_summarize")

    def verify(self, layer, cache: Cache, q, k, v, parent, out, gate=None, max_prefix_len=0,
               write_back=True, pos=None, stream=None):
        """q [S, T, Hq, D], k/v [S, T, Hkv, D] bf16; parent [S, T] int32; out [S, T, Hq, D]
        fp32; gate [S, T, Hq] bf16 or None; pos [S] int32 root positions (default: the
        cache's seq_len; ring layers need it and take write_back=False)."""
        args = VerifyArgs(q.shape[0], q.shape[1], _ptr(q), _ptr(k), _ptr(v), _ptr(parent),
                          _ptr(gate), _ptr(out), int(max_prefix_len), int(write_back), _ptr(pos))
        _check(lib.dattn_verify(self._h, layer, ctypes.byref(cache), ctypes.byref(args),
                                _stream_ptr(stream, self.device)), "dattn_verify")

    def commit(self, layer, cache: Cache, k, v, parent, accepted, num_accepted, pos, stream=None):
        """Write each stream's accepted path (accepted [S, T] int32 node indices root
        first, num_accepted [S]) at the cache's next indices, rotated at pos + d;
        k, v, parent as given to the verify call."""
        _check(lib.dattn_commit(self._h, layer, ctypes.byref(cache), k.shape[0], k.shape[1], _ptr(k),
                                _ptr(v), _ptr(parent), _ptr(accepted), _ptr(num_accepted), _ptr(pos),
                                _stream_ptr(stream, self.device)), "dattn_commit")

    def prefill(self, layer, cache: Cache, q, k, v, count, start_pos, out, gate=None, stream=None):
        """Ragged prefill: q [S, T, Hq, D], k/v [S, T, Hkv, D] bf16, count/start_pos [S] int32,
        out [S, T, Hq, D] fp32 (rows t < count written), gate [S, T, Hq] bf16 or None."""
        B, T = q.shape[0], q.shape[1]
        if self._kinds.get(layer) == CACHE_STATE:
            self._check_state(cache, B)
        _check(lib.dattn_prefill(self._h, layer, ctypes.byref(cache), B, T, _ptr(q), _ptr(k),
                                 _ptr(v), _ptr(gate), _ptr(count), _ptr(start_pos), _ptr(out),
                                 _stream_ptr(stream, self.device)), "dattn_prefill")

    def debug_config(self, flags=0, wait_limit_us=0):
        """Testing aid: the limit of the device's bounded waits and fault
        injection on the host's side of the wait (see dattn_debug_config)."""
        _check(lib.dattn_debug_config(self._h, int(flags), int(wait_limit_us)), "dattn_debug_config")

    def get_error(self, stream=None) -> int:
        """Synchronize the stream; return and clear the sticky device status."""
        return lib.dattn_get_error(self._h, _stream_ptr(stream, self.device))


def decode_noalloc(config: Config, layer, cache: Cache, q, k_new, v_new, pos, out, gate=None,
                   max_seq_len=0, write_back=True, stream=None):
    """Decode without a handle, for callers that cannot allocate device memory:
    the library's fixed scratch array stands in for a handle's workspace.
    `config` is a Config structure (for instance Handle.config)."""
    args = DecodeArgs(q.shape[0], _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(gate), _ptr(pos),
                      _ptr(out), int(max_seq_len), int(write_back))
    _check(lib.dattn_decode_noalloc(ctypes.byref(config), layer, ctypes.byref(cache),
                                    ctypes.byref(args), _stream_ptr(stream)), "dattn_decode_noalloc")
