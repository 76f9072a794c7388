"""Python binding of libq8attn.so (ctypes).

Argument marshalling only: every step of the computation runs in the
library's CUDA kernels.  Tensors are torch CUDA tensors; their device pointers
and the current torch stream are handed to the C ABI declared in
include/q8attn.h.  There is no CPU fallback: if the library is missing or fails
to load, every call raises.  No call records history for torch's autograd: results
do not require a gradient, whatever their inputs do.
"""

import ctypes
import functools
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# Q8ATTN_LIBRARY selects another in-tree build of the same library (the
# sanitizer build the host-code tests load); it is never a fallback.
LIB_PATH = os.environ.get("Q8ATTN_LIBRARY") or os.path.join(_HERE, "libq8attn.so")

Q8A_OK = 0
Q8A_ERR_INVALID_ARG = -1
Q8A_ERR_MISALIGNED = -2
Q8A_ERR_UNSUPPORTED = -3
Q8A_ERR_CUDA = -4
Q8A_ERR_TIMEOUT = -5
ROW_BYTES = 68
HEAD_DIM = 64

# name -> (restype, argtypes); mirrors include/q8attn.h
_I64, _I32, _U32, _U64, _P, _F = (ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32, ctypes.c_uint64,
                                  ctypes.c_void_p, ctypes.c_float)
SIGNATURES = {
    "q8a_abi_version": (_U32, []),
    "q8a_last_error": (ctypes.c_char_p, []),
    "q8a_plane_stride_bytes": (_I64, [_I64]),
    "q8a_plane_stride_bytes_for": (_I64, [_I64, _I32]),
    "q8kv_quantize": (ctypes.c_int, [_P, _P, _I64, _I64, _I32, _I32, _I64, _P]),
    "attn_state_init": (ctypes.c_int, [_P, _P, _P, _I64, _I32, _I64, _I32, _P]),
    "attn_chunk_step": (ctypes.c_int, [_P, _I64, _P, _P, _I64, _I64, _I64, _P, _P, _P, _I64, _I32,
                                       _I64, _I32, _F, _I32, _P]),
    "attn_chunk_step_gqa": (ctypes.c_int, [_P, _I64, _P, _P, _I64, _I64, _I64, _P, _P, _P, _I64,
                                           _I32, _I32, _I64, _I32, _F, _I32, _P]),
    "attn_chunk_step_split": (ctypes.c_int, [_P, _I64, _P, _P, _I64, _I64, _I64, _P, _P, _P, _I64,
                                             _I32, _I64, _I32, _F, _I32, _I64, _P, _I64, _P]),
    "attn_chunk_step_split_gqa": (ctypes.c_int, [_P, _I64, _P, _P, _I64, _I64, _I64, _P, _P, _P, _I64,
                                                 _I32, _I32, _I64, _I32, _F, _I32, _I64, _P, _I64, _P]),
    "q8a_split_workspace_floats": (_I64, [_I64, _I32, _I64, _I64, _I64]),
    "q8a_split_workspace_floats_for": (_I64, [_I64, _I32, _I64, _I64, _I64, _I32]),
    "attn_chunk_step_split_static": (ctypes.c_int, [_P, _I64, _P, _P, _I64, _I64, _I64, _P, _P, _P,
                                                    _I64, _I32, _I64, _I32, _F, _I32, _I64, _P]),
    "q8a_static_split_scratch_floats": (_I64, []),
    "attn_finalize": (ctypes.c_int, [_P, _P, _P, _I64, _I32, _I64, _I32, _P]),
    "attn_prefill_pipelined": (ctypes.c_int, [_P, _P, _P, _P, _I64, _I32, _I64, _I32, _I64, _F, _I32,
                                              _P, _P, _I64, _P, _P, _I64, _P, _P, _P, _P, _P, _P]),
    "q8a_prefill_slot_floats": (_I64, [_I64, _I32, _I64]),
    "q8a_prefill_slot_floats_for": (_I64, [_I64, _I32, _I64, _I32]),
    "q8a_prefill_graph_create": (ctypes.c_int, [_P, _P, _P, _P, _P, _I64, _P, _P, _P, _P, _I64, _I32,
                                                _I64, _I32, _I64, _F, _I32, ctypes.POINTER(_P)]),
    "q8a_prefill_graph_launch": (ctypes.c_int, [_P, _P]),
    "q8a_prefill_graph_destroy": (ctypes.c_int, [_P]),
    "attn_rope": (ctypes.c_int, [_P, _P, _I32, _I64, _I32, _I32, _I64, _I64, _P, _P, _I32, _I32, _F, _I32,
                                 _P]),
    "q8kv_append_paged": (ctypes.c_int, [_P, _P, _I32, _I64, _I32, _I32, _I64, _I64, _P, _P, _P, _I64, _I32,
                                         _I64, _P, _P, _I32, _I32, _F, _P]),
    "q8kv_read_paged": (ctypes.c_int, [_P, _P, _I64, _I32, _I64, _P, _I64, _I32, _I32, _P, _P, _I32, _P]),
    "attn_paged": (ctypes.c_int, [_P, _I32, _I64, _I64, _I32, _I32, _I32, _P, _P, _I64, _I32, _I64, _P, _I64,
                                  _P, _P, _I64, _I64, _I64, _F, _I32, _P, _P, _I64, _P]),
    "q8a_paged_workspace_floats": (_I64, [_I64, _I64, _I32, _I32, _I64, _I64, _I32]),
    "q8a_device_status": (ctypes.c_int, [_P, ctypes.POINTER(_U32), _I32]),
    "q8a_status": (ctypes.c_int, [_P]),
    "q8a_set_wait_timeout_ns": (ctypes.c_int, [_U64]),
    "q8a_test_inject": (ctypes.c_int, [_I32]),
}

_lib = None


class Q8AttnError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"q8attn error {code}: {msg}")
        self.code = code


def load():
    """Load the in-tree shared library (raises if it is missing)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _check(rc):
    if rc != Q8A_OK:
        raise Q8AttnError(rc, load().q8a_last_error().decode())


def _stream(t):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def row_bytes(head_dim):
    """Bytes of one Q8_0 head row: head_dim / 32 blocks of 34 bytes."""
    return head_dim // 32 * 34


def plane_stride(n_tokens, head_dim=HEAD_DIM):
    return int(load().q8a_plane_stride_bytes_for(n_tokens, head_dim))


def q8kv_quantize(x, out=None, stride=None):
    """x: fp32 CUDA [B, M, H, D] (D = 64 or 128) -> uint8 [B, H, stride] Q8_0
    planes (rows of D/32*34 B)."""
    B, M, H, D = x.shape
    if stride is None:
        stride = plane_stride(M, D)
    if out is None:
        out = torch.empty((B, H, stride), dtype=torch.uint8, device=x.device)
    _check(load().q8kv_quantize(_ptr(x), _ptr(out), B, M, H, D, stride, _stream(x)))
    return out


class State:
    """Persistent per-row online-softmax state (fp32): m, l [B, H, n_q]; O [B, H, n_q, D]."""

    def __init__(self, batch, heads, n_q, device, init=True, head_dim=HEAD_DIM):
        self.m = torch.empty((batch, heads, n_q), dtype=torch.float32, device=device)
        self.l = torch.empty((batch, heads, n_q), dtype=torch.float32, device=device)
        self.o = torch.empty((batch, heads, n_q, head_dim), dtype=torch.float32, device=device)
        if init:
            attn_state_init(self)

    @property
    def shape(self):
        return self.m.shape

    @property
    def head_dim(self):
        return self.o.shape[-1]


def attn_state_init(state):
    B, H, n = state.shape
    _check(load().attn_state_init(_ptr(state.m), _ptr(state.l), _ptr(state.o), B, H, n, state.head_dim,
                                  _stream(state.m)))
    return state


def attn_chunk_step(q, k8, v8, kv_start, kv_len, state, q_pos0=0, scale=None, causal=True,
                    stride=None, k_offset_bytes=0):
    """Fold KV keys [kv_start, kv_start + kv_len) into `state`.

    q: fp16 [B, n_q, H, D]; k8, v8: uint8 Q8_0 planes [B, H, stride] whose byte
    `k_offset_bytes` is the chunk's key 0 (so a whole-sequence buffer is passed
    with k_offset_bytes = kv_start * row_bytes(D))."""
    B, n_q, H, D = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if stride is None:
        stride = k8.shape[-1]
    lib = load()
    kp = ctypes.c_void_p(k8.data_ptr() + k_offset_bytes)
    vp = ctypes.c_void_p(v8.data_ptr() + k_offset_bytes)
    _check(lib.attn_chunk_step(_ptr(q), q_pos0, kp, vp, stride, kv_start, kv_len, _ptr(state.m),
                               _ptr(state.l), _ptr(state.o), B, H, n_q, D, scale, int(bool(causal)),
                               _stream(q)))
    return state


def attn_chunk_step_gqa(q, k8, v8, kv_start, kv_len, state, q_pos0=0, scale=None, causal=True,
                        stride=None, k_offset_bytes=0):
    """attn_chunk_step for grouped-query attention: k8, v8 hold kv_heads =
    k8.shape[1] planes per batch entry and query head h reads plane
    h // (H // kv_heads)."""
    B, n_q, H, D = q.shape
    kv_heads = k8.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if stride is None:
        stride = k8.shape[-1]
    lib = load()
    kp = ctypes.c_void_p(k8.data_ptr() + k_offset_bytes)
    vp = ctypes.c_void_p(v8.data_ptr() + k_offset_bytes)
    _check(lib.attn_chunk_step_gqa(_ptr(q), q_pos0, kp, vp, stride, kv_start, kv_len, _ptr(state.m),
                                   _ptr(state.l), _ptr(state.o), B, H, kv_heads, n_q, D, scale,
                                   int(bool(causal)), _stream(q)))
    return state


def split_workspace_floats(batch, heads, n_q, kv_len, split_keys, head_dim=HEAD_DIM):
    n = int(load().q8a_split_workspace_floats_for(batch, heads, n_q, kv_len, split_keys, head_dim))
    if n < 0:
        raise Q8AttnError(Q8A_ERR_INVALID_ARG, "invalid sizes for the split workspace")
    return n


def split_keys_for(bh, kv_len, sms, max_waves=8, min_keys=2048):
    """Key-range length for attn_chunk_step_split.  The split launch runs one
    CTA per (batch, head) and key range, one CTA per SM, so the range count n
    is chosen to make n * bh a whole number of waves: the fewest waves (up to
    max_waves) whose CTA count bh divides, keeping ranges of at least min_keys
    keys; the length is rounded up to whole 128-key tiles.  Without such a
    count, ranges of 8,192 keys."""
    if bh <= 0 or kv_len <= 0 or sms <= 0:
        raise ValueError("bh, kv_len and sms must be positive")
    for waves in range(1, max_waves + 1):
        if (waves * sms) % bh == 0:
            n = waves * sms // bh
            length = -(-(-(-kv_len // n)) // 128) * 128
            if length >= min_keys:
                return length
    return 8192


def attn_chunk_step_split(q, k8, v8, kv_start, kv_len, state, split_keys, workspace=None, q_pos0=0,
                          scale=None, causal=True, stride=None, k_offset_bytes=0):
    """attn_chunk_step with the chunk's keys folded in parallel ranges of
    `split_keys` keys and merged.  `workspace`: fp32 CUDA tensor of at least
    split_workspace_floats(...) elements (allocated here when None)."""
    B, n_q, H, D = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if stride is None:
        stride = k8.shape[-1]
    need = split_workspace_floats(B, H, n_q, kv_len, split_keys, D)
    if workspace is None:
        workspace = torch.empty((max(need, 1),), dtype=torch.float32, device=q.device)
    lib = load()
    kp = ctypes.c_void_p(k8.data_ptr() + k_offset_bytes)
    vp = ctypes.c_void_p(v8.data_ptr() + k_offset_bytes)
    _check(lib.attn_chunk_step_split(_ptr(q), q_pos0, kp, vp, stride, kv_start, kv_len,
                                     _ptr(state.m), _ptr(state.l), _ptr(state.o), B, H, n_q, D,
                                     scale, int(bool(causal)), split_keys, _ptr(workspace),
                                     workspace.numel(), _stream(q)))
    return state


def attn_chunk_step_split_gqa(q, k8, v8, kv_start, kv_len, state, split_keys, workspace=None, q_pos0=0,
                              scale=None, causal=True, stride=None, k_offset_bytes=0):
    """attn_chunk_step_split with k8, v8 holding H_kv planes per sequence
    ([B, H_kv, stride]); query head h reads plane h // (H // H_kv)."""
    B, n_q, H, D = q.shape
    H_kv = k8.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if stride is None:
        stride = k8.shape[-1]
    need = split_workspace_floats(B, H, n_q, kv_len, split_keys, D)
    if workspace is None:
        workspace = torch.empty((max(need, 1),), dtype=torch.float32, device=q.device)
    kp = ctypes.c_void_p(k8.data_ptr() + k_offset_bytes)
    vp = ctypes.c_void_p(v8.data_ptr() + k_offset_bytes)
    _check(load().attn_chunk_step_split_gqa(_ptr(q), q_pos0, kp, vp, stride, kv_start, kv_len,
                                            _ptr(state.m), _ptr(state.l), _ptr(state.o), B, H, H_kv, n_q, D,
                                            scale, int(bool(causal)), split_keys, _ptr(workspace),
                                            workspace.numel(), _stream(q)))
    return state


def attn_finalize(state, out=None):
    """O / l -> fp16 [B, n_q, H, D]."""
    B, H, n = state.shape
    if out is None:
        out = torch.empty((B, n, H, state.head_dim), dtype=torch.float16, device=state.m.device)
    _check(load().attn_finalize(_ptr(state.l), _ptr(state.o), _ptr(out), B, H, n, state.head_dim,
                                _stream(state.m)))
    return out


def prefill_attention(q, k, v, chunk, scale=None, causal=True, k8=None, v8=None, state=None, out=None):
    """The whole path: quantise K and V, initialise the state, fold every KV
    chunk of `chunk` keys in order, finalise.  Returns (out, k8, v8)."""
    B, M, H, D = q.shape
    k8 = q8kv_quantize(k, k8)
    v8 = q8kv_quantize(v, v8)
    if state is None:
        state = State(B, H, M, q.device, init=True, head_dim=D)
    else:
        attn_state_init(state)
    for s0 in range(0, M, chunk):
        n = min(chunk, M - s0)
        attn_chunk_step(q, k8, v8, s0, n, state, scale=scale, causal=causal,
                        k_offset_bytes=s0 * row_bytes(D))
    out = attn_finalize(state, out)
    return out, k8, v8


class PrefillGraph:
    """prefill_attention captured once into a CUDA graph
    (q8a_prefill_graph_create) and replayed with one launch per call.  The
    graph keeps the tensors' addresses: their contents may change between
    launches, so a new prefill of the same shape writes its Q, K and V into
    .q/.k/.v (the caller's tensors) and launches again."""

    def __init__(self, q, k, v, chunk, scale=None, causal=True):
        B, M, H, D = q.shape
        if scale is None:
            scale = 1.0 / math.sqrt(D)
        self.q, self.k, self.v = q, k, v
        self.stride = plane_stride(M, D)
        self.k8 = torch.empty((B, H, self.stride), dtype=torch.uint8, device=q.device)
        self.v8 = torch.empty((B, H, self.stride), dtype=torch.uint8, device=q.device)
        self.state = State(B, H, M, q.device, init=False, head_dim=D)
        self.out = torch.empty((B, M, H, D), dtype=torch.float16, device=q.device)
        self._h = None
        h = ctypes.c_void_p()
        st = self.state
        with torch.cuda.device(q.device):
            _check(load().q8a_prefill_graph_create(
                _ptr(q), _ptr(k), _ptr(v), _ptr(self.k8), _ptr(self.v8), self.stride, _ptr(st.m),
                _ptr(st.l), _ptr(st.o), _ptr(self.out), B, H, M, D, chunk, scale, int(bool(causal)),
                ctypes.byref(h)))
        self._h = h

    def launch(self, stream=None):
        """Enqueue one replay on `stream` (default: the current stream); returns .out."""
        s = stream if stream is not None else torch.cuda.current_stream(self.out.device)
        with torch.cuda.device(self.out.device):
            _check(load().q8a_prefill_graph_launch(self._h, ctypes.c_void_p(s.cuda_stream)))
        return self.out

    def close(self):
        if self._h is not None and _lib is not None:
            _lib.q8a_prefill_graph_destroy(self._h)
        self._h = None

    def __del__(self):
        self.close()


class PipelineBuffers:
    """Device buffers of attn_prefill_pipelined for one problem size and chunk:
    Q and the output (whole sequence), two chunk slots of fp32 K and V, the
    Q8_0 planes of the whole sequence and the state."""

    def __init__(self, batch, n_tokens, heads, device, chunk, head_dim=HEAD_DIM):
        shape = (batch, n_tokens, heads, head_dim)
        self.chunk = chunk
        self.q = torch.empty(shape, dtype=torch.float16, device=device)
        self.out = torch.empty(shape, dtype=torch.float16, device=device)
        n_slot = int(load().q8a_prefill_slot_floats_for(batch, heads, min(chunk, n_tokens), head_dim))
        if n_slot < 0:
            raise Q8AttnError(Q8A_ERR_INVALID_ARG, "invalid sizes for the prefill slots")
        self.kv_slots = torch.empty((n_slot,), dtype=torch.float32, device=device)
        self.stride = plane_stride(n_tokens, head_dim)
        self.k8 = torch.empty((batch, heads, self.stride), dtype=torch.uint8, device=device)
        self.v8 = torch.empty((batch, heads, self.stride), dtype=torch.uint8, device=device)
        self.state = State(batch, heads, n_tokens, device, init=False, head_dim=head_dim)
        self.copy_stream = torch.cuda.Stream(device=device)


def attn_prefill_pipelined(q_host, k_host, v_host, out_host, bufs, scale=None, causal=True):
    """The whole prefill from host tensors (page-locked for overlap) in chunks of
    bufs.chunk tokens: K/V chunk copies on bufs.copy_stream into two device
    slots overlap quantise + chunk step on the current stream; the output lands
    in out_host once the current stream drains."""
    B, M, H, D = q_host.shape
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    st = bufs.state
    _check(load().attn_prefill_pipelined(
        _ptr(q_host), _ptr(k_host), _ptr(v_host), _ptr(out_host), B, H, M, D, bufs.chunk, scale,
        int(bool(causal)), _ptr(bufs.q), _ptr(bufs.kv_slots), bufs.kv_slots.numel(), _ptr(bufs.k8),
        _ptr(bufs.v8), bufs.stride, _ptr(st.m), _ptr(st.l), _ptr(st.o), _ptr(bufs.out),
        _stream(bufs.q), ctypes.c_void_p(bufs.copy_stream.cuda_stream)))
    return out_host


# ---- rotary positions and the paged cache -----------------------------------
# What can be told from shapes, types and devices is refused here, before the call;
# the indices that device tensors hold are checked by the kernels.  A step of a
# server makes these calls once per layer, so an accepted call costs one
# condition: the messages are formed only by the functions that refuse.

_DTYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}


def _refuse(msg):
    raise Q8AttnError(Q8A_ERR_INVALID_ARG, msg)


def _bad_packed(**tensors):
    """Refuse packed [T, H, D] tensors: type, device, shape or strides."""
    for name, t in tensors.items():
        if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 3 and t.dtype in _DTYPES):
            _refuse(f"{name}: a CUDA tensor [tokens, heads, head_dim] of fp16, bf16 or fp32 is needed")
    shapes = {n: (tuple(t.shape), t.dtype, str(t.device)) for n, t in tensors.items()}
    _refuse(f"packed tensors must agree in shape, type and device, each token's heads contiguous: {shapes}")


def _bad_index(name, t, dtype, n, device):
    got = (t.dtype, tuple(t.shape), str(t.device)) if isinstance(t, torch.Tensor) else type(t)
    _refuse(f"{name}: {n} contiguous values of {dtype} on cuda:{device} are needed, got {got}")


def _index(name, t, dtype, n, device):
    """Check a one-dimensional index tensor of n values; its address."""
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.dim() == 1 and t.shape[0] == n and
            t.is_contiguous() and t.get_device() == device):
        _bad_index(name, t, dtype, n, device)
    return t.data_ptr()


def _packed(name, t, device):
    """(dtype code, T, H, D, token stride in elements) of a packed tensor whose heads are contiguous."""
    code = _DTYPES.get(t.dtype) if isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 3 else None
    if code is None or t.get_device() != device:
        _bad_packed(**{name: t})
    T, H, D = t.shape
    st, sh, sd = t.stride()
    if (D > 1 and sd != 1) or (H > 1 and sh != D):
        _bad_packed(**{name: t})
    return code, T, H, D, (st if T > 1 else max(H * D, 1))


def _device_of(t):
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        _refuse("CUDA tensors are needed")
    return t.get_device()


def _pool(k_pages, v_pages, device):
    """(n_pages, kv_heads, page_tokens, head_dim, page stride in bytes) of uint8 pages [n_pages, H_kv,
    page_tokens, row bytes], contiguous within a page (the pools may be interleaved, page by page)."""
    ok = (isinstance(k_pages, torch.Tensor) and isinstance(v_pages, torch.Tensor) and k_pages.dim() == 4 and
          k_pages.dtype == v_pages.dtype == torch.uint8 and k_pages.get_device() == v_pages.get_device() == device and
          k_pages.shape == v_pages.shape and k_pages.stride() == v_pages.stride())
    if ok:
        n, H, P, rb = k_pages.shape
        sn, sh, sp, sb = k_pages.stride()
        ok = rb in (68, 136) and sb == 1 and (sp == rb or P <= 1) and (sh == P * rb or H <= 1)
    if not ok:
        _refuse(f"k_pages and v_pages: uint8 tensors [n_pages, kv_heads, page_tokens, 68 or 136] of the same shape "
                f"and strides on cuda:{device}, each page contiguous, are needed")
    return n, H, P, rb // 34 * 32, (sn if n > 1 else H * P * rb)


def _rope_table(inv_freq, device):
    if not (isinstance(inv_freq, torch.Tensor) and inv_freq.dtype == torch.float64 and inv_freq.dim() == 1 and
            inv_freq.is_contiguous() and inv_freq.get_device() == device):
        _bad_index("inv_freq", inv_freq, torch.float64, "rot_dim / 2", device)
    return inv_freq.data_ptr(), 2 * inv_freq.shape[0]


def _call(fn, device, *args):
    """fn(*args, current stream of `device`) with that device current."""
    stream = torch._C._cuda_getCurrentRawStream(device)
    if torch._C._cuda_getDevice() == device:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, stream)
    if rc != Q8A_OK:
        _check(rc)


def rope_inv_freq(rot_dim, base=10000.0, factor=1.0, scaling="linear", original_len=None, low=1.0, high=4.0,
                  device=None):
    """fp64 [rot_dim / 2] radians per position: base^(-2i / rot_dim), for a context
    `factor` times as long as the original:
      "linear"  every frequency divided by factor (positions interpolated);
      "base"    the base raised to base * factor^(rot_dim / (rot_dim - 2)), which divides the lowest
                frequency by factor and leaves the highest;
      "bands"   frequencies that turn more than `high` times within original_len tokens are kept, those
                that turn less than `low` times are divided by factor, those between are blended."""
    if rot_dim <= 0 or rot_dim % 2:
        raise ValueError("rot_dim must be even and positive")
    if factor <= 0 or base <= 0:
        raise ValueError("base and factor must be positive")
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    if scaling == "base":
        if rot_dim > 2:
            base = base * factor ** (rot_dim / (rot_dim - 2))
        f = base ** (-i / rot_dim)
    elif scaling == "linear":
        f = base ** (-i / rot_dim) / factor
    elif scaling == "bands":
        if original_len is None or original_len <= 0 or high <= low:
            raise ValueError("bands need original_len > 0 and high > low")
        f = base ** (-i / rot_dim)
        keep = ((original_len * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    else:
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.to(device) if device is not None else f


def attn_rope(x, positions, inv_freq, interleaved=False, mscale=1.0, inverse=False, out=None):
    """Rotary positions of packed x [T, H, D] (fp16, bf16 or fp32; a slice of a wider buffer is fine):
    the first 2 * len(inv_freq) channels of every head turned by positions [T] (int64) times inv_freq
    (fp64, see rope_inv_freq).  `out` may be x.  `inverse` turns back: of a gradient in out, the gradient in x
    (torch's autograd does not call it by itself)."""
    device = _device_of(x)
    code, T, H, D, stride = _packed("x", x, device)
    pos = _index("positions", positions, torch.int64, T, device)
    table, rot = _rope_table(inv_freq, device)
    if out is None:
        out = torch.empty((T, H, D), dtype=x.dtype, device=x.device)
        out_stride = max(H * D, 1)
    else:
        out_code, *shape, out_stride = _packed("out", out, device)
        if out_code != code or shape != [T, H, D]:
            _bad_packed(x=x, out=out)
    _call(load().attn_rope, device, x.data_ptr(), out.data_ptr(), code, T, H, D, stride, out_stride, pos, table, rot,
          1 if interleaved else 0, mscale, 1 if inverse else 0)
    return out


def q8kv_append_paged(k, v, k_pages, v_pages, slots, positions=None, inv_freq=None, interleaved=False, mscale=1.0):
    """Quantise packed k, v [T, H_kv, D] (fp16, bf16 or fp32) into pages: uint8 k_pages, v_pages
    [n_pages, H_kv, page_tokens, D / 32 * 34], row t to slot slots[t] (int64: page * page_tokens + offset;
    negative: skipped).  With positions and inv_freq the keys are rotated first, as attn_rope does."""
    device = _device_of(k)
    code, T, H, D, k_stride = _packed("k", k, device)
    v_code, *shape, v_stride = _packed("v", v, device)
    n_pages, kv_heads, page_tokens, head_dim, page_stride = _pool(k_pages, v_pages, device)
    if v_code != code or shape != [T, H, D] or H != kv_heads or D != head_dim:
        _refuse(f"k {tuple(k.shape)}, v {tuple(v.shape)} and the pages ({kv_heads} heads, head_dim {head_dim}) must agree")
    at = _index("slots", slots, torch.int64, T, device)
    if (positions is None) != (inv_freq is None):
        _refuse("positions and inv_freq come together")
    pos = table = rot = 0
    if positions is not None:
        pos = _index("positions", positions, torch.int64, T, device)
        table, rot = _rope_table(inv_freq, device)
    _call(load().q8kv_append_paged, device, k.data_ptr(), v.data_ptr(), code, T, H, D, k_stride, v_stride, at,
          k_pages.data_ptr(), v_pages.data_ptr(), n_pages, page_tokens, page_stride, pos or None, table or None, rot,
          1 if interleaved else 0, mscale)


def q8kv_read_paged(k_pages, v_pages, slots, dtype=torch.float16, out=None):
    """The rows at `slots` (int64 [T]) dequantised: (k, v), each [T, H_kv, D] of dtype.  `out`: a pair of
    such tensors to write into; a negative slot leaves its row there as it was."""
    device = _device_of(slots)
    n_pages, kv_heads, page_tokens, head_dim, page_stride = _pool(k_pages, v_pages, device)
    T = slots.shape[0] if slots.dim() == 1 else -1
    at = _index("slots", slots, torch.int64, T, device)
    code = _DTYPES.get(dtype)
    if code is None:
        _refuse(f"dtype {dtype} is not supported")
    shape = (T, kv_heads, head_dim)
    if out is None:
        k = torch.empty(shape, dtype=dtype, device=slots.device)
        v = torch.empty(shape, dtype=dtype, device=slots.device)
        out = (k, v)
    else:
        k, v = out
        for t in (k, v):
            if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.get_device() == device and
                    t.shape == shape and t.is_contiguous()):
                _refuse(f"out: two contiguous tensors {shape} of {dtype} on cuda:{device} are needed")
    _call(load().q8kv_read_paged, device, k_pages.data_ptr(), v_pages.data_ptr(), n_pages, page_tokens, page_stride, at,
          T, kv_heads, head_dim, k.data_ptr(), v.data_ptr(), code)
    return out


@functools.lru_cache(maxsize=1024)
def paged_workspace_floats(batch, total_q, heads, kv_heads, max_q, max_kv, head_dim=HEAD_DIM):
    """Floats of attn_paged's workspace for these bounds."""
    n = int(load().q8a_paged_workspace_floats(batch, total_q, heads, kv_heads, max_q, max_kv, head_dim))
    if n < 0:
        raise Q8AttnError(Q8A_ERR_INVALID_ARG, "invalid sizes for the paged workspace")
    return n


def attn_paged(q, k_pages, v_pages, block_table, kv_lens, cu_q, max_q, max_kv, scale=None, causal=True, out=None,
               workspace=None):
    """Attention of packed new tokens q [total_q, H, D] (fp16 or bf16) over the pages of their sequences,
    one token to whole prompts a sequence: sequence b has the rows cu_q[b] .. cu_q[b + 1] - 1 (int32 [B + 1])
    and kv_lens[b] keys (int32 [B], the new tokens' own keys last) in the pages block_table[b] (int32
    [B, width]).  max_q, max_kv: bounds of the rows and keys of a sequence.  `workspace`: fp32 CUDA tensor
    of paged_workspace_floats(...) elements (allocated here when None).  Returns [total_q, H, D]."""
    device = _device_of(q)
    code, T, H, D, stride = _packed("q", q, device)
    n_pages, kv_heads, page_tokens, head_dim, page_stride = _pool(k_pages, v_pages, device)
    if D != head_dim:
        _refuse(f"q has head_dim {D}, the pages {head_dim}")
    if not (isinstance(block_table, torch.Tensor) and block_table.dtype == torch.int32 and block_table.dim() == 2 and
            block_table.is_contiguous() and block_table.get_device() == device):
        _refuse(f"block_table: a contiguous int32 tensor [batch, width] on cuda:{device} is needed")
    B, width = block_table.shape
    lens = _index("kv_lens", kv_lens, torch.int32, B, device)
    cu = _index("cu_q", cu_q, torch.int32, B + 1, device)
    if out is None:
        out = torch.empty((T, H, D), dtype=q.dtype, device=q.device)
    elif not (isinstance(out, torch.Tensor) and out.dtype == q.dtype and out.get_device() == device and
              out.shape == q.shape and out.is_contiguous()):
        _refuse(f"out: a contiguous tensor {(T, H, D)} of {q.dtype} on cuda:{device} is needed")
    ws = floats = 0
    if workspace is None:
        floats = paged_workspace_floats(B, T, H, kv_heads, max_q, max_kv, D)
        if floats:
            workspace = torch.empty(floats, dtype=torch.float32, device=q.device)
            ws = workspace.data_ptr()
    elif not (isinstance(workspace, torch.Tensor) and workspace.dtype == torch.float32 and
              workspace.get_device() == device and workspace.is_contiguous()):
        _refuse(f"workspace: a contiguous fp32 tensor on cuda:{device} is needed")
    else:
        ws, floats = workspace.data_ptr(), workspace.numel()
    _call(load().attn_paged, device, q.data_ptr(), code, stride, T, H, kv_heads, D, k_pages.data_ptr(),
          v_pages.data_ptr(), n_pages, page_tokens, page_stride, block_table.data_ptr(), width, lens, cu, B, max_q,
          max_kv, 1.0 / math.sqrt(D) if scale is None else scale, 1 if causal else 0, out.data_ptr(),
          ws, floats)
    return out


def device_status(clear=True, stream=None):
    """(rc, status bits) of the current device; synchronises the stream.  Bit 0: a device-side wait ran out
    (Q8A_ERR_TIMEOUT); bit 1: a paged call met an index out of range (alone Q8A_ERR_INVALID_ARG)."""
    st = ctypes.c_uint32(0)
    s = ctypes.c_void_p(stream.cuda_stream if stream is not None else torch.cuda.current_stream().cuda_stream)
    rc = load().q8a_device_status(s, ctypes.byref(st), 1 if clear else 0)
    return rc, st.value


def status(stream=None):
    """Return code of the sync-free status check (q8a_status): Q8A_OK, Q8A_ERR_TIMEOUT once a kernel of
    any device has recorded a run-out wait, or Q8A_ERR_INVALID_ARG once a paged call has met an index out
    of range."""
    s = ctypes.c_void_p(stream.cuda_stream if stream is not None else None)
    return load().q8a_status(s)


def set_wait_timeout_ns(ns):
    _check(load().q8a_set_wait_timeout_ns(int(ns)))


def test_inject(kind):
    _check(load().q8a_test_inject(int(kind)))
