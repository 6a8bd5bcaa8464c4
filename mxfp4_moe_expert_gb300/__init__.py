"""MXFP4 Mixture-of-Experts expert layer for GB300 (sm_103a).

Thin ctypes binding of the C ABI in include/moe_mxfp4.h: the functions below
carry the C names and only marshal arguments; every step of the layer runs in
the library's CUDA kernels.  PyTorch is used by callers for device memory and
streams only.  Importing this package does not load the library; the first
call does, and raises if the built library is missing (there is no fallback).
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libmoe_mxfp4.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_CUDA = -3
MOE_ERR_TIMEOUT = -4
MOE_ERR_BAD_SCALE = -5
MOE_ERR_WORKSPACE = -6
MOE_ERR_CACHE_FULL = -7
MOE_ERR_CACHE_STATE = -8

MOE_FLAG_NORM = 1 << 0
MOE_FLAG_OUT_BF16 = 1 << 1
MOE_FLAG_MULTI_KERNEL = 1 << 2
MOE_FLAG_NO_DENSE = 1 << 3
MOE_FLAG_DEBUG_STALL = 1 << 4
MOE_FLAG_TRACE = 1 << 5

MOE_DTYPE_BF16 = 0
MOE_DTYPE_FP16 = 1

EXPORTED = (
    "moe_mxfp4_create",
    "moe_mxfp4_workspace_bytes",
    "moe_mxfp4_forward",
    "moe_mxfp4_forward_host",
    "moe_mxfp4_check",
    "moe_mxfp4_destroy",
    "moe_mxfp4_status_string",
    "moe_mxfp4_quantize",
    "moe_mxfp4_forward_static",
    "moe_mxfp4_accept",
    "moe_mxfp4_packed_bytes",
    "moe_mxfp4_pack",
    "moe_mxfp4_split_terms",
    "moe_mxfp4_cache_create",
    "moe_mxfp4_cache_destroy",
    "moe_mxfp4_cache_state_bytes",
    "moe_mxfp4_cache_reserve",
    "moe_mxfp4_cache_append",
    "moe_mxfp4_cache_truncate",
    "moe_mxfp4_cache_commit",
    "moe_mxfp4_cache_fork",
    "moe_mxfp4_cache_compact",
    "moe_mxfp4_cache_attend_bytes",
    "moe_mxfp4_cache_attend",
    "moe_mxfp4_cache_check",
)

MOE_MXFP4_STATIC_WORKSPACE_BYTES = 16 << 20


class moe_mxfp4_config(ctypes.Structure):
    _fields_ = [
        ("num_layers", ctypes.c_int32),
        ("hidden", ctypes.c_int32),
        ("inter", ctypes.c_int32),
        ("num_experts", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("max_tokens", ctypes.c_int32),
        ("rms_eps", ctypes.c_float),
        ("flags", ctypes.c_uint32),
        ("expert_begin", ctypes.c_int32),
        ("expert_end", ctypes.c_int32),
        ("timeout_us", ctypes.c_int32),
    ]


class moe_mxfp4_layer(ctypes.Structure):
    _fields_ = [
        ("router_w_dev", ctypes.c_void_p),
        ("router_b_dev", ctypes.c_void_p),
        ("gate_q_dev", ctypes.c_void_p),
        ("gate_s_dev", ctypes.c_void_p),
        ("up_q_dev", ctypes.c_void_p),
        ("up_s_dev", ctypes.c_void_p),
        ("down_q_dev", ctypes.c_void_p),
        ("down_s_dev", ctypes.c_void_p),
        ("norm_w_dev", ctypes.c_void_p),
        ("packed_dev", ctypes.c_void_p),
    ]


class moe_mxfp4_debug(ctypes.Structure):
    _fields_ = [
        ("topk_idx_dev", ctypes.c_void_p),
        ("topk_gate_dev", ctypes.c_void_p),
        ("expert_counts_dev", ctypes.c_void_p),
        ("expert_offsets_dev", ctypes.c_void_p),
        ("perm_dev", ctypes.c_void_p),
        ("expert_events", ctypes.c_void_p),
    ]


class moe_mxfp4_cache_config(ctypes.Structure):
    _fields_ = [
        ("num_layers", ctypes.c_int32),
        ("num_streams", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("page_tokens", ctypes.c_int32),
        ("kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("page_stride", ctypes.c_int64),
        ("timeout_us", ctypes.c_int32),
    ]


class moe_mxfp4_cache_layer(ctypes.Structure):
    _fields_ = [("k_dev", ctypes.c_void_p), ("v_dev", ctypes.c_void_p)]


class moe_mxfp4_attend_args(ctypes.Structure):
    _fields_ = [
        ("q_dev", ctypes.c_void_p),
        ("q_stride", ctypes.c_int64),
        ("out_dev", ctypes.c_void_p),
        ("lse_dev", ctypes.c_void_p),
        ("lengths_dev", ctypes.c_void_p),
        ("mask_dev", ctypes.c_void_p),
        ("streams", ctypes.c_int32),
        ("block", ctypes.c_int32),
        ("q_heads", ctypes.c_int32),
        ("shared_stream", ctypes.c_int32),
        ("shared_tokens", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


_lib = None


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Loads the shared library (once) and declares the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m mxfp4_moe_expert_gb300.build`")
    lib = ctypes.CDLL(path)
    P = ctypes.c_void_p
    lib.moe_mxfp4_create.argtypes = [ctypes.POINTER(moe_mxfp4_config), ctypes.POINTER(moe_mxfp4_layer),
                                     ctypes.POINTER(P)]
    lib.moe_mxfp4_create.restype = ctypes.c_int
    lib.moe_mxfp4_workspace_bytes.argtypes = [P, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]
    lib.moe_mxfp4_workspace_bytes.restype = ctypes.c_int
    lib.moe_mxfp4_forward.argtypes = [P, P, ctypes.c_int32, P, P, ctypes.c_size_t, P,
                                      ctypes.POINTER(moe_mxfp4_debug)]
    lib.moe_mxfp4_forward.restype = ctypes.c_int
    lib.moe_mxfp4_forward_host.argtypes = [P, P, ctypes.c_int32, P, P, ctypes.c_size_t, P]
    lib.moe_mxfp4_forward_host.restype = ctypes.c_int
    lib.moe_mxfp4_check.argtypes = [P, P, P]
    lib.moe_mxfp4_check.restype = ctypes.c_int
    lib.moe_mxfp4_destroy.argtypes = [P]
    lib.moe_mxfp4_destroy.restype = None
    lib.moe_mxfp4_status_string.argtypes = [ctypes.c_int]
    lib.moe_mxfp4_status_string.restype = ctypes.c_char_p
    lib.moe_mxfp4_quantize.argtypes = [P, ctypes.c_int64, ctypes.c_int64, P, P, P]
    lib.moe_mxfp4_quantize.restype = ctypes.c_int
    lib.moe_mxfp4_forward_static.argtypes = [P, P, ctypes.c_int32, P, P]
    lib.moe_mxfp4_forward_static.restype = ctypes.c_int
    lib.moe_mxfp4_accept.argtypes = [P, P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int64, P, P, P, P]
    lib.moe_mxfp4_accept.restype = ctypes.c_int
    lib.moe_mxfp4_packed_bytes.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                           ctypes.POINTER(ctypes.c_size_t)]
    lib.moe_mxfp4_packed_bytes.restype = ctypes.c_int
    lib.moe_mxfp4_pack.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(moe_mxfp4_layer),
                                   P, ctypes.c_size_t, P]
    lib.moe_mxfp4_pack.restype = ctypes.c_int
    lib.moe_mxfp4_split_terms.argtypes = [P, ctypes.c_int64, P, P, P]
    lib.moe_mxfp4_split_terms.restype = ctypes.c_int
    I32, I64, SIZE = ctypes.c_int32, ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)
    for name, args in (
            ("create", [ctypes.POINTER(moe_mxfp4_cache_config), ctypes.POINTER(moe_mxfp4_cache_layer), ctypes.POINTER(P)]),
            ("state_bytes", [P, SIZE]),
            ("reserve", [P, P, P, I32, P]),
            ("append", [P, P, I32, P, P, I64, I32, I32, P, P]),
            ("truncate", [P, P, P, P]),
            ("commit", [P, P, P, P]),
            ("fork", [P, P, P, P, I32, P]),
            ("compact", [P, P, P]),
            ("attend_bytes", [P, I32, I32, I32, SIZE]),
            ("attend", [P, P, I32, ctypes.POINTER(moe_mxfp4_attend_args), P, ctypes.c_size_t, P]),
            ("check", [P, P, P])):
        fn = getattr(lib, "moe_mxfp4_cache_" + name)
        fn.argtypes, fn.restype = args, ctypes.c_int
    lib.moe_mxfp4_cache_destroy.argtypes = [P]
    lib.moe_mxfp4_cache_destroy.restype = None
    _lib = lib
    return lib


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {moe_mxfp4_status_string(status)} ({status})")


def _check(status: int, what: str) -> int:
    if status != MOE_OK:
        raise MoeError(status, what)
    return status


# ----------------------------------------------------------------------------- C entry points


def moe_mxfp4_status_string(status: int) -> str:
    return load_library().moe_mxfp4_status_string(int(status)).decode()


def moe_mxfp4_create(cfg: moe_mxfp4_config, layers) -> tuple[int, int]:
    """Returns (status, handle).  layers: a sequence of moe_mxfp4_layer."""
    arr = (moe_mxfp4_layer * len(layers))(*layers)
    out = ctypes.c_void_p()
    st = load_library().moe_mxfp4_create(ctypes.byref(cfg), arr, ctypes.byref(out))
    return st, out.value


def moe_mxfp4_workspace_bytes(handle: int, num_tokens: int) -> tuple[int, int]:
    n = ctypes.c_size_t()
    st = load_library().moe_mxfp4_workspace_bytes(handle, num_tokens, ctypes.byref(n))
    return st, n.value


def moe_mxfp4_forward(handle, x_ptr, num_tokens, y_ptr, ws_ptr, ws_bytes, stream_ptr, dbg=None) -> int:
    return load_library().moe_mxfp4_forward(handle, x_ptr, num_tokens, y_ptr, ws_ptr, ws_bytes, stream_ptr,
                                            ctypes.byref(dbg) if dbg is not None else None)


def moe_mxfp4_forward_host(handle, x_host_ptr, num_tokens, y_host_ptr, ws_ptr, ws_bytes, stream_ptr) -> int:
    return load_library().moe_mxfp4_forward_host(handle, x_host_ptr, num_tokens, y_host_ptr, ws_ptr, ws_bytes,
                                                 stream_ptr)


def moe_mxfp4_check(handle, ws_ptr, stream_ptr) -> int:
    return load_library().moe_mxfp4_check(handle, ws_ptr, stream_ptr)


def moe_mxfp4_destroy(handle) -> None:
    if handle:
        load_library().moe_mxfp4_destroy(handle)


def moe_mxfp4_quantize(w_ptr, rows, cols, q_ptr, s_ptr, stream_ptr) -> int:
    return load_library().moe_mxfp4_quantize(w_ptr, rows, cols, q_ptr, s_ptr, stream_ptr)


def moe_mxfp4_forward_static(handle, x_ptr, num_tokens, y_ptr, stream_ptr) -> int:
    """Forward with the library's own static workspace (no device allocation
    anywhere); synchronises the stream and returns the device status."""
    return load_library().moe_mxfp4_forward_static(handle, x_ptr, num_tokens, y_ptr, stream_ptr)


def moe_mxfp4_packed_bytes(hidden, inter, num_experts) -> tuple[int, int]:
    n = ctypes.c_size_t()
    st = load_library().moe_mxfp4_packed_bytes(hidden, inter, num_experts, ctypes.byref(n))
    return st, n.value


def moe_mxfp4_pack(hidden, inter, num_experts, layer: moe_mxfp4_layer, packed_ptr, packed_bytes, stream_ptr) -> int:
    return load_library().moe_mxfp4_pack(hidden, inter, num_experts, ctypes.byref(layer), packed_ptr, packed_bytes,
                                         stream_ptr)


def moe_mxfp4_split_terms(x_ptr, n_blocks, codes_ptr, scales_ptr, stream_ptr) -> int:
    return load_library().moe_mxfp4_split_terms(x_ptr, n_blocks, codes_ptr, scales_ptr, stream_ptr)


def moe_mxfp4_cache_create(cfg: moe_mxfp4_cache_config, layers) -> tuple[int, int]:
    """Returns (status, handle).  layers: a sequence of moe_mxfp4_cache_layer."""
    arr = (moe_mxfp4_cache_layer * len(layers))(*layers)
    out = ctypes.c_void_p()
    st = load_library().moe_mxfp4_cache_create(ctypes.byref(cfg), arr, ctypes.byref(out))
    return st, out.value


def moe_mxfp4_cache_destroy(cache) -> None:
    if cache:
        load_library().moe_mxfp4_cache_destroy(cache)


def moe_mxfp4_cache_state_bytes(cache) -> tuple[int, int]:
    n = ctypes.c_size_t()
    st = load_library().moe_mxfp4_cache_state_bytes(cache, ctypes.byref(n))
    return st, n.value


def moe_mxfp4_cache_reserve(cache, state_ptr, add_ptr, add, stream_ptr) -> int:
    return load_library().moe_mxfp4_cache_reserve(cache, state_ptr, add_ptr, add, stream_ptr)


def moe_mxfp4_cache_append(cache, state_ptr, layer, k_ptr, v_ptr, row_stride, streams, block, lengths_ptr,
                           stream_ptr) -> int:
    return load_library().moe_mxfp4_cache_append(cache, state_ptr, layer, k_ptr, v_ptr, row_stride, streams, block,
                                                 lengths_ptr, stream_ptr)


def moe_mxfp4_cache_truncate(cache, state_ptr, new_length_ptr, stream_ptr) -> int:
    return load_library().moe_mxfp4_cache_truncate(cache, state_ptr, new_length_ptr, stream_ptr)


def moe_mxfp4_cache_commit(cache, state_ptr, accepted_ptr, stream_ptr) -> int:
    return load_library().moe_mxfp4_cache_commit(cache, state_ptr, accepted_ptr, stream_ptr)


def moe_mxfp4_cache_fork(cache, state_ptr, src_ptr, dst_ptr, n, stream_ptr) -> int:
    return load_library().moe_mxfp4_cache_fork(cache, state_ptr, src_ptr, dst_ptr, n, stream_ptr)


def moe_mxfp4_cache_compact(cache, state_ptr, stream_ptr) -> int:
    return load_library().moe_mxfp4_cache_compact(cache, state_ptr, stream_ptr)


def moe_mxfp4_cache_attend_bytes(cache, streams, block, q_heads) -> tuple[int, int]:
    n = ctypes.c_size_t()
    st = load_library().moe_mxfp4_cache_attend_bytes(cache, streams, block, q_heads, ctypes.byref(n))
    return st, n.value


def moe_mxfp4_cache_attend(cache, state_ptr, layer, args: moe_mxfp4_attend_args, ws_ptr, ws_bytes, stream_ptr) -> int:
    return load_library().moe_mxfp4_cache_attend(cache, state_ptr, layer, ctypes.byref(args), ws_ptr, ws_bytes, stream_ptr)


def moe_mxfp4_cache_check(cache, state_ptr, stream_ptr) -> int:
    return load_library().moe_mxfp4_cache_check(cache, state_ptr, stream_ptr)


# ----------------------------------------------------------------------------- torch convenience


def _layer_desc(L) -> moe_mxfp4_layer:
    def p(name):
        t = L.get(name)
        return t.data_ptr() if t is not None else None
    return moe_mxfp4_layer(p("router_w"), p("router_b"), p("gate_q"), p("gate_s"), p("up_q"), p("up_s"),
                           p("down_q"), p("down_s"), p("norm_w"), p("packed"))


def pack(layer: dict, hidden: int, inter: int, num_experts: int, stream=None):
    """The packed (tile-major) copy of one layer's experts (moe_mxfp4_pack) as a new uint8
    CUDA tensor; `layer` holds the canonical gate_q .. down_s tensors."""
    import torch
    dev = layer["gate_q"].device
    st_, n = moe_mxfp4_packed_bytes(hidden, inter, num_experts)
    _check(st_, "moe_mxfp4_packed_bytes")
    out = torch.empty(n + 256, dtype=torch.uint8, device=dev)
    off = (-out.data_ptr()) % 256                     # 256-byte aligned view
    out = out[off:off + n]
    st = stream if stream is not None else torch.cuda.current_stream(dev).cuda_stream
    canon = {k: v for k, v in layer.items() if k != "packed"}
    _check(moe_mxfp4_pack(hidden, inter, num_experts, _layer_desc(canon), out.data_ptr(), n, st), "moe_mxfp4_pack")
    return out


def moe_mxfp4_accept(logits_ptr, tokens_ptr, num_streams, block, vocab, target_ptr, accepted_ptr,
                     next_token_ptr, stream_ptr) -> int:
    return load_library().moe_mxfp4_accept(logits_ptr, tokens_ptr, num_streams, block, vocab, target_ptr,
                                           accepted_ptr, next_token_ptr, stream_ptr)


def accept(logits, tokens, stream=None):
    """logits: fp32 CUDA [S, B, V]; tokens: int32 CUDA [S, B].  Returns (target [S, B],
    accepted [S], next_token [S]) as int32 CUDA tensors (see moe_mxfp4_accept)."""
    import torch
    S, B, V = logits.shape
    target = torch.empty((S, B), dtype=torch.int32, device=logits.device)
    acc = torch.empty((S,), dtype=torch.int32, device=logits.device)
    nxt = torch.empty((S,), dtype=torch.int32, device=logits.device)
    st = stream if stream is not None else torch.cuda.current_stream(logits.device).cuda_stream
    _check(moe_mxfp4_accept(logits.data_ptr(), tokens.data_ptr(), S, B, V, target.data_ptr(), acc.data_ptr(),
                            nxt.data_ptr(), st), "moe_mxfp4_accept")
    return target, acc, nxt


def split_terms(x, stream=None):
    """x: fp32 CUDA [n, 32] blocks.  Returns (codes uint32 [n, 32], scales uint8 [n, 8])."""
    import torch
    n = x.shape[0]
    codes = torch.empty((n, 32), dtype=torch.int32, device=x.device)
    scales = torch.empty((n, 8), dtype=torch.uint8, device=x.device)
    st = stream if stream is not None else torch.cuda.current_stream(x.device).cuda_stream
    _check(moe_mxfp4_split_terms(x.data_ptr(), n, codes.data_ptr(), scales.data_ptr(), st), "moe_mxfp4_split_terms")
    return codes, scales


def quantize(w, q=None, s=None, stream=None):
    """MXFP4-encodes an fp32 CUDA tensor [rows, cols] with the library kernel."""
    import torch
    assert w.is_cuda and w.dtype == torch.float32 and w.dim() == 2 and w.is_contiguous()
    rows, cols = w.shape
    q = q if q is not None else torch.empty((rows, cols // 2), dtype=torch.uint8, device=w.device)
    s = s if s is not None else torch.empty((rows, cols // 32), dtype=torch.uint8, device=w.device)
    st = stream if stream is not None else torch.cuda.current_stream(w.device).cuda_stream
    _check(moe_mxfp4_quantize(w.data_ptr(), rows, cols, q.data_ptr(), s.data_ptr(), st), "moe_mxfp4_quantize")
    return q, s


class MoeLayers:
    """Owns a handle over caller-provided device tensors (kept alive here).

    layers: list of dicts with router_w (bf16 [E,H]), router_b (fp32 [E] or None),
    gate_q/gate_s/up_q/up_s/down_q/down_s (uint8), norm_w (bf16 [H] or None) and
    optionally packed (the layer's experts in the packed layout, see pack()).
    """

    def __init__(self, *, hidden, inter, num_experts, top_k, max_tokens, layers, flags=0, rms_eps=1e-6,
                 expert_begin=0, expert_end=0, timeout_us=0):
        self._keep = layers
        self.cfg = moe_mxfp4_config(len(layers), hidden, inter, num_experts, top_k, max_tokens, rms_eps, flags,
                                    expert_begin, expert_end, timeout_us)
        descs = [_layer_desc(L) for L in layers]
        self.handle = None
        st, h = moe_mxfp4_create(self.cfg, descs)
        _check(st, "moe_mxfp4_create")
        self.handle = h
        self.hidden, self.top_k, self.num_experts = hidden, top_k, num_experts
        self.num_layers = len(layers)
        self.out_bf16 = bool(flags & MOE_FLAG_OUT_BF16)

    def workspace_bytes(self, num_tokens: int) -> int:
        st, n = moe_mxfp4_workspace_bytes(self.handle, num_tokens)
        _check(st, "moe_mxfp4_workspace_bytes")
        return n

    def new_workspace(self, num_tokens: int, device="cuda"):
        import torch
        return torch.empty(self.workspace_bytes(num_tokens), dtype=torch.uint8, device=device)

    def _own_workspace(self, num_tokens: int, device):
        """The workspace forward() uses when the caller passes none: one per device, kept
        here and grown when a larger block needs more (a workspace carries the persistent
        forward's state section from one forward to the next, so it is not re-allocated)."""
        cache = self.__dict__.setdefault("_ws", {})
        key = str(device)
        need = self.workspace_bytes(num_tokens)
        ws = cache.get(key)
        if ws is None or ws.numel() < need:
            ws = cache[key] = self.new_workspace(num_tokens, device)
        return ws

    def debug_buffers(self, num_tokens: int, device="cuda"):
        import torch
        L, T, k, E = self.num_layers, num_tokens, self.top_k, self.num_experts
        i32 = dict(dtype=torch.int32, device=device)
        bufs = dict(topk_idx=torch.full((L, T, k), -1, **i32),
                    topk_gate=torch.zeros((L, T, k), dtype=torch.float32, device=device),
                    expert_counts=torch.zeros((L, E), **i32), expert_offsets=torch.zeros((L, E + 1), **i32),
                    perm=torch.full((L, T * k), -1, **i32))
        dbg = moe_mxfp4_debug(*(bufs[n].data_ptr() for n in
                                ("topk_idx", "topk_gate", "expert_counts", "expert_offsets", "perm")), None)
        return bufs, dbg

    def expert_timing(self, events):
        """A debug descriptor that only records `events` (2 per layer, torch.cuda.Event
        created with enable_timing) around each layer's expert kernel."""
        arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
        dbg = moe_mxfp4_debug(None, None, None, None, None, ctypes.cast(arr, ctypes.c_void_p))
        dbg._events_keepalive = arr
        return dbg

    def forward(self, x, y=None, workspace=None, stream=None, dbg=None, check=False):
        """x: bf16 CUDA [T, H].  Returns y (fp32, or bf16 with MOE_FLAG_OUT_BF16)."""
        import torch
        T = x.shape[0]
        if y is None:
            y = torch.empty((T, self.hidden), dtype=torch.bfloat16 if self.out_bf16 else torch.float32,
                            device=x.device)
        if workspace is None:
            workspace = self._own_workspace(T, x.device)
        st = stream if stream is not None else torch.cuda.current_stream(x.device).cuda_stream
        _check(moe_mxfp4_forward(self.handle, x.data_ptr(), T, y.data_ptr(), workspace.data_ptr(),
                                 workspace.numel(), st, dbg), "moe_mxfp4_forward")
        if check:
            _check(moe_mxfp4_check(self.handle, workspace.data_ptr(), st), "moe_mxfp4_check")
        return y

    def forward_host(self, x_host, y_host, workspace, stream=None):
        import torch
        st = stream if stream is not None else torch.cuda.current_stream().cuda_stream
        return _check(moe_mxfp4_forward_host(self.handle, x_host.data_ptr(), x_host.shape[0], y_host.data_ptr(),
                                             workspace.data_ptr(), workspace.numel(), st), "moe_mxfp4_forward_host")

    def close(self):
        if getattr(self, "handle", None):
            moe_mxfp4_destroy(self.handle)
            self.handle = None
        self.__dict__.pop("_ws", None)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class KvCache:
    """The paged key/value cache of a verify forward (moe_mxfp4.h, "paged key/value cache").

    layers: a list of (k, v) pool tensors [num_pages, kv_heads, page_tokens, head_dim], bf16 or fp16 on one CUDA
    device, contiguous within a page (all with the same stride between pages, which share no memory); kept alive here.
    The books are views of one int32 tensor: length [S], held [S], page_table [S, max_pages], refcount [num_pages]; they
    are zeroed on the stream that is current when the cache is made.  Every call runs on `stream` (a cudaStream_t as int;
    default: torch's current stream on the cache's device), and what it makes belongs to that stream; device-side errors
    are raised by check().
    """

    def __init__(self, *, layers, num_streams, max_pages, timeout_us=0):
        import torch
        self.handle = None
        if not layers:
            raise ValueError("layers: at least one (k, v) pair")
        k0 = layers[0][0]
        if not k0.is_cuda or k0.dim() != 4 or k0.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("a pool is a bf16 or fp16 CUDA tensor [num_pages, kv_heads, page_tokens, head_dim]")
        pages, heads, tokens, dim = k0.shape
        for pool in (p for kv in layers for p in kv):
            if (pool.shape != k0.shape or pool.dtype != k0.dtype or pool.device != k0.device
                    or pool.stride()[1:] != (tokens * dim, dim, 1) or (pages > 1 and pool.stride(0) != k0.stride(0))):
                raise ValueError("the pools of a cache have one shape, type, device and page stride")
        if pages > 1 and k0.stride(0) < heads * tokens * dim:
            raise ValueError("the pages of a pool do not share memory")
        self._keep = [tuple(kv) for kv in layers]
        self.device, self.dtype = k0.device, k0.dtype      # (a tensor's device has its index)
        self.num_layers, self.num_streams, self.max_pages = len(layers), num_streams, max_pages
        self.num_pages, self.kv_heads, self.page_tokens, self.head_dim = pages, heads, tokens, dim
        cfg = moe_mxfp4_cache_config(len(layers), num_streams, max_pages, pages, tokens, heads, dim,
                                     MOE_DTYPE_BF16 if k0.dtype == torch.bfloat16 else MOE_DTYPE_FP16,
                                     k0.stride(0) if pages > 1 else 0, timeout_us)
        with torch.cuda.device(self.device):
            st, self.handle = moe_mxfp4_cache_create(
                cfg, [moe_mxfp4_cache_layer(k.data_ptr(), v.data_ptr()) for k, v in layers])
        _check(st, "moe_mxfp4_cache_create")
        st, n = moe_mxfp4_cache_state_bytes(self.handle)
        _check(st, "moe_mxfp4_cache_state_bytes")
        self.state = torch.zeros(n // 4, dtype=torch.int32, device=self.device)
        self._state_ptr = self.state.data_ptr()
        S, at = num_streams, 16
        self.length, at = self.state[at:at + S], at + S
        self.held, at = self.state[at:at + S], at + S
        self.page_table, at = self.state[at:at + S * max_pages].view(S, max_pages), at + S * max_pages
        self.refcount = self.state[at:at + pages]
        self._lib = load_library()
        self._index, self._append = k0.get_device(), self._lib.moe_mxfp4_cache_append
        self._ws, self._ws_bytes, self._ws_kept = None, {}, []
        self._layouts, self._pairs = {}, {}     # shapes and strides seen so far -> how a call lays them out
        self._i32, self._f32, self._u8, self._mask_types = torch.int32, torch.float32, torch.uint8, (torch.int64, torch.uint64)
        # the raw handle of the current stream (torch.cuda.current_stream() builds a Stream object around it)
        self._current_stream = torch._C._cuda_getCurrentRawStream

    # -- the books

    def reserve(self, tokens, stream=None):
        """Room for `tokens` more tokens: an int (in every stream) or an int32 tensor [num_streams]."""
        if type(tokens) is int or not hasattr(tokens, "data_ptr"):
            tokens = int(tokens)
            if not -(1 << 31) <= tokens < 1 << 31:
                raise ValueError("tokens: a 32-bit count")
            add, n = None, tokens
        else:
            add, n = self._books("tokens", tokens, self.num_streams), 0
        st = self._lib.moe_mxfp4_cache_reserve(self.handle, self._state_ptr, add, n, self._stream(stream))
        if st:
            _check(st, "moe_mxfp4_cache_reserve")

    def commit(self, accepted, stream=None):
        """length += accepted (int32 [num_streams]); the pages behind are given back.  accept()'s output has a value for
        each stream of the batch: slots that are not in it need one too (0: what was reserved there is given back,
        negative: left alone)."""
        _check(self._lib.moe_mxfp4_cache_commit(self.handle, self._state_ptr,
                                                self._books("accepted", accepted, self.num_streams), self._stream(stream)),
               "moe_mxfp4_cache_commit")

    def truncate(self, new_length, stream=None):
        """length = new_length (int32 [num_streams]; negative: left alone); the pages behind are given back."""
        _check(self._lib.moe_mxfp4_cache_truncate(self.handle, self._state_ptr,
                                                  self._books("new_length", new_length, self.num_streams),
                                                  self._stream(stream)), "moe_mxfp4_cache_truncate")

    def fork(self, src, dst, stream=None):
        """The empty streams dst[i] get the tokens of src[i], holding the same pages (int32 tensors of one length)."""
        if src.numel() != dst.numel():
            raise ValueError("src and dst have one length")
        n = src.numel()
        _check(self._lib.moe_mxfp4_cache_fork(self.handle, self._state_ptr, self._books("src", src, n),
                                              self._books("dst", dst, n), n, self._stream(stream)), "moe_mxfp4_cache_fork")

    def compact(self, stream=None):
        """Moves the pages in use to the front of the pool."""
        _check(self._lib.moe_mxfp4_cache_compact(self.handle, self._state_ptr, self._stream(stream)),
               "moe_mxfp4_cache_compact")

    def check(self, stream=None):
        """Waits for the stream; raises MoeError for the first error the device recorded, and clears it."""
        _check(self._lib.moe_mxfp4_cache_check(self.handle, self._state_ptr, self._stream(stream)), "moe_mxfp4_cache_check")

    # -- a layer's keys and values

    def append(self, layer, k, v, lengths=None, stream=None):
        """k, v: [streams, block, kv_heads, head_dim], contiguous or rows of one wider tensor (a fused projection's
        output), each token in memory of its own (an expanded tensor is refused); lengths: int32 [streams], tokens in use of each block."""
        layout = self._pairs.get((k.shape, k.stride(), v.shape, v.stride()))
        if (layout is None or k.dtype is not self.dtype or v.dtype is not self.dtype or k.get_device() != self._index
                or v.get_device() != self._index):
            layout = self._pair(k, v)
        S, B, row = layout
        st = self._append(self.handle, self._state_ptr, layer, k.data_ptr(), v.data_ptr(), row, S, B,
                          None if lengths is None else self._books("lengths", lengths, S),
                          self._current_stream(self._index) if stream is None else stream)
        if st:
            _check(st, "moe_mxfp4_cache_append")

    def attend(self, layer, q, lengths=None, mask=None, shared_stream=0, shared_tokens=0, scale=None, out=None, lse=None,
               workspace=None, stream=None):
        """Attention of a block (moe_mxfp4_cache_attend).  q: [streams, block, q_heads, head_dim], as k in append; mask:
        int64 [streams, block], bit i = sees block position i (default: causal); scale: default 1 / sqrt(head_dim).
        Returns (out, lse): out like q, contiguous; lse fp32 [streams, block, q_heads].  Rows that `lengths` leaves
        out are zero in an out (lse) that is made here and unchanged in one that is given.  Calls that may overlap on
        the GPU (on two streams) are given a `workspace` each (uint8, attend_bytes long, 256-byte aligned)."""
        S, B, H, D, row = self._rows("q", q)
        if D != self.head_dim:
            raise ValueError("q is [streams, block, q_heads, head_dim]")
        if stream is None:
            stream = self._current_stream(self._index)
        if out is None:
            out = self._new((S, B, H, D), self.dtype, stream, zero=lengths is not None)
        if lse is None:
            lse = self._new((S, B, H), self._f32, stream, zero=lengths is not None)
        if (out.shape != (S, B, H, D) or out.dtype is not self.dtype or out.get_device() != self._index
                or not out.is_contiguous()):
            raise ValueError("out: contiguous, of q's shape and type")
        if (lse.shape != (S, B, H) or lse.dtype is not self._f32 or lse.get_device() != self._index
                or not lse.is_contiguous()):
            raise ValueError("lse: contiguous fp32 [streams, block, q_heads]")
        if mask is not None and (mask.shape != (S, B) or mask.dtype not in self._mask_types
                                 or mask.get_device() != self._index or not mask.is_contiguous()):
            raise ValueError("mask: contiguous int64 [streams, block]")
        if workspace is None:
            ws, n = self._workspace(S, B, H, stream)
        elif workspace.get_device() != self._index or not workspace.is_contiguous():
            raise ValueError(f"workspace: contiguous, on {self.device}")
        else:
            ws, n = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        a = moe_mxfp4_attend_args(q.data_ptr(), row, out.data_ptr(), lse.data_ptr(),
                                  None if lengths is None else self._books("lengths", lengths, S),
                                  None if mask is None else mask.data_ptr(), S, B, H, shared_stream, shared_tokens,
                                  self.head_dim ** -0.5 if scale is None else scale)
        st = self._lib.moe_mxfp4_cache_attend(self.handle, self._state_ptr, layer, a, ws, n, stream)
        if st:
            _check(st, "moe_mxfp4_cache_attend")
        return out, lse

    def attend_bytes(self, streams, block, q_heads) -> int:
        st, n = moe_mxfp4_cache_attend_bytes(self.handle, streams, block, q_heads)
        _check(st, "moe_mxfp4_cache_attend_bytes")
        return n

    # -- arguments

    def _stream(self, stream):
        return self._current_stream(self._index) if stream is None else stream

    def _books(self, name, t, n):
        if t.dtype is not self._i32 or t.get_device() != self._index or t.numel() != n or not t.is_contiguous():
            raise ValueError(f"{name}: {n} contiguous int32 values on {self.device}")
        return t.data_ptr()

    def _pair(self, k, v):
        """(streams, block, elements between tokens) of new keys and values; remembered by shape and stride."""
        S, B, H, D, row = self._rows("k", k)
        if (H, D) != (self.kv_heads, self.head_dim) or self._rows("v", v)[:4] != (S, B, H, D):
            raise ValueError("k and v are [streams, block, kv_heads, head_dim]")
        if S * B > 1 and self._rows("v", v)[4] != row:
            raise ValueError("k and v have one stride between tokens")
        if len(self._pairs) >= 1024:
            self._pairs.clear()
        layout = self._pairs[(k.shape, k.stride(), v.shape, v.stride())] = (S, B, row)
        return layout

    def _rows(self, name, t):
        """(streams, block, heads, head_dim, elements between tokens) of a tensor of rows."""
        if t.dtype is not self.dtype or t.get_device() != self._index:
            raise ValueError(f"{name}: a 4-dimensional {self.dtype} tensor on {self.device}")
        key = (t.shape, t.stride())
        rows = self._layouts.get(key)
        if rows is None:
            if t.dim() != 4:
                raise ValueError(f"{name}: a 4-dimensional {self.dtype} tensor on {self.device}")
            (S, B, H, D), st = key
            if t.numel() and ((D > 1 and st[3] != 1) or (H > 1 and st[2] != D) or (S > 1 and B > 1 and st[0] != B * st[1])):
                raise ValueError(f"{name}: heads are contiguous, tokens one stride apart")
            row = st[1] if B > 1 else st[0] if S > 1 else H * D
            if t.numel() and row < H * D:      # (expanded ones have 0, which the library takes for contiguous rows)
                raise ValueError(f"{name}: tokens do not share memory")
            if len(self._layouts) >= 1024:
                self._layouts.clear()
            rows = self._layouts[key] = (S, B, H, D, row)
        return rows

    def _new(self, shape, dtype, stream, zero=False):
        """A tensor made on a call's stream: its fill is ordered with the call, and so is what still uses its memory."""
        import torch
        make = torch.zeros if zero else torch.empty
        if stream == self._current_stream(self._index):
            return make(shape, dtype=dtype, device=self.device)
        on = torch.cuda.ExternalStream(stream, self.device) if stream else torch.cuda.default_stream(self.device)
        with torch.cuda.stream(on):
            return make(shape, dtype=dtype, device=self.device)

    def _workspace(self, S, B, H, stream):
        """The cache's own workspace, at least doubled when a call needs more; earlier ones are kept, since captured
        graphs may hold their addresses (all together, at most four times what the largest call needs)."""
        key = (S, B, H)
        n = self._ws_bytes.get(key)
        if n is None:
            n = self._ws_bytes[key] = self.attend_bytes(S, B, H)
        ws = self._ws
        if ws is None or ws.numel() < n:
            n = max(n, 2 * ws.numel() if ws is not None else 0)
            raw = self._new(n + 256, self._u8, stream)
            off = (-raw.data_ptr()) % 256
            ws = self._ws = raw[off:off + n]
            self._ws_kept.append(ws)
        return ws.data_ptr(), ws.numel()

    def close(self):
        if getattr(self, "handle", None):
            moe_mxfp4_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
