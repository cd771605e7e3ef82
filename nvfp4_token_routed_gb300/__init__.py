"""nvfp4_token_routed_gb300 -- Python binding of libmoe_nvfp4.so.

A single-GPU routed mixture-of-experts expert layer in NVFP4 for GB300
(sm_103a).  Every stage runs in the library's own CUDA kernels; this module
only marshals torch tensors (device memory + the current stream) into the C
ABI declared in include/moe_nvfp4.h.  The functions named moe_nvfp4_* mirror
the C entry points one to one; the lower-case helpers allocate buffers.

There is no CPU fallback: if the compiled library is missing, importing the
binding's entry points raises.
"""
import ctypes as C
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_nvfp4.so")

ACT = {"relu2": 0, "swiglu": 1}

STATUS = {
    0: "ok", 1: "invalid argument", 2: "unsupported shape", 3: "misaligned pointer",
    4: "workspace too small", 5: "unsupported device", 6: "CUDA error",
    7: "bad expert id", 8: "device wait timeout",
}


class MoeError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)} ({code})")


class moe_dims(C.Structure):
    _fields_ = [("E", C.c_int32), ("H", C.c_int32), ("I", C.c_int32), ("act", C.c_int32)]


class moe_nvfp4_weights(C.Structure):
    _fields_ = [("fc1_codes", C.c_void_p), ("fc1_sf", C.c_void_p), ("fc1_alpha", C.c_void_p),
                ("fc2_codes", C.c_void_p), ("fc2_sf", C.c_void_p), ("fc2_alpha", C.c_void_p)]


_LAYOUT_FIELDS = ["total", "rows_cap", "status", "counts", "group_row0", "tiles",
                  "chunk_counts", "chunk_prefix", "inv", "perm", "xq_codes", "xq_sf",
                  "xq_scale", "act", "fc2q_codes", "fc2q_sf", "fc2q_scale", "x_perm", "act_bf16",
                  "route", "tile_sync", "act_f16", "act_scale"]


class moe_forward_opts(C.Structure):
    _fields_ = [("ids_int64", C.c_int32), ("swiglu_limit", C.c_float)]


class moe_logits(C.Structure):
    _fields_ = [("data", C.c_void_p), ("ld", C.c_int64), ("rows", C.c_int32), ("cols", C.c_int32),
                ("dtype", C.c_int32)]


class moe_policy_opts(C.Structure):
    _fields_ = [("clip_low", C.c_float), ("clip_high", C.c_float), ("kl_coef", C.c_float),
                ("temperature", C.c_float)]


class moe_teacher(C.Structure):
    _fields_ = [("ids", C.c_void_p), ("logits", C.c_void_p), ("lse", C.c_void_p),
                ("K", C.c_int32), ("ids_int64", C.c_int32), ("dtype", C.c_int32)]


class moe_router_batch(C.Structure):
    _fields_ = [("logits", moe_logits), ("topk_ids", C.c_void_p), ("token_mask", C.c_void_p),
                ("seq_offsets", C.c_void_p), ("K", C.c_int32), ("S", C.c_int32),
                ("ids_int64", C.c_int32), ("balance_coef", C.c_float), ("z_coef", C.c_float)]


class moe_mx(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("rows", C.c_int32),
                ("cols", C.c_int32)]


class moe_ws_layout(C.Structure):
    _fields_ = [(n, C.c_int64 if n == "rows_cap" else C.c_size_t) for n in _LAYOUT_FIELDS]


_lib = None


def lib():
    """Load libmoe_nvfp4.so (built by nvfp4_token_routed_gb300.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run `python -m nvfp4_token_routed_gb300.build`")
        L = C.CDLL(LIB_PATH)
        vp, i32, sz = C.c_void_p, C.c_int32, C.c_size_t
        L.moe_nvfp4_abi_version.restype = i32
        L.moe_nvfp4_status_string.restype = C.c_char_p
        L.moe_nvfp4_status_string.argtypes = [C.c_int]
        L.moe_nvfp4_weight_sizes.argtypes = [C.POINTER(moe_dims), C.POINTER(C.c_size_t)]
        L.moe_nvfp4_prepare_weights.argtypes = [C.POINTER(moe_dims), vp, vp,
                                                C.POINTER(moe_nvfp4_weights), vp]
        L.moe_nvfp4_quantize_tokens.argtypes = [i32, i32, vp, vp, vp, vp, vp]
        L.moe_nvfp4_workspace_bytes.restype = sz
        L.moe_nvfp4_workspace_bytes.argtypes = [C.POINTER(moe_dims), i32, i32, i32]
        L.moe_nvfp4_forward_kernel_count.restype = i32
        L.moe_nvfp4_forward_kernel_count.argtypes = [C.POINTER(moe_dims), i32, i32, i32]
        L.moe_nvfp4_workspace_layout.argtypes = [C.POINTER(moe_dims), i32, i32, i32,
                                                 C.POINTER(moe_ws_layout)]
        L.moe_nvfp4_forward.argtypes = [C.POINTER(moe_dims), C.POINTER(moe_nvfp4_weights), i32,
                                        i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_nvfp4_forward_w4a16.argtypes = [C.POINTER(moe_dims), C.POINTER(moe_nvfp4_weights),
                                              i32, i32, vp, vp, vp, vp, vp, sz, vp]
        L.moe_nvfp4_read_status.argtypes = [vp, vp]
        L.moe_nvfp4_forward_noalloc.argtypes = [C.POINTER(moe_dims), C.POINTER(moe_nvfp4_weights),
                                                i32, i32, vp, vp, vp, vp, vp, vp, vp]
        L.moe_nvfp4_profile_events.argtypes = [C.POINTER(C.c_void_p), i32]
        L.moe_nvfp4_profile_spans.argtypes = [vp]
        L.moe_nvfp4_prepare_weights_per_tensor.argtypes = [
            C.POINTER(moe_dims), vp, vp, vp, vp, C.POINTER(moe_nvfp4_weights), vp]
        L.moe_nvfp4_quantize_tokens_static.argtypes = [i32, i32, vp, vp, vp, vp, vp]
        L.moe_nvfp4_forward_per_tensor.argtypes = [C.POINTER(moe_dims),
                                                   C.POINTER(moe_nvfp4_weights), i32, i32, vp, vp,
                                                   vp, vp, vp, vp, vp, sz, vp]
        L.moe_nvfp4_route_topk.argtypes = [i32, i32, i32, vp, vp, vp, vp]
        L.moe_nvfp4_selftest_wait_timeout.argtypes = [vp, sz, vp]
        L.moe_nvfp4_forward_ex.argtypes = [C.POINTER(moe_dims), C.POINTER(moe_nvfp4_weights), i32,
                                           i32, vp, vp, vp, vp, vp, vp, vp, sz,
                                           C.POINTER(moe_forward_opts), vp]
        L.moe_nvfp4_forward_w4a16_ex.argtypes = [C.POINTER(moe_dims),
                                                 C.POINTER(moe_nvfp4_weights), i32, i32, vp, vp,
                                                 vp, vp, vp, sz, C.POINTER(moe_forward_opts), vp]
        f32, i64, zp = C.c_float, C.c_int64, C.POINTER(moe_logits)
        po, tp, rb = C.POINTER(moe_policy_opts), C.POINTER(moe_teacher), C.POINTER(moe_router_batch)
        L.moe_nvfp4_token_logp.argtypes = [zp, vp, i32, f32, vp, vp]
        L.moe_nvfp4_policy_loss.argtypes = [zp, vp, i32, vp, vp, vp, po, vp, vp, vp]
        L.moe_nvfp4_policy_loss_grad.argtypes = [zp, vp, i32, vp, vp, vp, vp, po, vp, vp, vp, i64,
                                                 vp]
        L.moe_nvfp4_selftest_loss_timeout.argtypes = [zp, vp, i32, vp, vp, i32, i32, i32, vp, vp,
                                                      vp, i64, vp]
        L.moe_nvfp4_distill_loss.argtypes = [zp, tp, f32, vp, vp]
        L.moe_nvfp4_distill_loss_grad.argtypes = [zp, tp, vp, f32, vp, vp, i64, vp]
        L.moe_nvfp4_router_loss_workspace_bytes.restype = sz
        L.moe_nvfp4_router_loss_workspace_bytes.argtypes = [i32, i32, i32]
        L.moe_nvfp4_router_loss.argtypes = [rb, vp, vp, vp, vp, sz, vp]
        L.moe_nvfp4_router_loss_grad.argtypes = [rb, vp, vp, vp, vp, vp, vp, i64, vp]
        mp = C.POINTER(moe_mx)
        L.moe_nvfp4_sort_routes_workspace_bytes.restype = sz
        L.moe_nvfp4_sort_routes_workspace_bytes.argtypes = [i32, i32, i32]
        L.moe_nvfp4_sort_routes.argtypes = [i32, i32, i32, vp, i32, vp, vp, vp, vp, sz, vp]
        L.moe_nvfp4_dispatch.argtypes = [zp, i32, vp, vp, i64, vp]
        L.moe_nvfp4_combine.argtypes = [zp, i32, i32, vp, vp, vp, i64, vp]
        L.moe_nvfp4_combine_grad.argtypes = [zp, i32, i32, vp, vp, vp, i64, vp, i64, vp, vp]
        L.moe_nvfp4_checkpoint.argtypes = [zp, vp, vp, vp, vp]
        L.moe_nvfp4_restore.argtypes = [vp, vp, zp, vp, vp]
        L.moe_nvfp4_expert_act.argtypes = [zp, i32, f32, vp, i64, vp, vp, vp, vp]
        L.moe_nvfp4_expert_act_grad.argtypes = [vp, vp, i32, f32, zp, vp, i64, vp, vp]
        L.moe_nvfp4_mx_sizes.argtypes = [i32, i32, C.POINTER(sz)]
        L.moe_nvfp4_mx_quantize.argtypes = [zp, mp, vp, vp]
        L.moe_nvfp4_mx_quantize_transposed.argtypes = [i32, i32, i32, vp, i32, mp, vp]
        L.moe_nvfp4_mx_restore.argtypes = [mp, zp, vp, vp]
        L.moe_nvfp4_mx_dispatch.argtypes = [mp, i32, vp, mp, vp]
        L.moe_nvfp4_mx_product.argtypes = [mp, mp, i32, vp, i32, vp, i64, vp]
        L.moe_nvfp4_selftest_product_timeout.argtypes = [mp, mp, i32, vp, i32, i32, vp, i64, vp]
        for f in ["moe_nvfp4_sort_routes", "moe_nvfp4_dispatch", "moe_nvfp4_combine",
                  "moe_nvfp4_combine_grad", "moe_nvfp4_checkpoint", "moe_nvfp4_restore",
                  "moe_nvfp4_expert_act", "moe_nvfp4_expert_act_grad", "moe_nvfp4_mx_sizes",
                  "moe_nvfp4_mx_quantize", "moe_nvfp4_mx_quantize_transposed",
                  "moe_nvfp4_mx_restore", "moe_nvfp4_mx_dispatch", "moe_nvfp4_mx_product",
                  "moe_nvfp4_selftest_product_timeout",
                  "moe_nvfp4_token_logp", "moe_nvfp4_policy_loss", "moe_nvfp4_policy_loss_grad",
                  "moe_nvfp4_selftest_loss_timeout",
                  "moe_nvfp4_distill_loss", "moe_nvfp4_distill_loss_grad",
                  "moe_nvfp4_router_loss", "moe_nvfp4_router_loss_grad",
                  "moe_nvfp4_selftest_wait_timeout",
                  "moe_nvfp4_route_topk", "moe_nvfp4_forward_ex", "moe_nvfp4_forward_w4a16_ex",
                  "moe_nvfp4_prepare_weights_per_tensor", "moe_nvfp4_quantize_tokens_static",
                  "moe_nvfp4_forward_per_tensor",
                  "moe_nvfp4_weight_sizes", "moe_nvfp4_prepare_weights",
                  "moe_nvfp4_quantize_tokens", "moe_nvfp4_workspace_layout", "moe_nvfp4_forward",
                  "moe_nvfp4_forward_w4a16", "moe_nvfp4_read_status", "moe_nvfp4_profile_events",
                  "moe_nvfp4_profile_spans", "moe_nvfp4_forward_noalloc"]:
            getattr(L, f).restype = C.c_int
        _lib = L
        from . import experts
        experts._attach(L)
    return _lib


def _check(code, where):
    if code != 0:
        raise MoeError(code, where)


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors (no CPU path exists)")
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def padded(n):
    """The stored size of a hidden or intermediate dimension: n rounded up to 256."""
    return (n + 255) // 256 * 256


def dims(E, H, I, act):
    return moe_dims(E, H, I, ACT[act] if isinstance(act, str) else int(act))


# ------------------------------------------------------------------ one-to-one C entry points

def moe_nvfp4_abi_version():
    return lib().moe_nvfp4_abi_version()


def moe_nvfp4_status_string(code):
    return lib().moe_nvfp4_status_string(code).decode()


def moe_nvfp4_weight_sizes(d):
    out = (C.c_size_t * 6)()
    _check(lib().moe_nvfp4_weight_sizes(C.byref(d), out), "moe_nvfp4_weight_sizes")
    return list(out)


def moe_nvfp4_prepare_weights(d, fc1_bf16, fc2_bf16, w, stream=None):
    _need_cuda(fc1_bf16, fc2_bf16)
    _check(lib().moe_nvfp4_prepare_weights(C.byref(d), _ptr(fc1_bf16), _ptr(fc2_bf16),
                                           C.byref(w.c), _stream(stream)),
           "moe_nvfp4_prepare_weights")


def moe_nvfp4_quantize_tokens(x_bf16, codes, sf, scale, stream=None):
    _need_cuda(x_bf16, codes, sf, scale)
    T, H = x_bf16.shape
    _check(lib().moe_nvfp4_quantize_tokens(T, H, _ptr(x_bf16), _ptr(codes), _ptr(sf),
                                           _ptr(scale), _stream(stream)),
           "moe_nvfp4_quantize_tokens")


def moe_nvfp4_prepare_weights_per_tensor(d, fc1_bf16, fc2_bf16, a1_scale, a2_scale, w,
                                         stream=None):
    _need_cuda(fc1_bf16, fc2_bf16, a1_scale, a2_scale)
    _check(lib().moe_nvfp4_prepare_weights_per_tensor(
        C.byref(d), _ptr(fc1_bf16), _ptr(fc2_bf16), _ptr(a1_scale), _ptr(a2_scale), C.byref(w.c),
        _stream(stream)), "moe_nvfp4_prepare_weights_per_tensor")


def moe_nvfp4_quantize_tokens_static(x_bf16, a1_scale, codes, sf, stream=None):
    _need_cuda(x_bf16, a1_scale, codes, sf)
    T, H = x_bf16.shape
    _check(lib().moe_nvfp4_quantize_tokens_static(T, H, _ptr(x_bf16), _ptr(a1_scale), _ptr(codes),
                                                  _ptr(sf), _stream(stream)),
           "moe_nvfp4_quantize_tokens_static")


def moe_nvfp4_forward_per_tensor(d, w, codes, sf, a2_scale, topk_ids, topk_w, out, ws,
                                 stream=None):
    _need_cuda(codes, sf, a2_scale, topk_ids, topk_w, out, ws)
    T, K = topk_ids.shape
    _check(lib().moe_nvfp4_forward_per_tensor(C.byref(d), C.byref(w.c), T, K, _ptr(codes),
                                              _ptr(sf), _ptr(a2_scale), _ptr(topk_ids),
                                              _ptr(topk_w), _ptr(out), _ptr(ws),
                                              ws.numel() * ws.element_size(), _stream(stream)),
           "moe_nvfp4_forward_per_tensor")


def moe_nvfp4_selftest_wait_timeout(ws, stream=None):
    _need_cuda(ws)
    _check(lib().moe_nvfp4_selftest_wait_timeout(_ptr(ws), ws.numel() * ws.element_size(),
                                                 _stream(stream)),
           "moe_nvfp4_selftest_wait_timeout")


def moe_nvfp4_route_topk(logits, topk_ids, topk_w, stream=None):
    _need_cuda(logits, topk_ids, topk_w)
    T, E = logits.shape
    K = topk_ids.shape[1]
    _check(lib().moe_nvfp4_route_topk(T, E, K, _ptr(logits), _ptr(topk_ids), _ptr(topk_w),
                                      _stream(stream)), "moe_nvfp4_route_topk")


def moe_nvfp4_workspace_bytes(d, T_max, K, w4a16=False):
    return int(lib().moe_nvfp4_workspace_bytes(C.byref(d), T_max, K, int(bool(w4a16))))


def moe_nvfp4_forward_kernel_count(d, T, K, w4a16=False):
    return int(lib().moe_nvfp4_forward_kernel_count(C.byref(d), T, K, int(bool(w4a16))))


def moe_nvfp4_workspace_layout(d, T, K, w4a16=False):
    L = moe_ws_layout()
    _check(lib().moe_nvfp4_workspace_layout(C.byref(d), T, K, int(bool(w4a16)), C.byref(L)),
           "moe_nvfp4_workspace_layout")
    return {n: int(getattr(L, n)) for n in _LAYOUT_FIELDS}


def moe_nvfp4_forward(d, w, codes, sf, scale, topk_ids, topk_w, out, ws, stream=None):
    _need_cuda(codes, sf, scale, topk_ids, topk_w, out, ws)
    T, K = topk_ids.shape
    _check(lib().moe_nvfp4_forward(C.byref(d), C.byref(w.c), T, K, _ptr(codes), _ptr(sf),
                                   _ptr(scale), _ptr(topk_ids), _ptr(topk_w), _ptr(out), _ptr(ws),
                                   ws.numel() * ws.element_size(), _stream(stream)),
           "moe_nvfp4_forward")


def moe_nvfp4_forward_ex(d, w, codes, sf, scale, topk_ids, topk_w, out, ws, opts, stream=None):
    """opts: moe_forward_opts (int64 ids are taken from topk_ids' dtype)."""
    _need_cuda(codes, sf, scale, topk_ids, topk_w, out, ws)
    T, K = topk_ids.shape
    _check(lib().moe_nvfp4_forward_ex(C.byref(d), C.byref(w.c), T, K, _ptr(codes), _ptr(sf),
                                      _ptr(scale), _ptr(topk_ids), _ptr(topk_w), _ptr(out),
                                      _ptr(ws), ws.numel() * ws.element_size(), C.byref(opts),
                                      _stream(stream)), "moe_nvfp4_forward_ex")


def moe_nvfp4_forward_w4a16_ex(d, w, x_bf16, topk_ids, topk_w, out, ws, opts, stream=None):
    _need_cuda(x_bf16, topk_ids, topk_w, out, ws)
    T, K = topk_ids.shape
    _check(lib().moe_nvfp4_forward_w4a16_ex(C.byref(d), C.byref(w.c), T, K, _ptr(x_bf16),
                                            _ptr(topk_ids), _ptr(topk_w), _ptr(out), _ptr(ws),
                                            ws.numel() * ws.element_size(), C.byref(opts),
                                            _stream(stream)), "moe_nvfp4_forward_w4a16_ex")


def moe_nvfp4_forward_w4a16(d, w, x_bf16, topk_ids, topk_w, out, ws, stream=None):
    _need_cuda(x_bf16, topk_ids, topk_w, out, ws)
    T, K = topk_ids.shape
    _check(lib().moe_nvfp4_forward_w4a16(C.byref(d), C.byref(w.c), T, K, _ptr(x_bf16),
                                         _ptr(topk_ids), _ptr(topk_w), _ptr(out), _ptr(ws),
                                         ws.numel() * ws.element_size(), _stream(stream)),
           "moe_nvfp4_forward_w4a16")


def moe_nvfp4_forward_noalloc(d, w, codes, sf, scale, topk_ids, topk_w, out, stream=None):
    """The W4A4 forward on the library's own 64 MiB device scratch array, for
    callers that cannot allocate device memory (see include/moe_nvfp4.h)."""
    _need_cuda(codes, sf, scale, topk_ids, topk_w, out)
    T, K = topk_ids.shape
    _check(lib().moe_nvfp4_forward_noalloc(C.byref(d), C.byref(w.c), T, K, _ptr(codes), _ptr(sf),
                                           _ptr(scale), _ptr(topk_ids), _ptr(topk_w), _ptr(out),
                                           _stream(stream)),
           "moe_nvfp4_forward_noalloc")


def moe_nvfp4_read_status(ws, stream=None):
    """Device-reported status code of the last forward on `ws` (syncs the stream)."""
    return int(lib().moe_nvfp4_read_status(_ptr(ws), _stream(stream)))


def moe_nvfp4_profile_events(events):
    """Register torch.cuda.Event objects (already recorded once) as stage markers."""
    if not events:
        _check(lib().moe_nvfp4_profile_events(None, 0), "moe_nvfp4_profile_events")
        return
    arr = (C.c_void_p * len(events))(*[e.cuda_event for e in events])
    _check(lib().moe_nvfp4_profile_events(arr, len(events)), "moe_nvfp4_profile_events")


def moe_nvfp4_profile_spans(spans):
    """Register a CUDA int64 tensor of 4 elements (or None to unregister) that
    the grouped GEMM launches fold their %globaltimer spans into: [0]/[1] the
    FC1 (or one-launch) launch's earliest CTA start / latest CTA end, [2]/[3]
    the FC2 launch's.  Reset [0], [2] to the maximum and [1], [3] to 0 first."""
    if spans is not None and (not spans.is_cuda or spans.dtype != torch.int64
                              or spans.numel() < 4 or not spans.is_contiguous()):
        raise ValueError("spans: a contiguous CUDA int64 tensor of 4 elements")
    _check(lib().moe_nvfp4_profile_spans(None if spans is None else _ptr(spans)),
           "moe_nvfp4_profile_spans")


# ------------------------------------------------------------------ allocating helpers

class PreparedWeights:
    """Device buffers of the prepared NVFP4 weights (layouts in include/moe_nvfp4.h)."""

    def __init__(self, E, H, I, act, device="cuda"):
        self.dims = dims(E, H, I, act)
        self.E, self.H, self.I, self.act = E, H, I, act
        sizes = moe_nvfp4_weight_sizes(self.dims)
        Hp, Ip = padded(H), padded(I)
        N1 = 2 * Ip if act == "swiglu" else Ip
        self.fc1_codes = torch.empty(E, N1, Hp // 2, dtype=torch.uint8, device=device)
        self.fc1_sf = torch.empty(sizes[1], dtype=torch.uint8, device=device)
        self.fc1_alpha = torch.empty(E, dtype=torch.float32, device=device)
        self.fc2_codes = torch.empty(E, Hp, Ip // 2, dtype=torch.uint8, device=device)
        self.fc2_sf = torch.empty(sizes[4], dtype=torch.uint8, device=device)
        self.fc2_alpha = torch.empty(E, dtype=torch.float32, device=device)
        assert self.fc1_codes.numel() == sizes[0] and self.fc2_codes.numel() == sizes[3]
        self.c = moe_nvfp4_weights(*[t.data_ptr() for t in (
            self.fc1_codes, self.fc1_sf, self.fc1_alpha, self.fc2_codes, self.fc2_sf,
            self.fc2_alpha)])

    def nbytes(self):
        return sum(t.numel() * t.element_size() for t in (
            self.fc1_codes, self.fc1_sf, self.fc1_alpha, self.fc2_codes, self.fc2_sf,
            self.fc2_alpha))


def prepare_weights(fc1_bf16, fc2_bf16, act, out=None, stream=None):
    """Quantize BF16 stacks fc1 [E,N1,H] ([gate; up] for SwiGLU) and fc2 [E,H,I]."""
    E, N1, H = fc1_bf16.shape
    I = fc2_bf16.shape[2]
    w = out if out is not None else PreparedWeights(E, H, I, act, device=fc1_bf16.device)
    moe_nvfp4_prepare_weights(w.dims, fc1_bf16, fc2_bf16, w, stream)
    return w


def quantize_tokens(x_bf16, stream=None):
    T, H = x_bf16.shape
    dev = x_bf16.device
    Hp = padded(H)  # rows are zero-padded to Hp columns
    codes = torch.empty(T, Hp // 2, dtype=torch.uint8, device=dev)
    sf = torch.empty(T, Hp // 16, dtype=torch.uint8, device=dev)
    scale = torch.empty(T, dtype=torch.float32, device=dev)
    moe_nvfp4_quantize_tokens(x_bf16, codes, sf, scale, stream)
    return codes, sf, scale


def prepare_weights_per_tensor(fc1_bf16, fc2_bf16, act, a1_scale, a2_scale, out=None,
                               stream=None):
    """Per-tensor recipe weights: codes/scales as prepare_weights, alphas with the
    static device scalars a1_scale / a2_scale folded in."""
    E, N1, H = fc1_bf16.shape
    I = fc2_bf16.shape[2]
    w = out if out is not None else PreparedWeights(E, H, I, act, device=fc1_bf16.device)
    moe_nvfp4_prepare_weights_per_tensor(w.dims, fc1_bf16, fc2_bf16, a1_scale, a2_scale, w, stream)
    return w


def quantize_tokens_static(x_bf16, a1_scale, stream=None):
    T, H = x_bf16.shape
    Hp = padded(H)
    codes = torch.empty(T, Hp // 2, dtype=torch.uint8, device=x_bf16.device)
    sf = torch.empty(T, Hp // 16, dtype=torch.uint8, device=x_bf16.device)
    moe_nvfp4_quantize_tokens_static(x_bf16, a1_scale, codes, sf, stream)
    return codes, sf


def forward_per_tensor(w, codes, sf, a2_scale, topk_ids, topk_w, ws=None, out=None, stream=None):
    T, K = topk_ids.shape
    if ws is None:
        ws = workspace(w, T, K, device=codes.device)
    if out is None:
        out = torch.empty(T, w.H, dtype=torch.bfloat16, device=codes.device)
    moe_nvfp4_forward_per_tensor(w.dims, w, codes, sf, a2_scale, topk_ids, topk_w, out, ws, stream)
    return out


def route_topk(logits, K, stream=None):
    """Plain top-K router: fp32 logits [T,E] -> (int32 ids [T,K], fp32 scores [T,K])."""
    T = logits.shape[0]
    ids = torch.empty(T, K, dtype=torch.int32, device=logits.device)
    w = torch.empty(T, K, dtype=torch.float32, device=logits.device)
    moe_nvfp4_route_topk(logits, ids, w, stream)
    return ids, w


def workspace(w, T_max, K, w4a16=False, device="cuda"):
    n = moe_nvfp4_workspace_bytes(w.dims, T_max, K, w4a16)
    if n == 0:
        raise MoeError(2, "moe_nvfp4_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def forward(w, codes, sf, scale, topk_ids, topk_w, ws=None, out=None, stream=None):
    T, K = topk_ids.shape
    if ws is None:
        ws = workspace(w, T, K, device=codes.device)
    if out is None:
        out = torch.empty(T, w.H, dtype=torch.bfloat16, device=codes.device)
    moe_nvfp4_forward(w.dims, w, codes, sf, scale, topk_ids, topk_w, out, ws, stream)
    return out


def forward_opts(topk_ids, swiglu_limit=0.0):
    """Options for the *_ex calls: int64 ids follow from the tensor's dtype."""
    return moe_forward_opts(1 if topk_ids.dtype == torch.int64 else 0, float(swiglu_limit))


def forward_ex(w, codes, sf, scale, topk_ids, topk_w, swiglu_limit=0.0, ws=None, out=None,
               stream=None):
    T, K = topk_ids.shape
    if ws is None:
        ws = workspace(w, T, K, device=codes.device)
    if out is None:
        out = torch.empty(T, w.H, dtype=torch.bfloat16, device=codes.device)
    moe_nvfp4_forward_ex(w.dims, w, codes, sf, scale, topk_ids, topk_w, out, ws,
                         forward_opts(topk_ids, swiglu_limit), stream)
    return out


def forward_w4a16_ex(w, x_bf16, topk_ids, topk_w, swiglu_limit=0.0, ws=None, out=None,
                     stream=None):
    T, K = topk_ids.shape
    if ws is None:
        ws = workspace(w, T, K, w4a16=True, device=x_bf16.device)
    if out is None:
        out = torch.empty(T, w.H, dtype=torch.bfloat16, device=x_bf16.device)
    moe_nvfp4_forward_w4a16_ex(w.dims, w, x_bf16, topk_ids, topk_w, out, ws,
                               forward_opts(topk_ids, swiglu_limit), stream)
    return out


def forward_w4a16(w, x_bf16, topk_ids, topk_w, ws=None, out=None, stream=None):
    T, K = topk_ids.shape
    if ws is None:
        ws = workspace(w, T, K, w4a16=True, device=x_bf16.device)
    if out is None:
        out = torch.empty(T, w.H, dtype=torch.bfloat16, device=x_bf16.device)
    moe_nvfp4_forward_w4a16(w.dims, w, x_bf16, topk_ids, topk_w, out, ws, stream)
    return out


def ws_view(ws, layout, name, dtype, shape):
    """A typed view of one workspace region (offsets from moe_nvfp4_workspace_layout)."""
    off = layout[name]
    n = 1
    for s in shape:
        n *= s
    nbytes = n * torch.empty((), dtype=dtype).element_size()
    return ws[off:off + nbytes].view(dtype).view(*shape)


# ------------------------------------------------------------------ training objectives
#
# Losses and gradients of the routed model's trained parts (formulas and row rules
# in include/moe_nvfp4.h).  Logits may be views of row-strided storage; every other
# tensor is contiguous.  Outputs passed in are written and returned, else allocated
# on the stream of the call.  With `stream`, the inputs must be ready on that stream.
# Nothing is recorded for autograd: losses come back detached, also from logits that
# require a gradient; the gradients are what the *_grad calls return (pass them on with
# logits.backward(dlogits)).

_DTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_IDS64 = {torch.int32: 0, torch.int64: 1}


def _matrix(t, name):
    """moe_logits of a 2-D CUDA tensor whose rows are contiguous."""
    dt = _DTYPE.get(t.dtype)
    if dt is None or t.dim() != 2:
        raise ValueError(f"{name}: a 2-D float32, bfloat16 or float16 tensor")
    dev = t.get_device()  # -1 on the CPU
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"{name}: a tensor of the current CUDA device (no CPU path exists)")
    rows, cols = t.shape
    ld, one = t.stride()
    if (one != 1 and cols > 1) or (ld < cols and rows > 1):
        raise ValueError(f"{name}: rows must be contiguous and must not overlap")
    return moe_logits(t.data_ptr(), ld if rows > 1 else cols, rows, cols, dt)


def _arg(t, name, shape, dtypes, like):
    """Pointer of a contiguous tensor of the given shape and type, on `like`'s device."""
    if t is None:
        return None
    if t.dtype not in dtypes or t.shape != shape:
        raise ValueError(f"{name}: expected {tuple(shape)} of {[str(d) for d in dtypes]}, got "
                         f"{tuple(t.shape)} of {t.dtype}")
    if t.get_device() != like.get_device():
        raise ValueError(f"{name}: expected a tensor on {like.device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


_F32, _I32, _ID = (torch.float32,), (torch.int32,), (torch.int32, torch.int64)
_FLOAT, _MASK = tuple(_DTYPE), (torch.bool, torch.uint8)


def _out(t, name, shape, dtype, like, stream):
    """An output tensor: `t` if given, else a new one that belongs to `stream`."""
    if t is not None:
        _arg(t, name, shape, (dtype,), like)
        return t
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _dlogits(t, logits, stream):
    """The gradient's tensor and its row stride; rows may be strided like the logits'."""
    if t is None:
        t = _out(None, "dlogits", logits.shape, logits.dtype, logits, stream)
    elif t.shape != logits.shape or t.dtype != logits.dtype:
        raise ValueError("dlogits: must have the logits' shape and type")
    return t, _matrix(t, "dlogits").ld


def _raw(stream):
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def token_logp(logits, actions, temperature=1.0, logp=None, stream=None):
    """Log-probability [N] fp32 of one chosen token per row of logits [N, V];
    actions int32 or int64 [N], outside [0, V): the row is left out (0)."""
    z = _matrix(logits, "logits")
    n = logits.shape[:1]
    a = _arg(actions, "actions", n, _ID, logits)
    logp = _out(logp, "logp", n, torch.float32, logits, stream)
    _check(lib().moe_nvfp4_token_logp(z, a, _IDS64[actions.dtype], temperature, logp.data_ptr(),
                                      _raw(stream)), "moe_nvfp4_token_logp")
    return logp


def _policy_args(logits, actions, old_logp, advantages, ref_logp):
    n = logits.shape[:1]
    return (_matrix(logits, "logits"), _arg(actions, "actions", n, _ID, logits),
            _IDS64[actions.dtype], _arg(old_logp, "old_logp", n, _F32, logits),
            _arg(advantages, "advantages", n, _F32, logits),
            _arg(ref_logp, "ref_logp", n, _F32, logits))


def policy_loss(logits, actions, old_logp, advantages, ref_logp=None, clip_low=0.2, clip_high=0.2,
                kl_coef=0.0, temperature=1.0, row_loss=None, logp=None, stream=None):
    """Clipped policy loss with a KL term: (row_loss [N], logp [N]) fp32, detached."""
    args = _policy_args(logits, actions, old_logp, advantages, ref_logp)
    n = logits.shape[:1]
    row_loss = _out(row_loss, "row_loss", n, torch.float32, logits, stream)
    logp = _out(logp, "logp", n, torch.float32, logits, stream)
    _check(lib().moe_nvfp4_policy_loss(*args, moe_policy_opts(clip_low, clip_high, kl_coef,
                                                              temperature),
                                       row_loss.data_ptr(), logp.data_ptr(), _raw(stream)),
           "moe_nvfp4_policy_loss")
    return row_loss, logp


def policy_loss_grad(logits, actions, old_logp, advantages, row_weight=None, ref_logp=None,
                     clip_low=0.2, clip_high=0.2, kl_coef=0.0, temperature=1.0, row_loss=None,
                     logp=None, dlogits=None, stream=None):
    """policy_loss and the gradient of sum(row_weight * row_loss) (weights None: 1):
    (row_loss, logp, dlogits).  dlogits may be the logits tensor itself.  Rows of logits and
    gradient that lie alike to 16 bytes are fastest: for a slice of a padded head give a
    dlogits with its row stride."""
    args = _policy_args(logits, actions, old_logp, advantages, ref_logp)
    n = logits.shape[:1]
    w = _arg(row_weight, "row_weight", n, _F32, logits)
    row_loss = _out(row_loss, "row_loss", n, torch.float32, logits, stream)
    logp = _out(logp, "logp", n, torch.float32, logits, stream)
    dlogits, ld = _dlogits(dlogits, logits, stream)
    _check(lib().moe_nvfp4_policy_loss_grad(*args, w, moe_policy_opts(clip_low, clip_high, kl_coef,
                                                                      temperature),
                                            row_loss.data_ptr(), logp.data_ptr(),
                                            dlogits.data_ptr(), ld, _raw(stream)),
           "moe_nvfp4_policy_loss_grad")
    return row_loss, logp, dlogits


def moe_nvfp4_selftest_loss_timeout(logits, actions, old_logp, advantages, role, rank, row):
    """policy_loss_grad by a kernel in which one role leaves (include/moe_nvfp4.h):
    (row_loss, logp, dlogits)."""
    args = _policy_args(logits, actions, old_logp, advantages, None)[:5]
    row_loss, logp = torch.empty_like(old_logp), torch.empty_like(old_logp)
    dlogits, ld = _dlogits(None, logits, None)
    _check(lib().moe_nvfp4_selftest_loss_timeout(*args, role, rank, row, row_loss.data_ptr(),
                                                 logp.data_ptr(), dlogits.data_ptr(), ld,
                                                 _raw(None)), "moe_nvfp4_selftest_loss_timeout")
    return row_loss, logp, dlogits


def _teacher(logits, ids, t_logits, lse):
    if ids.dim() != 2 or ids.shape[0] != logits.shape[0]:
        raise ValueError("teacher_ids: one row of slots per row of logits")
    return moe_teacher(_arg(ids, "teacher_ids", ids.shape, _ID, logits),
                       _arg(t_logits, "teacher_logits", ids.shape, _FLOAT, logits),
                       _arg(lse, "teacher_lse", logits.shape[:1], _F32, logits),
                       ids.shape[1], _IDS64[ids.dtype], _DTYPE[t_logits.dtype])


def distill_loss(logits, teacher_ids, teacher_logits, teacher_lse=None, temperature=1.0,
                 row_loss=None, stream=None):
    """KL divergence [N] fp32 (detached) of softmax(logits / temperature) from a teacher's
    top logits: teacher_ids int32 / int64 [N, K] (outside [0, V): empty slot) and
    teacher_logits [N, K]; teacher_lse [N]: the teacher's whole row's, at the same
    temperature (else the slots are renormalised)."""
    z = _matrix(logits, "logits")
    t = _teacher(logits, teacher_ids, teacher_logits, teacher_lse)
    row_loss = _out(row_loss, "row_loss", logits.shape[:1], torch.float32, logits, stream)
    _check(lib().moe_nvfp4_distill_loss(z, t, temperature, row_loss.data_ptr(), _raw(stream)),
           "moe_nvfp4_distill_loss")
    return row_loss


def distill_loss_grad(logits, teacher_ids, teacher_logits, row_weight=None, teacher_lse=None,
                      temperature=1.0, row_loss=None, dlogits=None, stream=None):
    """distill_loss and the gradient of sum(row_weight * row_loss) (weights None: 1):
    (row_loss, dlogits).  dlogits may be the logits tensor itself."""
    z = _matrix(logits, "logits")
    t = _teacher(logits, teacher_ids, teacher_logits, teacher_lse)
    n = logits.shape[:1]
    w = _arg(row_weight, "row_weight", n, _F32, logits)
    row_loss = _out(row_loss, "row_loss", n, torch.float32, logits, stream)
    dlogits, ld = _dlogits(dlogits, logits, stream)
    _check(lib().moe_nvfp4_distill_loss_grad(z, t, w, temperature, row_loss.data_ptr(),
                                             dlogits.data_ptr(), ld, _raw(stream)),
           "moe_nvfp4_distill_loss_grad")
    return row_loss, dlogits


def _router_batch(logits, topk_ids, balance_coef, z_coef, seq_offsets, token_mask):
    z = _matrix(logits, "logits")
    T = logits.shape[0]
    if topk_ids.dim() != 2 or topk_ids.shape[0] != T:
        raise ValueError("topk_ids: one row of expert ids per row of logits")
    if seq_offsets is not None and (seq_offsets.dim() != 1 or seq_offsets.shape[0] < 2):
        raise ValueError("seq_offsets: S + 1 row numbers")
    S = 1 if seq_offsets is None else seq_offsets.shape[0] - 1
    return moe_router_batch(
        z, _arg(topk_ids, "topk_ids", topk_ids.shape, _ID, logits),
        _arg(token_mask, "token_mask", logits.shape[:1], _MASK, logits),
        None if seq_offsets is None else _arg(seq_offsets, "seq_offsets", seq_offsets.shape, _I32,
                                              logits),
        topk_ids.shape[1], S, _IDS64[topk_ids.dtype], balance_coef, z_coef)


def moe_nvfp4_router_loss_workspace_bytes(T, E, S=1):
    return int(lib().moe_nvfp4_router_loss_workspace_bytes(T, E, S))


def router_loss_workspace(T_max, E, S=1, device="cuda"):
    """A workspace for router_loss with up to T_max rows and S sequences."""
    n = moe_nvfp4_router_loss_workspace_bytes(T_max, E, S)
    if n == 0:
        raise MoeError(2, "moe_nvfp4_router_loss_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def router_loss(logits, topk_ids, balance_coef, z_coef=0.0, seq_offsets=None, token_mask=None,
                ws=None, losses=None, counts=None, tokens=None, stream=None):
    """Balance and z loss of router logits [T, E] and the load of the chosen experts
    topk_ids [T, K]: (losses [2] fp32, counts [S, E] int32, tokens [S + 1] int32: rows
    that count per sequence, then in all), detached.  seq_offsets int32 [S + 1] on the
    device; token_mask bool [T], False: left out."""
    b = _router_batch(logits, topk_ids, balance_coef, z_coef, seq_offsets, token_mask)
    T, E = logits.shape
    S = b.S
    losses = _out(losses, "losses", (2,), torch.float32, logits, stream)
    counts = _out(counts, "counts", (S, E), torch.int32, logits, stream)
    tokens = _out(tokens, "tokens", (S + 1,), torch.int32, logits, stream)
    L = lib()
    if ws is None:
        n = L.moe_nvfp4_router_loss_workspace_bytes(T, E, S)
        ws = _out(None, "ws", (n,), torch.uint8, logits, stream)
    else:
        n = ws.numel()
        _arg(ws, "ws", ws.shape, (torch.uint8,), logits)
    _check(L.moe_nvfp4_router_loss(b, losses.data_ptr(), counts.data_ptr(), tokens.data_ptr(),
                                   ws.data_ptr(), n, _raw(stream)), "moe_nvfp4_router_loss")
    return losses, counts, tokens


def router_loss_grad(logits, topk_ids, counts, tokens, balance_coef, z_coef=0.0, seq_offsets=None,
                     token_mask=None, loss_grad=None, topk_w=None, d_topk_w=None, dlogits=None,
                     stream=None):
    """Gradient [T, E] of router_loss with respect to the logits, given its counts and
    tokens; loss_grad [2]: upstream gradients of the two losses (None: 1).  With topk_w
    and d_topk_w [T, K] (route_topk's scores and their upstream gradients) the scores'
    gradient is added."""
    b = _router_batch(logits, topk_ids, balance_coef, z_coef, seq_offsets, token_mask)
    E = logits.shape[1]
    dlogits, ld = _dlogits(dlogits, logits, stream)
    _check(lib().moe_nvfp4_router_loss_grad(
        b, _arg(counts, "counts", (b.S, E), _I32, logits),
        _arg(tokens, "tokens", (b.S + 1,), _I32, logits),
        _arg(loss_grad, "loss_grad", (2,), _F32, logits),
        _arg(topk_w, "topk_w", topk_ids.shape, _F32, logits),
        _arg(d_topk_w, "d_topk_w", topk_ids.shape, _F32, logits),
        dlogits.data_ptr(), ld, _raw(stream)), "moe_nvfp4_router_loss_grad")
    return dlogits


# ------------------------------------------------------------------ routed rows

from .experts import (  # noqa: E402
    Checkpoint, MxExperts, MxTensor, RoutePlan, checkpoint, combine, combine_grad, dispatch,
    dispatch_grad, expert_act, expert_act_grad, moe_nvfp4_selftest_product_timeout,
    moe_nvfp4_sort_routes_workspace_bytes, mx_product, mx_quantize, mx_quantize_transposed,
    mx_restore, restore, sort_routes, sort_routes_workspace)
