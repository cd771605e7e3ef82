"""A differentiable pass through routed experts: routes sorted by expert, token rows to the
experts and back, activations kept in 8 bits, products in microscaled FP4, and MxExperts,
which runs them together.

Formulas, layouts and limits are in include/moe_nvfp4.h ("routed rows").  Rows may be views
of row-strided storage; every other tensor is contiguous.  Outputs passed in are written and
returned, else allocated on the stream of the call.  With `stream`, the inputs must be ready
on that stream.  Nothing is recorded for autograd: the gradients are what the *_grad calls
return.
"""
import ctypes as C
import math
from collections import namedtuple

import torch

from . import (_DTYPE, _F32, _I32, _ID, _IDS64, ACT, MoeError, _arg, _check, _matrix, _out, _raw,
               lib, moe_logits, moe_mx, padded)

_U8 = (torch.uint8,)


class _Interpreted:
    """In place of the compiled calls (csrc/calls.c): no call is theirs."""

    def __getattr__(self, name):
        return lambda *args: None


_fast = _Interpreted()
_FAST = ["sort_routes", "dispatch", "combine", "combine_grad", "checkpoint", "restore",
         "expert_act", "expert_act_grad", "mx_quantize", "mx_product",
         "sort_routes_workspace_bytes"]


def _attach(L):
    """Give the compiled calls the library's entry points, and use them from now on: each
    returns None for a call that is not an ordinary one, which then goes the interpreted way
    with its checks and errors."""
    global _fast
    try:
        from . import _calls
    except ImportError:  # not built (no Python headers): every call is interpreted
        return
    if not hasattr(torch._C, "_cuda_getCurrentRawStream"):
        return
    _calls.attach((torch.Tensor, _empty, torch._C._cuda_getDevice,
                   torch._C._cuda_getCurrentRawStream),
                  (torch.float32, torch.bfloat16, torch.float16, torch.uint8, torch.int32,
                   torch.int64), (MxTensor, Checkpoint, RoutePlan),
                  tuple(C.cast(getattr(L, "moe_nvfp4_" + n), C.c_void_p).value for n in _FAST))
    _fast = _calls


def _empty_by_torch(size, stride, dtype):
    return torch.empty_strided(size, stride, dtype=dtype, device="cuda")


# New tensors on the current device by (size, stride, dtype).  After a launch torch.empty takes
# 4.2 us on the host and the allocation that torch's compiled programs make 1.2.
_empty = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None),
                 "_empty_strided_cuda", _empty_by_torch)


def _new(shape, dtype, like):
    """A new tensor of one or two dimensions on like's device."""
    if like.get_device() != torch._C._cuda_getDevice():
        return torch.empty(shape, dtype=dtype, device=like.device)
    return _empty(tuple(shape), (shape[1], 1) if len(shape) == 2 else (1,), dtype)


def _like(t, name, shape, dtype, like, stream):
    """An output matrix: `t` (rows may be strided) or a new one; its address and row stride."""
    if t is None:
        t = (_new(shape, dtype, like) if stream is None
             else _out(None, name, shape, dtype, like, stream))
        return t, t.data_ptr(), shape[1]
    if t.shape != torch.Size(shape) or t.dtype != dtype:
        raise ValueError(f"{name}: expected {tuple(shape)} of {dtype}, got {tuple(t.shape)} of "
                         f"{t.dtype}")
    m = _matrix(t, name)
    if t.get_device() != like.get_device():
        raise ValueError(f"{name}: expected a tensor on {like.device}, got {t.device}")
    return t, m.data, m.ld


def _type_of(dtype, out, default):
    """The result's type: `dtype`, out's or the default; a given out has to agree."""
    if out is None:
        return dtype or default
    if dtype is not None and dtype != out.dtype:
        raise ValueError(f"dtype: {dtype}, but out is of {out.dtype}")
    return out.dtype


def _n_rows(t, like):
    return _arg(t, "n_rows", (1,), _I32, like) if t is not None else None


# ------------------------------------------------------------------ routes

class RoutePlan(namedtuple("RoutePlan", "offsets perm inv")):
    """Routes sorted by expert: offsets [E + 1], perm [T * K] (route of each row, -1 behind
    the last), inv [T, K] (row of each route, -1: empty slot), all int32."""
    __slots__ = ()

    @property
    def n_rows(self):
        """Rows in use, a device int32 [1]: for the calls that take n_rows."""
        return self.offsets[-1:]


def moe_nvfp4_sort_routes_workspace_bytes(T, K, E):
    return int(lib().moe_nvfp4_sort_routes_workspace_bytes(T, K, E))


def sort_routes_workspace(T_max, K, E, device="cuda"):
    """A workspace for sort_routes with up to T_max tokens."""
    n = moe_nvfp4_sort_routes_workspace_bytes(T_max, K, E)
    if n == 0:
        raise MoeError(2, "moe_nvfp4_sort_routes_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def sort_routes(topk_ids, E, plan=None, ws=None, stream=None):
    """Stable counting sort of the routes topk_ids [T, K] (int32 or int64, -1: empty slot) by
    expert: a RoutePlan.  Ids outside [-1, E) are empty slots too; with a workspace of the
    caller's (sort_routes_workspace) moe_nvfp4_read_status(ws) reports them."""
    if plan is None and ws is None and stream is None:
        r = _fast.sort_routes(topk_ids, E)
        if r is not None:
            return r
    if topk_ids.dim() != 2:
        raise ValueError("topk_ids: one row of expert ids per token")
    dev = topk_ids.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError("topk_ids: a tensor of the current CUDA device (no CPU path exists)")
    shape = T, K = topk_ids.shape
    ids = _arg(topk_ids, "topk_ids", shape, _ID, topk_ids)
    L = lib()
    if plan is None:
        plan = RoutePlan(_out(None, "offsets", E + 1, torch.int32, topk_ids, stream),
                         _out(None, "perm", T * K, torch.int32, topk_ids, stream),
                         _out(None, "inv", shape, torch.int32, topk_ids, stream))
        ptrs = plan.offsets.data_ptr(), plan.perm.data_ptr(), plan.inv.data_ptr()
    else:
        ptrs = (_arg(plan.offsets, "offsets", (E + 1,), _I32, topk_ids),
                _arg(plan.perm, "perm", (T * K,), _I32, topk_ids),
                _arg(plan.inv, "inv", shape, _I32, topk_ids))
    if ws is None:
        n = 0 if T * K <= 32768 else L.moe_nvfp4_sort_routes_workspace_bytes(T, K, E)
        ws = _out(None, "ws", n, torch.uint8, topk_ids, stream) if n else None
        wp = ws.data_ptr() if n else None
    else:
        n, wp = ws.numel(), _arg(ws, "ws", ws.shape, _U8, topk_ids)
    _check(L.moe_nvfp4_sort_routes(T, K, E, ids, _IDS64[topk_ids.dtype], *ptrs, wp, n,
                                   _raw(stream)), "moe_nvfp4_sort_routes")
    return plan


def dispatch(x, plan, rows=None, stream=None):
    """Token rows x [T, H] to their routes' rows [T * K, H]; x may be an MxTensor.  Rows behind
    the last route are left as they were (a new tensor's: undefined)."""
    if stream is None:
        r = _fast.dispatch(x, plan, rows)
        if r is not None:
            return r
    T, K = plan.inv.shape
    if x.shape[0] != T:
        raise ValueError(f"x: expected {T} rows, got {x.shape[0]}")
    if isinstance(x, MxTensor):
        if len(x.shape) != 2:
            raise ValueError("x: an MxTensor of rows [T, H]")
        inv = _arg(plan.inv, "inv", (T, K), _I32, x.on())
        if rows is None:
            rows = MxTensor.empty((T * K, x.shape[1]), x.on(), stream)
        rows.on()
        _check(lib().moe_nvfp4_mx_dispatch(x.c, K, inv, rows.c, _raw(stream)),
               "moe_nvfp4_mx_dispatch")
        return rows
    m = _matrix(x, "x")
    rows, p, ld = _like(rows, "rows", (T * K, x.shape[1]), x.dtype, x, stream)
    _check(lib().moe_nvfp4_dispatch(m, K, _arg(plan.inv, "inv", (T, K), _I32, x), p, ld,
                                    _raw(stream)), "moe_nvfp4_dispatch")
    return rows


def combine(rows, plan, topk_w=None, out=None, stream=None):
    """Route rows [T * K, H] back to their tokens [T, H], times topk_w fp32 [T, K] (None: 1)."""
    if out is None and stream is None:
        r = _fast.combine(rows, plan, topk_w)
        if r is not None:
            return r
    m = _matrix(rows, "rows")
    T, K = plan.inv.shape
    out, p, ld = _like(out, "out", (T, rows.shape[1]), rows.dtype, rows, stream)
    _check(lib().moe_nvfp4_combine(m, T, K, _arg(plan.inv, "inv", (T, K), _I32, rows),
                                   _arg(topk_w, "topk_w", (T, K), _F32, rows), p, ld,
                                   _raw(stream)), "moe_nvfp4_combine")
    return out


def dispatch_grad(drows, plan, dx=None, stream=None):
    """Gradient [T, H] of dispatch: the sum of each token's route rows."""
    return combine(drows, plan, None, dx, stream)


def combine_grad(rows, plan, topk_w, dout, drows=None, d_topk_w=None, stream=None):
    """Gradients of combine: (drows [T * K, H], d_topk_w [T, K] fp32).  drows may be the rows
    tensor itself; its rows behind the last route are left as they were."""
    if d_topk_w is None and stream is None:
        r = _fast.combine_grad(rows, plan, topk_w, dout, drows)
        if r is not None:
            return r
    m = _matrix(rows, "rows")
    T, K = plan.inv.shape
    if dout.shape != (T, rows.shape[1]) or dout.dtype != rows.dtype:
        raise ValueError("dout: one row per token, of the rows' length and type")
    md = _matrix(dout, "dout")
    drows, p, ld = _like(drows, "drows", rows.shape, rows.dtype, rows, stream)
    dw = _out(d_topk_w, "d_topk_w", (T, K), torch.float32, rows, stream)
    _check(lib().moe_nvfp4_combine_grad(m, T, K, _arg(plan.inv, "inv", (T, K), _I32, rows),
                                        _arg(topk_w, "topk_w", (T, K), _F32, rows), md.data, md.ld,
                                        p, ld, dw.data_ptr(), _raw(stream)),
           "moe_nvfp4_combine_grad")
    return drows, dw


# ------------------------------------------------------------------ 8 bits

class _Held:
    """Codes and scales on one device: two tensors, or one buffer that they are cut from when
    asked for (an allocation and two views less a call).  Their addresses are kept; a call looks
    whether the tensors still lie there, as a program may give them other storage (`codes.data =
    ...`; offloading does), and takes the new ones."""
    __slots__ = ("_codes", "_scales", "_buf", "_cut", "device")

    def _set(self, codes, scales):
        shapes = self._shapes()
        for t in (codes, scales):
            if t.numel() and t.untyped_storage().nbytes() < t.storage_offset() + t.numel():
                raise ValueError("codes, scales: their storage has been freed")
        at = (_arg(codes, "codes", shapes[0], _U8, codes),
              _arg(scales, "scales", shapes[1], _U8, codes))
        self.device = codes.get_device()  # -1 on the CPU: described, but no call takes it
        self._codes, self._scales, self._buf, self._cut = codes, scales, None, None
        return at

    def _moved(self, codes, scales):
        """Whether the tensors lie elsewhere than at these addresses."""
        return (self._codes.data_ptr() != (codes or 0) or
                self._scales.data_ptr() != (scales or 0))

    def _alloc(self, n_codes, n_scales, like, stream):
        at = (n_codes + 255) & -256
        self._buf = buf = (
            _new((at + n_scales,), torch.uint8, like) if stream is None
            else _out(None, "codes", at + n_scales, torch.uint8, like, stream))
        self._codes = self._scales = None
        self._cut = n_codes, at
        self.device = like.get_device()
        p = buf.data_ptr()
        return p, p + at

    def _views(self):
        buf = self._buf
        if buf is not None:
            shapes = self._shapes()
            self._codes = buf[:self._cut[0]].view(shapes[0])
            self._scales = buf[self._cut[1]:].view(shapes[1])
            self._buf = None  # the views hold it, and are what counts from now on

    @property
    def codes(self):
        self._views()
        return self._codes

    @property
    def scales(self):
        self._views()
        return self._scales

    def nbytes(self):
        return sum(math.prod(s) for s in self._shapes())

    def on(self):
        """A tensor of it, which has to lie on the current device (as every matrix of rows)."""
        self._look()
        t = self._buf if self._buf is not None else self._codes
        if self.device < 0 or self.device != torch._C._cuda_getDevice():
            raise ValueError("codes: a tensor of the current CUDA device (no CPU path exists)")
        return t


def _limit(limit):
    """swiglu_limit as a float; one that is not 0 but that fp32 rounds to 0 (no limit) is refused."""
    limit = float(limit)
    if limit and C.c_float(limit).value == 0.0:
        raise ValueError(f"swiglu_limit: {limit} is 0 in fp32")
    return limit


class Checkpoint(_Held):
    """Rows kept in 8 bits: codes [R, halves, W32] and scales [R, halves, W32 / 32] uint8, of
    `cols` values a half.  act: None for checkpoint's, else the activation whose input it is."""
    __slots__ = ("rows", "halves", "cols", "dtype", "act", "swiglu_limit", "c")

    def __init__(self, codes, scales, cols, dtype, act=None, swiglu_limit=0.0):
        if act is not None and act not in ACT:
            raise ValueError(f"act: None or one of {sorted(ACT)}")
        self.rows, self.cols, self.dtype, self.act = codes.shape[0], cols, dtype, act
        self.halves, self.swiglu_limit = 2 if act == "swiglu" else 1, _limit(swiglu_limit)
        self.c = self._set(codes, scales)

    @classmethod
    def empty(cls, rows, cols, dtype, like, act=None, swiglu_limit=0.0, stream=None):
        k = cls.__new__(cls)
        k.rows, k.cols, k.dtype, k.act = rows, cols, dtype, act
        k.halves, k.swiglu_limit = 2 if act == "swiglu" else 1, _limit(swiglu_limit)
        n = rows * k.halves * ((cols + 31) >> 5)
        k.c = k._alloc(32 * n, n, like, stream)
        return k

    def __reduce__(self):  # copies and pickles: the addresses are not theirs
        return Checkpoint, (self.codes, self.scales, self.cols, self.dtype, self.act,
                            self.swiglu_limit)

    def _look(self):
        if self._buf is None and self._moved(*self.c):  # a buffer is nobody else's
            self.c = self._set(self._codes, self._scales)

    def _shapes(self):
        b = (self.cols + 31) // 32
        return (self.rows, self.halves, 32 * b), (self.rows, self.halves, b)

    def _for(self, rows, cols):
        if self.rows != rows or self.cols != cols:
            raise ValueError(f"kept: holds {self.rows} rows of {self.cols}, got {rows} of {cols}")
        self.on()
        return self.c


def checkpoint(x, kept=None, n_rows=None, stream=None):
    """Rows x [R, D] in 8 bits (E4M3, a power of two per 32 values): a Checkpoint."""
    if kept is None and n_rows is None and stream is None:
        r = _fast.checkpoint(x)
        if r is not None:
            return r
    m = _matrix(x, "x")
    R, D = x.shape
    if kept is None:
        kept = Checkpoint.empty(R, D, x.dtype, x, stream=stream)
    elif kept.act is not None:
        raise ValueError("kept: made for an activation's input")
    codes, scales = kept._for(R, D)
    _check(lib().moe_nvfp4_checkpoint(m, codes, scales, _n_rows(n_rows, x), _raw(stream)),
           "moe_nvfp4_checkpoint")
    return kept


def restore(kept, dtype=None, out=None, n_rows=None, stream=None):
    """The rows that checkpoint kept, of `dtype` (None: out's, else the type they had)."""
    if dtype is None and out is None and n_rows is None and stream is None:
        r = _fast.restore(kept)
        if r is not None:
            return r
    if kept.act is not None:
        raise ValueError("kept: an activation's input is read by expert_act_grad")
    R, D = kept.rows, kept.cols
    dtype = _type_of(dtype, out, kept.dtype)
    if dtype not in _DTYPE:
        raise ValueError("dtype: float32, bfloat16 or float16")
    out, p, ld = _like(out, "out", (R, D), dtype, kept.on(), stream)
    codes, scales = kept.c
    _check(lib().moe_nvfp4_restore(codes, scales, moe_logits(p, ld, R, D, _DTYPE[dtype]),
                                   _n_rows(n_rows, out), _raw(stream)), "moe_nvfp4_restore")
    return out


def expert_act(h, act, swiglu_limit=0.0, checkpoint=False, y=None, kept=None, n_rows=None,
               stream=None):
    """The experts' activation of FC1 rows h: [R, 2I] = [gate | up] ("swiglu") or [R, I]
    ("relu2") -> y [R, I].  With checkpoint (or `kept`, a Checkpoint to fill) h is kept in 8
    bits for expert_act_grad: (y, kept), else y.  A block of 32 with an infinity or a NaN is kept
    as NaN, also where the limit makes y finite."""
    if y is None and kept is None and n_rows is None and stream is None:
        r = _fast.expert_act(h, act, swiglu_limit, checkpoint)
        if r is not None:
            return r
    if act not in ACT:
        raise ValueError(f"act: one of {sorted(ACT)}")
    limit = _limit(swiglu_limit)
    m = _matrix(h, "h")
    R, I = h.shape
    if act == "swiglu":
        I //= 2
    y, p, ld = _like(y, "y", (R, I), h.dtype, h, stream)
    codes = scales = None
    if kept is None:
        if checkpoint:
            kept = Checkpoint.empty(R, I, h.dtype, h, act, limit, stream)
            codes, scales = kept.c
    else:
        if kept.act != act or kept.swiglu_limit != limit:
            raise ValueError("kept: made for another activation")
        codes, scales = kept._for(R, I)
    _check(lib().moe_nvfp4_expert_act(m, ACT[act], limit, p, ld, codes, scales,
                                      _n_rows(n_rows, h), _raw(stream)), "moe_nvfp4_expert_act")
    return y if kept is None else (y, kept)


def expert_act_grad(kept, dy, dh=None, n_rows=None, stream=None):
    """Gradient of expert_act at the values that `kept` holds: dy [R, I] -> dh [R, 2I] (swiglu)
    or [R, I], of dy's type."""
    if dh is None and n_rows is None and stream is None:
        r = _fast.expert_act_grad(kept, dy)
        if r is not None:
            return r
    if kept.act is None:
        raise ValueError("kept: expected what expert_act kept")
    m = _matrix(dy, "dy")
    R, I = dy.shape
    codes, scales = kept._for(R, I)
    dh, p, ld = _like(dh, "dh", (R, kept.halves * I), dy.dtype, dy, stream)
    _check(lib().moe_nvfp4_expert_act_grad(codes, scales, ACT[kept.act], kept.swiglu_limit, m,
                                           p, ld, _n_rows(n_rows, dy), _raw(stream)),
           "moe_nvfp4_expert_act_grad")
    return dh


# ------------------------------------------------------------------ microscaled FP4

class MxTensor(_Held):
    """A matrix [R, D], or a stack [E, N, D], in microscaled FP4: codes uint8 [rows, Dp / 2] and
    scales uint8 [Dp / 256, Rp, 8] (Dp: D rounded up to 256, rows: R or E * N, Rp: rows rounded
    up to even; layouts in include/moe_nvfp4.h)."""
    __slots__ = ("shape", "raw")  # raw: the bytes of its moe_mx

    def __init__(self, codes, scales, shape):
        self.shape = shape = tuple(shape)
        raw = _fast.mx_raw(codes, scales, shape)
        if raw is not None:
            self.device, self.raw = codes.get_device(), raw
            self._codes, self._scales, self._buf, self._cut = codes, scales, None, None
            return
        p, q = self._set(codes, scales)
        self.raw = bytes(moe_mx(p, q, _mx_rows(shape), shape[-1]))

    @property
    def c(self):
        self._look()
        return moe_mx.from_buffer_copy(self.raw)

    def __reduce__(self):  # as Checkpoint's
        return MxTensor, (self.codes, self.scales, self.shape)

    def _look(self):
        if self._buf is not None:
            return
        m = moe_mx.from_buffer_copy(self.raw)
        if self._moved(m.codes, m.scales):
            p, q = self._set(self._codes, self._scales)
            self.raw = bytes(moe_mx(p, q, m.rows, m.cols))

    @classmethod
    def empty(cls, shape, like, stream=None):
        t = cls.__new__(cls)
        t.shape = shape
        rows, d = _mx_rows(shape), shape[-1]
        dp = (d + 255) & -256
        p, q = t._alloc(rows * dp >> 1, (rows + 1 & -2) * dp >> 5, like, stream)
        t.raw = bytes(moe_mx(p, q, rows, d))
        return t

    def _shapes(self):
        rows, dp = _mx_rows(self.shape), padded(self.shape[-1])
        return (rows, dp // 2), (dp // 256, (rows + 1) // 2 * 2, 8)


def _mx_rows(shape):
    if len(shape) not in (2, 3):
        raise ValueError("shape: [rows, D] or [E, N, D]")
    return shape[0] * shape[1] if len(shape) == 3 else shape[0]


def _mx_out(out, shape, x, stream):
    if out is None:
        return MxTensor.empty(shape, x, stream)
    if out.shape != shape:
        raise ValueError(f"out: expected {shape}, got {out.shape}")
    out.on()
    return out


def mx_quantize(x, out=None, n_rows=None, stream=None):
    """x [R, D] (rows may be strided) or [E, N, D] (contiguous) in microscaled FP4 (E2M1, a power
    of two per 32 values of a row): an MxTensor.  Values about the type's largest round to the
    power of two behind it (f16 from 57344 on: 65536), which products take as it is."""
    if out is None and n_rows is None and stream is None:
        r = _fast.mx_quantize(x)
        if r is not None:
            return r
    shape = tuple(x.shape)
    if len(shape) == 3:
        if not x.is_contiguous():
            raise ValueError("x: a stack must be contiguous")
        x = x.view(-1, shape[2])
    m = _matrix(x, "x")
    out = _mx_out(out, shape, x, stream)
    _check(lib().moe_nvfp4_mx_quantize(m, out.c, _n_rows(n_rows, x), _raw(stream)),
           "moe_nvfp4_mx_quantize")
    return out


def mx_quantize_transposed(x, out=None, stream=None):
    """A stack x [E, D, C] (or a matrix [D, C]), transposed: an MxTensor of [E, C, D], scaled along
    D."""
    if x.dim() not in (2, 3) or x.dtype not in _DTYPE or not x.is_contiguous():
        raise ValueError("x: a contiguous float32, bfloat16 or float16 stack [E, D, C] or matrix")
    if not x.is_cuda or x.get_device() != torch.cuda.current_device():
        raise ValueError("x: a tensor of the current CUDA device (no CPU path exists)")
    D, C = x.shape[-2:]
    shape = (x.shape[0], C, D) if x.dim() == 3 else (C, D)
    out = _mx_out(out, shape, x, stream)
    _check(lib().moe_nvfp4_mx_quantize_transposed(x.shape[0] if x.dim() == 3 else 1, D, C,
                                                  x.data_ptr(), _DTYPE[x.dtype], out.c,
                                                  _raw(stream)),
           "moe_nvfp4_mx_quantize_transposed")
    return out


def mx_restore(x, dtype=None, out=None, n_rows=None, stream=None):
    """The values of an MxTensor, as a tensor of its shape (into `out`: as rows), of `dtype` (None:
    out's, else bfloat16); infinite where one passes the type's largest."""
    dtype = _type_of(dtype, out, torch.bfloat16)
    if dtype not in _DTYPE:
        raise ValueError("dtype: float32, bfloat16 or float16")
    rows, D = x.c.rows, x.c.cols
    given = out is not None
    out, p, ld = _like(out, "out", (rows, D), dtype, x.on(), stream)
    _check(lib().moe_nvfp4_mx_restore(x.c, moe_logits(p, ld, rows, D, _DTYPE[dtype]),
                                      _n_rows(n_rows, out), _raw(stream)), "moe_nvfp4_mx_restore")
    return out if given or len(x.shape) == 2 else out.view(x.shape)


def _product_args(x, w, offsets, dtype, out, stream):
    if len(x.shape) != 2:
        raise ValueError("x: an MxTensor of rows [R, D]")
    E, N = w.shape[:2] if len(w.shape) == 3 else (1, w.shape[0])
    like = x.on()
    w._look()
    if w.device != x.device:
        raise ValueError(f"w: on device {w.device}, the rows on {x.device}")
    dtype = _type_of(dtype, out, torch.bfloat16)
    dt = _DTYPE.get(dtype)
    if dt is None:
        raise ValueError("dtype: float32, bfloat16 or float16")
    if offsets is not None:
        offsets = _arg(offsets, "offsets", (E + 1,), _I32, like)
    elif E > 1:
        raise ValueError("offsets: needed for a stack of weights")
    out, p, ld = _like(out, "out", (x.shape[0], N), dtype, like, stream)
    return out, (x.c, w.c, E, offsets), (dt, p, ld, _raw(stream))


def mx_product(x, w, offsets=None, dtype=None, out=None, stream=None):
    """x [R, D] times the weights of each row's expert: w [E, N, D] with offsets int32 [E + 1]
    (RoutePlan.offsets), or one matrix [N, D].  -> [R, N] of `dtype` (None: out's, else
    bfloat16); rows outside the groups are left as they were."""
    if out is None and stream is None:
        r = _fast.mx_product(x, w, offsets, dtype or torch.bfloat16)
        if r is not None:
            return r
    out, args, rest = _product_args(x, w, offsets, dtype, out, stream)
    _check(lib().moe_nvfp4_mx_product(*args, *rest), "moe_nvfp4_mx_product")
    return out


def moe_nvfp4_selftest_product_timeout(x, w, offsets, item, dtype=torch.bfloat16):
    """mx_product by a kernel whose row loads leave before work item `item`
    (include/moe_nvfp4.h)."""
    out, args, rest = _product_args(x, w, offsets, dtype, None, None)
    _check(lib().moe_nvfp4_selftest_product_timeout(*args, item, *rest),
           "moe_nvfp4_selftest_product_timeout")
    return out


# ------------------------------------------------------------------ together

class SavedPass:
    """What MxExperts.backward needs of a forward.  The experts' rows are overwritten by their
    gradient, so it can be taken once."""
    __slots__ = ("plan", "rows", "kept", "topk_w")

    def __init__(self, plan, rows, kept, topk_w):
        self.plan, self.rows, self.kept, self.topk_w = plan, rows, kept, topk_w

    def take(self):
        if self.kept is None:
            raise ValueError("saved: from a forward with keep=False")
        if self.rows is None:
            raise ValueError("saved: backward has used it already")
        rows, self.rows = self.rows, None
        return self.plan, rows, self.kept, self.topk_w


class MxExperts:
    """Routed experts in microscaled FP4 through which gradients pass: the weights stay frozen,
    forward keeps the activations' input in 8 bits, and backward returns the gradients of the
    tokens and of the routing weights.

    fc1 [E, N1, H] ([gate; up] for "swiglu"), fc2 [E, H, I].  backward multiplies with the
    transposed stacks, quantised along their other side (quantisation itself passes gradients
    through unchanged).  y = combine(FC2(act(FC1(x)))).

    The gradients that backward multiplies are rounded to FP4 to nearest, in blocks of 32: below a
    24th to a 12th of the block's largest they become 0.  A captured backward belongs into the
    graph of its forward, whose rows it overwrites.
    """

    def __init__(self, fc1, fc2, act, swiglu_limit=0.0, stream=None):
        if act not in ACT:
            raise ValueError(f"act: one of {sorted(ACT)}")
        E, N1, H = fc1.shape
        I = N1 // 2 if act == "swiglu" else N1
        if fc2.shape != (E, H, I):
            raise ValueError(f"fc2: expected {(E, H, I)}, got {tuple(fc2.shape)}")
        self.E, self.H, self.I, self.act, self.limit = E, H, I, act, _limit(swiglu_limit)
        self.fc1, self.fc2 = mx_quantize(fc1, stream=stream), mx_quantize(fc2, stream=stream)
        self.fc1_t = mx_quantize_transposed(fc1, stream=stream)
        self.fc2_t = mx_quantize_transposed(fc2, stream=stream)

    def forward(self, x, topk_ids, topk_w, keep=True, stream=None):
        """x [T, H], topk_ids [T, K], topk_w fp32 [T, K] -> (y [T, H], saved for backward)."""
        plan = sort_routes(topk_ids, self.E, stream=stream)
        n, dt = plan.n_rows, x.dtype
        # a token's codes are the same on each of its routes: quantised once, then copied
        xq = dispatch(mx_quantize(x, stream=stream), plan, stream=stream)
        h = mx_product(xq, self.fc1, plan.offsets, dt, stream=stream)
        a, kept = expert_act(h, self.act, self.limit, True, n_rows=n, stream=stream) if keep else (
            expert_act(h, self.act, self.limit, n_rows=n, stream=stream), None)
        rows = mx_product(mx_quantize(a, n_rows=n, stream=stream), self.fc2, plan.offsets, dt,
                          stream=stream)
        y = combine(rows, plan, topk_w, stream=stream)
        return y, SavedPass(plan, rows, kept, topk_w)

    def backward(self, saved, dy, stream=None):
        """dy [T, H] -> (dx [T, H], d_topk_w [T, K] fp32), once for each forward."""
        plan, rows, kept, topk_w = saved.take()
        n, dt = plan.n_rows, dy.dtype
        try:
            drows, dw = combine_grad(rows, plan, topk_w, dy, drows=rows, stream=stream)
        except Exception:  # refused (dy's type, shape or device): the rows are as they were
            saved.rows = rows
            raise
        da = mx_product(mx_quantize(drows, n_rows=n, stream=stream), self.fc2_t, plan.offsets, dt,
                        stream=stream)
        dh = expert_act_grad(kept, da, n_rows=n, stream=stream)
        dxr = mx_product(mx_quantize(dh, n_rows=n, stream=stream), self.fc1_t, plan.offsets, dt,
                         stream=stream)
        return dispatch_grad(dxr, plan, stream=stream), dw
