"""ctypes binding of libsketchssm (include/sketchssm.h): argument marshalling only.

Every step of the flush and decode runs in the library's CUDA kernels; this module
only turns torch tensors into device pointers and status codes into exceptions.
PyTorch supplies the device memory and the stream.  If the library has not been
built, loading fails loudly: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libsketchssm.so")

DENSE = -1
KINDS = {"mamba2": 0, "gdn": 1, "kda": 2}
STATUS = {0: "SKETCHSSM_OK", 1: "SKETCHSSM_ERR_INVALID_ARG", 2: "SKETCHSSM_ERR_ALIGNMENT",
          3: "SKETCHSSM_ERR_UNSUPPORTED", 4: "SKETCHSSM_ERR_CUDA", 5: "SKETCHSSM_ERR_TIMEOUT"}

# every symbol include/sketchssm.h declares
EXPORTS = ("sketchssm_plan_create", "sketchssm_plan_query", "sketchssm_plan_check",
           "sketchssm_plan_set_wait_limit", "sketchssm_plan_destroy", "sketchssm_flush", "sketchssm_decode", "sketchssm_dense_decode",
           "sketchssm_decode_static_scratch", "sketchssm_step", "sketchssm_decode_rows",
           "sketchssm_flush_rows", "sketchssm_prefill", "sketchssm_status_string", "sketchssm_last_error",
           "sketchssm_delta_chunk", "sketchssm_delta_step", "sketchssm_gated_norm")


# sketchssm_dtype, sketchssm_gate
DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
GATES = {"silu": 0, "sigmoid": 1}


class SketchSSMError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}: {detail}")


class Desc(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in
                ("kind", "batch", "heads", "qk_heads", "key_dim", "value_dim", "window", "groups",
                 "basis_rows", "rank_cap")]


class TokenDesc(ctypes.Structure):
    """sketchssm_token_desc"""
    _fields_ = [("dtype", ctypes.c_int32), ("normalize_qk", ctypes.c_int32), ("scale", ctypes.c_float),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("y_stride", ctypes.c_int64)]


class NormDesc(ctypes.Structure):
    """sketchssm_norm_desc"""
    _fields_ = [(f, ctypes.c_int32) for f in
                ("x_dtype", "dtype", "groups", "width", "weight_groups", "gate", "gate_first")] + [
                    ("eps", ctypes.c_float), ("x_stride", ctypes.c_int64), ("z_stride", ctypes.c_int64),
                    ("out_stride", ctypes.c_int64)]


_lib = None


def load():
    """Load libsketchssm.so (raises if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m rank_state_read_b200.build` "
                           "(nvcc, sm_100a); there is no fallback implementation")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.sketchssm_plan_create.argtypes = [ctypes.POINTER(Desc), P, P, P, ctypes.POINTER(P)]
    lib.sketchssm_plan_query.argtypes = [P, ctypes.POINTER(I64), P, P, I32, P, ctypes.POINTER(I32)]
    lib.sketchssm_plan_check.argtypes = [P, P]
    lib.sketchssm_plan_set_wait_limit.argtypes = [P, I64]
    lib.sketchssm_plan_destroy.argtypes = [P]
    lib.sketchssm_flush.argtypes = [P, P, P, P, P, P, P, I32, P, P]
    lib.sketchssm_decode.argtypes = [P, I32, P, P, P, P, P, P, P, P, P, P, P, P, P, P]
    lib.sketchssm_dense_decode.argtypes = [P, I32, P, P, P, P, P, P, P, P, P, P, P, P]
    lib.sketchssm_decode_static_scratch.argtypes = [P, I32, P, P, P, P, P, P, P, P, P, P, P, P, P, P]
    lib.sketchssm_step.argtypes = [P, P, P, P, P, P, P, P, P]
    lib.sketchssm_decode_rows.argtypes = [P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P]
    lib.sketchssm_flush_rows.argtypes = [P, P, P, P, P, P, P, P, P, P]
    lib.sketchssm_prefill.argtypes = [P, I32, P, P, P, P, P, P, P, P]
    lib.sketchssm_delta_chunk.argtypes = [P, ctypes.POINTER(TokenDesc), I32, I32, P, P, P, P, P, P, P, P, P, P]
    lib.sketchssm_delta_step.argtypes = [P, ctypes.POINTER(TokenDesc), I32, P, P, P, P, P, P, P, P, P]
    lib.sketchssm_gated_norm.argtypes = [ctypes.POINTER(NormDesc), I32, P, P, P, P, P]
    for f in EXPORTS[:13] + EXPORTS[15:]:
        getattr(lib, f).restype = ctypes.c_int
    lib.sketchssm_status_string.argtypes = [ctypes.c_int]
    lib.sketchssm_status_string.restype = ctypes.c_char_p
    lib.sketchssm_last_error.argtypes = []
    lib.sketchssm_last_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(status: int, where: str) -> None:
    if status != 0:
        raise SketchSSMError(status, where, load().sketchssm_last_error().decode())


# the current stream's handle without the Stream object around it (3 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> Optional[int]:
    if stream is None:
        if _raw_stream is not None and torch.cuda.is_initialized():
            return _raw_stream(_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t: Optional[torch.Tensor], name: str, numel: Optional[int] = None):
    if t is None or (numel == 0 and t.numel() == 0):
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
    return t.data_ptr()


class Plan:
    """A layer shape at a fixed batch plus its rank table (sketchssm_plan)."""

    def __init__(self, kind: str, *, batch: int, heads: int, qk_heads: int, key_dim: int,
                 value_dim: int, window: int, groups: int, basis_rows: int, rank_cap: int,
                 rank: Sequence[int], group: Optional[Sequence[int]] = None, stream=None):
        lib = load()
        self.kind = kind
        self.desc = Desc(KINDS[kind], batch, heads, qk_heads, key_dim, value_dim, window, groups,
                         basis_rows, rank_cap)
        if len(rank) != heads:
            raise ValueError("rank table must have one entry per head")
        rank_arr = (ctypes.c_int32 * heads)(*[int(r) for r in rank])
        group_arr = None
        if group is not None:
            if len(group) != heads:
                raise ValueError("group table must have one entry per head")
            group_arr = (ctypes.c_int32 * heads)(*[int(g) for g in group])
        handle = ctypes.c_void_p()
        _check(lib.sketchssm_plan_create(ctypes.byref(self.desc), ctypes.cast(rank_arr, ctypes.c_void_p),
                                         None if group_arr is None else ctypes.cast(group_arr, ctypes.c_void_p),
                                         _stream(stream), ctypes.byref(handle)), "sketchssm_plan_create")
        self.handle = handle
        self.rank = [int(r) for r in rank]
        rt = ctypes.c_int64()
        off = (ctypes.c_int32 * (heads + 1))()
        rmax = (ctypes.c_int32 * groups)()
        _check(lib.sketchssm_plan_query(handle, ctypes.byref(rt), ctypes.cast(off, ctypes.c_void_p),
                                        ctypes.cast(rmax, ctypes.c_void_p), 1, None, None),
               "sketchssm_plan_query")
        self.r_total = int(rt.value)
        self.offsets = list(off)
        self.rmax = list(rmax)
        self._state_numel = batch * heads * key_dim * value_dim
        self.work = {}
        for n in range(1, window + 1):
            nw = ctypes.c_int32()
            work = (ctypes.c_int32 * (groups + heads))()
            _check(lib.sketchssm_plan_query(handle, None, None, None, n,
                                            ctypes.cast(work, ctypes.c_void_p), ctypes.byref(nw)),
                   "sketchssm_plan_query")
            self.work[n] = list(work)[: nw.value]

    # shapes of the caller-owned tensors (include/sketchssm.h, "Layouts")
    @property
    def shapes(self) -> dict:
        d = self.desc
        B, H, Q, K, V, W, G = d.batch, d.heads, d.qk_heads, d.key_dim, d.value_dim, d.window, d.groups
        kda = self.kind == "kda"
        return {"S": (B, H, K, V), "omega": (G, d.basis_rows, K), "Y": (B, self.r_total, V),
                "q": (B, Q, K), "k": (B, Q, K), "v": (B, H, V), "a": (B, H, K) if kda else (B, H),
                "beta": (B, H), "kbuf": (B, Q, W, K), "vbuf": (B, H, W, V),
                "abuf": (B, H, W, K) if kda else (B, H, W), "bbuf": (B, H, W), "y": (B, H, V)}

    def numel(self, name: str) -> int:
        n = 1
        for x in self.shapes[name]:
            n *= x
        return n

    def check(self, stream=None) -> None:
        """Synchronise and raise if a kernel recorded a timeout (sketchssm_plan_check)."""
        _check(load().sketchssm_plan_check(self.handle, _stream(stream)), "sketchssm_plan_check")

    def set_wait_limit(self, cycles: int) -> None:
        """Cycles a CTA waits for its own copies before it records a timeout
        (sketchssm_plan_set_wait_limit; default 2e9)."""
        _check(load().sketchssm_plan_set_wait_limit(self.handle, int(cycles)), "sketchssm_plan_set_wait_limit")

    def close(self) -> None:
        if getattr(self, "handle", None) is not None and self.handle.value:
            load().sketchssm_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def sketchssm_plan_create(kind: str, rank: Sequence[int], stream=None, **shape) -> Plan:
    return Plan(kind, rank=rank, stream=stream, **shape)


def sketchssm_plan_destroy(plan: Plan) -> None:
    plan.close()


def sketchssm_flush(plan: Plan, S, omega, kbuf, vbuf, abuf, bbuf, n_tokens: int, Y, stream=None) -> None:
    n = plan.numel
    _check(load().sketchssm_flush(
        plan.handle, _ptr(S, "S", n("S")), _ptr(omega, "omega", n("omega")),
        _ptr(kbuf, "kbuf", n("kbuf")), _ptr(vbuf, "vbuf", n("vbuf")), _ptr(abuf, "abuf", n("abuf")),
        _ptr(bbuf, "bbuf", n("bbuf")), int(n_tokens), _ptr(Y, "Y", n("Y")), _stream(stream)),
        "sketchssm_flush")


def sketchssm_decode(plan: Plan, pos: int, q, k, v, a, beta, kbuf, vbuf, abuf, bbuf, Y, omega, S, y,
                     stream=None) -> None:
    n = plan.numel
    _check(load().sketchssm_decode(
        plan.handle, int(pos), _ptr(q, "q", n("q")), _ptr(k, "k", n("k")), _ptr(v, "v", n("v")),
        _ptr(a, "a", n("a")), _ptr(beta, "beta", n("beta")), _ptr(kbuf, "kbuf", n("kbuf")),
        _ptr(vbuf, "vbuf", n("vbuf")), _ptr(abuf, "abuf", n("abuf")), _ptr(bbuf, "bbuf", n("bbuf")),
        _ptr(Y, "Y", n("Y")), _ptr(omega, "omega", n("omega")), _ptr(S, "S", n("S")),
        _ptr(y, "y", n("y")), _stream(stream)), "sketchssm_decode")


def sketchssm_dense_decode(plan: Plan, pos: int, q, k, v, a, beta, kbuf, vbuf, abuf, bbuf, S, y,
                           stream=None) -> None:
    n = plan.numel
    _check(load().sketchssm_dense_decode(
        plan.handle, int(pos), _ptr(q, "q", n("q")), _ptr(k, "k", n("k")), _ptr(v, "v", n("v")),
        _ptr(a, "a", n("a")), _ptr(beta, "beta", n("beta")), _ptr(kbuf, "kbuf", n("kbuf")),
        _ptr(vbuf, "vbuf", n("vbuf")), _ptr(abuf, "abuf", n("abuf")), _ptr(bbuf, "bbuf", n("bbuf")),
        _ptr(S, "S", n("S")), _ptr(y, "y", n("y")), _stream(stream)), "sketchssm_dense_decode")


def sketchssm_decode_static_scratch(plan: Plan, pos: int, q, k, v, a, beta, kbuf, vbuf, abuf, bbuf, Y, omega,
                                    S, y, stream=None) -> None:
    """sketchssm_decode with its scratch in the library's static device array (no allocation)."""
    n = plan.numel
    _check(load().sketchssm_decode_static_scratch(
        plan.handle, int(pos), _ptr(q, "q", n("q")), _ptr(k, "k", n("k")), _ptr(v, "v", n("v")),
        _ptr(a, "a", n("a")), _ptr(beta, "beta", n("beta")), _ptr(kbuf, "kbuf", n("kbuf")),
        _ptr(vbuf, "vbuf", n("vbuf")), _ptr(abuf, "abuf", n("abuf")), _ptr(bbuf, "bbuf", n("bbuf")),
        _ptr(Y, "Y", n("Y")), _ptr(omega, "omega", n("omega")), _ptr(S, "S", n("S")),
        _ptr(y, "y", n("y")), _stream(stream)), "sketchssm_decode_static_scratch")


def sketchssm_step(plan: Plan, q, k, v, a, beta, S, y, stream=None) -> None:
    """The standard per-step decode (sketchssm_step): S updated in place, y = S^T q."""
    n = plan.numel
    _check(load().sketchssm_step(
        plan.handle, _ptr(q, "q", n("q")), _ptr(k, "k", n("k")), _ptr(v, "v", n("v")), _ptr(a, "a", n("a")),
        _ptr(beta, "beta", n("beta")), _ptr(S, "S", n("S")), _ptr(y, "y", n("y")), _stream(stream)),
        "sketchssm_step")


def sketchssm_prefill(plan: Plan, T: int, k, v, a, beta, S, omega, Y, stream=None) -> None:
    """Prefill handoff (sketchssm_prefill): the prompt's T tokens applied to S in place,
    then Y formed from the new state.  k [B][T][Hqk][K], v [B][T][H][V], a [B][T][H]
    (KDA [B][T][H][K]), beta [B][T][H] (None for Mamba-2)."""
    d, n = plan.desc, plan.numel
    T = int(T)
    per_tok = {"k": d.batch * d.qk_heads * d.key_dim, "v": d.batch * d.heads * d.value_dim,
               "a": n("a"), "beta": d.batch * d.heads}
    if T == 0:
        k = v = a = beta = None
    _check(load().sketchssm_prefill(
        plan.handle, T, _ptr(k, "k", T * per_tok["k"]), _ptr(v, "v", T * per_tok["v"]),
        _ptr(a, "a", T * per_tok["a"]), _ptr(beta, "beta", T * per_tok["beta"]),
        _ptr(S, "S", n("S")), _ptr(omega, "omega", n("omega")), _ptr(Y, "Y", n("Y")), _stream(stream)),
        "sketchssm_prefill")


def _rows(t, name: str, B: int):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 CUDA tensor")
    if t.numel() != B:
        raise ValueError(f"{name} has {t.numel()} elements, expected {B}")
    return t.data_ptr()


def sketchssm_decode_rows(plan: Plan, pos, q, k, v, a, beta, kbuf, vbuf, abuf, bbuf, Y, omega, S, y,
                          stream=None) -> None:
    """sketchssm_decode with a buffer position per batch row (pos: int32 [B] on the device)."""
    n = plan.numel
    _check(load().sketchssm_decode_rows(
        plan.handle, _rows(pos, "pos", plan.desc.batch), _ptr(q, "q", n("q")), _ptr(k, "k", n("k")),
        _ptr(v, "v", n("v")), _ptr(a, "a", n("a")), _ptr(beta, "beta", n("beta")), _ptr(kbuf, "kbuf", n("kbuf")),
        _ptr(vbuf, "vbuf", n("vbuf")), _ptr(abuf, "abuf", n("abuf")), _ptr(bbuf, "bbuf", n("bbuf")),
        _ptr(Y, "Y", n("Y")), _ptr(omega, "omega", n("omega")), _ptr(S, "S", n("S")), _ptr(y, "y", n("y")),
        _stream(stream)), "sketchssm_decode_rows")


def sketchssm_flush_rows(plan: Plan, S, omega, kbuf, vbuf, abuf, bbuf, n_tokens, Y, stream=None) -> None:
    """sketchssm_flush with a token count per batch row (n_tokens: int32 [B] on the device)."""
    n = plan.numel
    _check(load().sketchssm_flush_rows(
        plan.handle, _ptr(S, "S", n("S")), _ptr(omega, "omega", n("omega")), _ptr(kbuf, "kbuf", n("kbuf")),
        _ptr(vbuf, "vbuf", n("vbuf")), _ptr(abuf, "abuf", n("abuf")), _ptr(bbuf, "bbuf", n("bbuf")),
        _rows(n_tokens, "n_tokens", plan.desc.batch), _ptr(Y, "Y", n("Y")), _stream(stream)),
        "sketchssm_flush_rows")


def _rows3(t, name: str, dtype, shape):
    """Pointer and row stride (0: packed) of a tensor of this shape, [n][x][y], whose rows are contiguous."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.shape == shape and t.is_contiguous():
        return (t.data_ptr() if shape[0] else None), 0
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    n, x, y = shape
    if n == 0:
        return None, 0
    s0, s1, s2 = t.stride()
    if (s2 != 1 and y != 1) or (s1 != y and x != 1):
        raise ValueError(f"the rows of {name} must be contiguous")
    if n == 1:
        return t.data_ptr(), 0
    if s0 < x * y:
        raise ValueError(f"the rows of {name} overlap")
    return t.data_ptr(), s0


def _count(n: int) -> int:
    """A number of rows or tokens, which the C interface takes in 32 bits."""
    if n > 0x7FFFFFFF:
        raise ValueError(f"{n} rows are more than a call takes")
    return n


def _ints(t, name: str, numel: int):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 CUDA tensor")
    if t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
    return t.data_ptr()


def _delta(plan: Plan, n: int, q, k, v, a, beta, S, y, normalize_qk, scale):
    d = plan.desc
    H = d.heads
    qk, hv = (n, d.qk_heads, d.key_dim), (n, H, d.value_dim)
    dtype = getattr(q, "dtype", None)
    if dtype not in DTYPES:
        raise TypeError(f"q must be a float32, bfloat16 or float16 tensor, got {dtype}")
    qp, qs = _rows3(q, "q", dtype, qk)
    kp, ks = _rows3(k, "k", dtype, qk)
    vp, vs = _rows3(v, "v", dtype, hv)
    yp, ys = _rows3(y, "y", dtype, hv)
    td = TokenDesc(DTYPES[dtype], bool(normalize_qk), scale, qs, ks, vs, ys)
    return td, (qp, kp, vp, _ptr(a, "a", n * H), _ptr(beta, "beta", n * H), _ptr(S, "S", plan._state_numel), yp)


def sketchssm_delta_chunk(plan: Plan, cu, q, k, v, a, beta, S, y, *, slot=None, normalize_qk: bool = False,
                          scale: float = 1.0, stream=None) -> None:
    """The gated delta rule on packed prompts (sketchssm_delta_chunk): sequence i holds the tokens
    cu[i] .. cu[i+1]-1 and continues state slot[i] (None: state i) of S in place; y gets the
    tokens' outputs.  cu [seqs+1], slot [seqs]: int32 on the device; q, k [N][Hqk][K], v, y
    [N][H][V] of one type (fp32, bf16, fp16), contiguous but for the stride between tokens; a,
    beta [N][H] fp32.  With ``normalize_qk`` q and k are brought to unit length first; ``scale``
    multiplies q."""
    if not isinstance(cu, torch.Tensor) or cu.numel() < 1:
        raise TypeError("cu must be an int32 CUDA tensor of one entry more than there are sequences")
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    n, seqs = _count(q.shape[0]), _count(cu.numel() - 1)
    td, ptrs = _delta(plan, n, q, k, v, a, beta, S, y, normalize_qk, scale)
    _check(load().sketchssm_delta_chunk(plan.handle, td, seqs, n, _ints(cu, "cu", seqs + 1),
                                        _ints(slot, "slot", seqs), *ptrs, _stream(stream)), "sketchssm_delta_chunk")


def sketchssm_delta_step(plan: Plan, q, k, v, a, beta, S, y, *, slot=None, normalize_qk: bool = False,
                         scale: float = 1.0, stream=None) -> None:
    """The gated delta rule on one token a row (sketchssm_delta_step): row i on state slot[i] (None:
    state i).  Tensors as for sketchssm_delta_chunk."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    n = _count(q.shape[0])
    td, ptrs = _delta(plan, n, q, k, v, a, beta, S, y, normalize_qk, scale)
    _check(load().sketchssm_delta_step(plan.handle, td, n, _ints(slot, "slot", n), *ptrs, _stream(stream)),
           "sketchssm_delta_step")


def sketchssm_gated_norm(x, z, weight, out, *, eps: float = 1e-6, activation: str = "silu",
                         gate_first: bool = False, stream=None) -> None:
    """The gated norm behind a layer's read (sketchssm_gated_norm): RMS norm of x [rows][groups][width]
    over each group, times weight ([width], or [groups][width]) and the gate of z (None: no gate),
    which multiplies after the norm or, with ``gate_first``, before it.  x, z, out may be strided
    between rows; out has z's type (without z: its own) and may be x or z itself."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3 or x.dtype not in DTYPES:
        raise TypeError("x must be a float32, bfloat16 or float16 tensor [rows][groups][width]")
    if not isinstance(out, torch.Tensor) or out.dtype not in DTYPES:
        raise TypeError("out must be a float32, bfloat16 or float16 tensor")
    if activation not in GATES:
        raise ValueError(f"activation must be one of {sorted(GATES)}, got {activation!r}")
    n, groups, width = shape = x.shape
    _count(max(n, groups, width))
    xp, xs = _rows3(x, "x", x.dtype, shape)
    zp, zs = (None, 0) if z is None else _rows3(z, "z", out.dtype, shape)
    op, os_ = _rows3(out, "out", out.dtype, shape)
    wg = 1 if isinstance(weight, torch.Tensor) and weight.numel() == width else groups
    nd = NormDesc(DTYPES[x.dtype], DTYPES[out.dtype], groups, width, wg, GATES[activation], bool(gate_first), eps,
                  xs, zs, os_)
    _check(load().sketchssm_gated_norm(nd, n, xp, zp, _ptr(weight, "weight", wg * width), op, _stream(stream)),
           "sketchssm_gated_norm")
