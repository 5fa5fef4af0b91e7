"""Thin ctypes binding of libcpdr.so (include/cpdr.h).

Argument marshalling only: tensors are passed as raw device pointers and the
current torch CUDA stream as a cudaStream_t; every step of the computation
runs in the library's CUDA kernels.  The library must have been built
(``python -c "import __graft_entry__ as g; g.build()"``); loading raises if it
is missing -- there is no fallback of any kind.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcpdr.so")

OK, ERR_INVALID, ERR_UNSUPPORTED, ERR_CUDA, ERR_WORKSPACE, ERR_TIMEOUT = range(6)
FLAG_HOST_ONLY = 1 << 0
FLAG_FORCE_SIMT = 1 << 1
FLAG_LAYOUT_ZIGZAG = 1 << 2
FLAG_STATE_V_FIRST = 1 << 3
FRAG_CONT_PREV, FRAG_CONT_NEXT, FRAG_ENDS_SEQ = 1, 2, 4

EXPORTED = ["cpdr_ctx_create", "cpdr_ctx_destroy", "cpdr_buffer_sizes", "cpdr_plan_num_fragments",
            "cpdr_plan_fragments", "cpdr_plan_counts", "cpdr_wy_bytes", "cpdr_wy_build", "cpdr_preprocess",
            "cpdr_merge", "cpdr_fwd", "cpdr_host_workspace_bytes",
            "cpdr_forward_host", "cpdr_forward_noalloc", "cpdr_check_device_status", "cpdr_selftest_wait_timeout",
            "cpdr_conv1d_fwd", "cpdr_plan_conv_tokens", "cpdr_bwd_workspace_bytes", "cpdr_bwd",
            "cpdr_glr_carry_bytes", "cpdr_plan_glr", "cpdr_glr_fwd", "cpdr_glr_bwd", "cpdr_glr_step", "cpdr_rmsnorm_fwd",
            "cpdr_rmsnorm_bwd_workspace_bytes", "cpdr_rmsnorm_bwd", "cpdr_plan_linear", "cpdr_linear_fwd",
            "cpdr_linear_bwd_workspace_bytes", "cpdr_linear_bwd", "cpdr_last_error", "cpdr_version"]


_F32, _BF16, _E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
ACTIVATIONS = {None: 0, "none": 0, "silu": 1, "gelu": 2}


class CpdrError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"cpdr status {status}: {msg}")
        self.status = status


class Desc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("dk", ctypes.c_int32), ("dv", ctypes.c_int32),
                ("R", ctypes.c_int32), ("num_seqs", ctypes.c_int32), ("T", ctypes.c_int64),
                ("cu_seqlens_host", ctypes.POINTER(ctypes.c_int64)), ("gate_kind", ctypes.c_int32),
                ("in_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32), ("scale", ctypes.c_float),
                ("Hq", ctypes.c_int32), ("conv_width", ctypes.c_int32)]


class Fragment(ctypes.Structure):
    _fields_ = [("tok0", ctypes.c_int64), ("len", ctypes.c_int32), ("seg", ctypes.c_int32),
                ("seq", ctypes.c_int32), ("flags", ctypes.c_int32)]


_lib = None
_lock = threading.Lock()


def load():
    """Load libcpdr.so and declare its signatures (raises if it is missing)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        lib = ctypes.CDLL(LIB_PATH)
        vp, sz = ctypes.c_void_p, ctypes.c_size_t
        st = ctypes.c_int
        lib.cpdr_ctx_create.argtypes = [ctypes.POINTER(Desc), ctypes.POINTER(vp)]
        lib.cpdr_ctx_destroy.argtypes = [vp]
        lib.cpdr_ctx_destroy.restype = None
        lib.cpdr_buffer_sizes.argtypes = [vp] + [ctypes.POINTER(sz)] * 4
        lib.cpdr_plan_num_fragments.argtypes = [vp, ctypes.POINTER(ctypes.c_int32)]
        lib.cpdr_plan_fragments.argtypes = [vp, ctypes.POINTER(Fragment), ctypes.c_int32]
        lib.cpdr_plan_counts.argtypes = [vp, ctypes.POINTER(ctypes.c_int32)]
        lib.cpdr_wy_bytes.argtypes = [vp, ctypes.POINTER(sz)]
        lib.cpdr_wy_build.argtypes = [vp] * 7
        lib.cpdr_preprocess.argtypes = [vp] * 9
        lib.cpdr_merge.argtypes = [vp] * 5
        lib.cpdr_fwd.argtypes = [vp] * 11
        lib.cpdr_host_workspace_bytes.argtypes = [vp, ctypes.POINTER(sz)]
        lib.cpdr_conv1d_fwd.argtypes = [vp, vp, vp, vp, ctypes.c_int32, ctypes.c_int32, vp, vp]
        lib.cpdr_plan_conv_tokens.argtypes = [vp, ctypes.POINTER(ctypes.c_int32), ctypes.c_int32]
        lib.cpdr_bwd_workspace_bytes.argtypes = [vp, ctypes.POINTER(sz)]
        lib.cpdr_bwd.argtypes = [vp] * 16 + [sz, vp]
        lib.cpdr_forward_host.argtypes = [vp] * 9 + [sz, vp]
        lib.cpdr_forward_noalloc.argtypes = [vp] * 9
        i32, i64, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        lib.cpdr_glr_carry_bytes.argtypes = [vp, i32, ctypes.POINTER(sz)]
        lib.cpdr_plan_glr.argtypes = [vp, i32, i32, ctypes.POINTER(i32)]
        lib.cpdr_glr_fwd.argtypes = [vp] * 4 + [i32] + [vp] * 4
        lib.cpdr_glr_bwd.argtypes = [vp] * 6 + [i32] + [vp] * 4
        lib.cpdr_glr_step.argtypes = [vp] * 6 + [i32] * 3 + [vp] * 2
        lib.cpdr_rmsnorm_fwd.argtypes = [vp, i64, i32, vp, vp, vp, f32] + [vp] * 5
        lib.cpdr_rmsnorm_bwd_workspace_bytes.argtypes = [vp, i64, i32, ctypes.POINTER(sz)]
        lib.cpdr_rmsnorm_bwd.argtypes = [vp, i64, i32, vp, vp, f32] + [vp] * 5 + [sz, vp]
        lib.cpdr_plan_linear.argtypes = [vp, i64, i32, i32, i32, ctypes.POINTER(i32)]
        lib.cpdr_linear_fwd.argtypes = [vp, i64, i32, i32] + [vp] * 5 + [i32] + [vp] * 4
        lib.cpdr_linear_bwd_workspace_bytes.argtypes = [vp, i64, i32, i32, i32, ctypes.POINTER(sz)]
        lib.cpdr_linear_bwd.argtypes = [vp, i64, i32, i32] + [vp] * 4 + [i32] + [vp] * 4 + [sz, vp]
        lib.cpdr_check_device_status.argtypes = [vp, vp]
        lib.cpdr_selftest_wait_timeout.argtypes = [vp, ctypes.c_longlong, vp]
        for name in EXPORTED:
            f = getattr(lib, name)
            if name not in ("cpdr_ctx_destroy", "cpdr_last_error", "cpdr_version"):
                f.restype = st
        lib.cpdr_last_error.restype = ctypes.c_char_p
        lib.cpdr_version.restype = ctypes.c_char_p
        _lib = lib
        return lib


def _check(status: int):
    if status != OK:
        raise CpdrError(status, load().cpdr_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _bad_tensor(name: str, t, shape, dtype, dev):
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {list(shape)} {dtype} tensor, got {list(t.shape)} {t.dtype}")
    raise ValueError(f"{name} must be on the context's device {dev}, got {t.device}")


def _addr(name: str, t, shape, dtype, dev):
    """The address of t, which must be a contiguous CUDA tensor of that shape
    and dtype on device index ``dev``; None (NULL) for None, which the library
    refuses where it must not be.  (A decoding step is bound by what the host
    does: the checks are few and cheap.)"""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous() or t.get_device() != dev:
        _bad_tensor(name, t, shape, dtype, dev)
    return t.data_ptr()


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _space(t, dev):
    """Address and bytes of a workspace tensor."""
    if not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"workspace must be a contiguous tensor on the context's device {dev}")
    return t.data_ptr(), t.numel() * t.element_size()


def _owned_by(stream):
    """Tensors made inside belong to ``stream`` (None: torch's current one):
    what a call makes and uses on a stream must not come from another one's
    memory."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _raw_stream(stream, dev):
    """cudaStream_t of ``stream``, or of torch's current stream on device ``dev``."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


class Context:
    """One planned problem: shapes, the R-segment cut, dtype and gate kind.

    ``gate`` is "gdn" (scalar gate g [B,T,H]) or "kda" (per-dim gk [B,T,H,d]);
    ``dtype`` is "fp32" or "bf16" for q, k, v, beta and o; gates are fp32.
    With ``cu_seqlens`` (N+1 offsets) the batch is packed: B must be 1.
    ``layout="zigzag"`` takes the token axis in the zigzag order of R ranks
    (2R parts, rank r holding parts r and 2R-1-r); ``Hq`` (a multiple of H)
    gives q and o grouped query heads; ``state_v_first`` stores the dk x dv
    states S_ext, S_init and final_state as [.., dv, dk].  ``conv_width``
    (1..8) enables ``conv1d_fwd``, the causal conv1d on the same segments.
    """

    def __init__(self, B, T, H, d, R, gate="gdn", dtype="bf16", cu_seqlens=None, scale=1.0,
                 host_only=False, force_simt=False, layout="contiguous", Hq=None, state_v_first=False,
                 conv_width=0):
        lib = load()
        if layout not in ("contiguous", "zigzag"):
            raise ValueError(f"layout must be 'contiguous' or 'zigzag', got {layout!r}")
        self.B, self.T, self.H, self.d, self.R = int(B), int(T), int(H), int(d), int(R)
        self.layout = layout
        # segments of the exchange buffers: the ranks, or 2R zigzag pieces
        self.pieces = 2 * self.R if layout == "zigzag" else self.R
        self.Hq = self.H if Hq is None else int(Hq)
        self.state_v_first = bool(state_v_first)
        self.conv_width = int(conv_width)
        self.gate, self.dtype = gate, dtype
        self.torch_dtype = torch.float32 if dtype == "fp32" else torch.bfloat16
        self._cu = None
        n = self.B
        cu_ptr = None
        if cu_seqlens is not None:
            cu = [int(x) for x in (cu_seqlens.tolist() if hasattr(cu_seqlens, "tolist") else cu_seqlens)]
            self._cu = (ctypes.c_int64 * len(cu))(*cu)
            cu_ptr = ctypes.cast(self._cu, ctypes.POINTER(ctypes.c_int64))
            n = len(cu) - 1
        self.N = n
        flags = ((FLAG_HOST_ONLY if host_only else 0) | (FLAG_FORCE_SIMT if force_simt else 0) |
                 (FLAG_LAYOUT_ZIGZAG if layout == "zigzag" else 0) |
                 (FLAG_STATE_V_FIRST if self.state_v_first else 0))
        desc = Desc(self.B, self.H, self.d, self.d, self.R, n, self.T, cu_ptr,
                    0 if gate == "gdn" else 1, 0 if dtype == "fp32" else 1, flags, float(scale), self.Hq,
                    self.conv_width)
        h = ctypes.c_void_p()
        _check(lib.cpdr_ctx_create(ctypes.byref(desc), ctypes.byref(h)))
        self._h = h
        self._lib = lib
        # the device of every tensor that a call takes (none: a host-only context launches nothing)
        self._dev = None if host_only else torch.cuda.current_device()

    def close(self):
        if getattr(self, "_h", None):
            self._lib.cpdr_ctx_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ---- plan ---------------------------------------------------------
    def fragments(self):
        n = ctypes.c_int32()
        _check(self._lib.cpdr_plan_num_fragments(self._h, ctypes.byref(n)))
        arr = (Fragment * max(1, n.value))()
        _check(self._lib.cpdr_plan_fragments(self._h, arr, n.value))
        return [(f.tok0, f.len, f.seg, f.seq, f.flags) for f in arr[:n.value]]

    def counts(self):
        """Plan counters: fragments, pre items, merge chains, zeroed S_ext/M
        segments, zeroed S_init segments, empty sequences, kernel launches per
        step, tensor-core path selected."""
        out = (ctypes.c_int32 * 8)()
        _check(self._lib.cpdr_plan_counts(self._h, out))
        keys = ["fragments", "pre_items", "chains", "zero_pre", "zero_init", "empty_seqs", "launches", "tc"]
        return dict(zip(keys, list(out)))

    def buffer_sizes(self):
        s = [ctypes.c_size_t() for _ in range(4)]
        _check(self._lib.cpdr_buffer_sizes(self._h, *[ctypes.byref(x) for x in s]))
        return [x.value for x in s]

    def wy_bytes(self):
        """Bytes of the WY tile workspace (0 on the CUDA-core path)."""
        n = ctypes.c_size_t()
        _check(self._lib.cpdr_wy_bytes(self._h, ctypes.byref(n)))
        return n.value

    def alloc_buffers(self, device="cuda"):
        """Caller-owned exchange buffers S_ext, M, S_init and final_state (fp32)
        and the WY tile workspace ``wy`` (bytes; None when not needed).  The
        segment axis has one entry per segment (2R in the zigzag layout); the
        last two axes of the states are (dk, dv), or (dv, dk) with
        ``state_v_first``."""
        d, R, B, H, N = self.d, self.pieces, self.B, self.H, self.N
        f32 = torch.float32
        nwy = self.wy_bytes()
        return dict(S_ext=torch.empty((R, B, H, d, d), dtype=f32, device=device),
                    M=torch.empty((R, B, H, d, d), dtype=f32, device=device),
                    S_init=torch.empty((R, B, H, d, d), dtype=f32, device=device),
                    final_state=torch.empty((N, H, d, d), dtype=f32, device=device),
                    wy=torch.empty(nwy, dtype=torch.uint8, device=device) if nwy else None)

    # ---- the three stages ------------------------------------------------
    def _check_inputs(self, **ts):
        B, T, H, d, Hq = self.B, self.T, self.H, self.d, self.Hq
        shapes = dict(q=(B, T, Hq, d), k=(B, T, H, d), v=(B, T, H, d), beta=(B, T, H), o=(B, T, Hq, d),
                      g=(B, T, H) if self.gate == "gdn" else (B, T, H, d))
        for name, t in ts.items():
            if t is None:
                continue
            if tuple(t.shape) != shapes[name]:
                raise ValueError(f"{name}: expected shape {shapes[name]}, got {tuple(t.shape)}")
            want = torch.float32 if name == "g" else self.torch_dtype
            if t.dtype != want:
                raise ValueError(f"{name}: expected {want}, got {t.dtype}")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")

    def wy_build(self, q, k, beta, g, wy, stream=None):
        """WY tiles (and, for the per-dim gate, the pre-gated operand tiles,
        which read q) into ``wy``."""
        self._check_inputs(q=q, k=k, beta=beta, g=g)
        _check(self._lib.cpdr_wy_build(self._h, _ptr(q), _ptr(k), _ptr(beta), _ptr(g), _ptr(wy),
                                       _stream(stream)))

    def preprocess(self, k, v, beta, g, S_ext, M, wy=None, stream=None):
        self._check_inputs(k=k, v=v, beta=beta, g=g)
        _check(self._lib.cpdr_preprocess(self._h, _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(wy), _ptr(S_ext),
                                         _ptr(M), _stream(stream)))

    def merge(self, S_ext, M, S_init, stream=None):
        _check(self._lib.cpdr_merge(self._h, _ptr(S_ext), _ptr(M), _ptr(S_init), _stream(stream)))

    def fwd(self, q, k, v, beta, g, S_init, o, final_state=None, wy=None, stream=None):
        self._check_inputs(q=q, k=k, v=v, beta=beta, g=g, o=o)
        _check(self._lib.cpdr_fwd(self._h, _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(wy),
                                  _ptr(S_init), _ptr(o), _ptr(final_state), _stream(stream)))

    def run(self, q, k, v, beta, g, bufs=None, o=None, stream=None):
        """WY build -> preprocess -> merge -> fwd on device tensors; returns (o, buffers)."""
        if bufs is None:
            bufs = self.alloc_buffers(q.device)
        if o is None:
            o = torch.empty((self.B, self.T, self.Hq, self.d), dtype=v.dtype, device=v.device)
        wy = bufs.get("wy")
        self.wy_build(q, k, beta, g, wy, stream)
        self.preprocess(k, v, beta, g, bufs["S_ext"], bufs["M"], wy=wy, stream=stream)
        self.merge(bufs["S_ext"], bufs["M"], bufs["S_init"], stream)
        self.fwd(q, k, v, beta, g, bufs["S_init"], o, bufs["final_state"], wy=wy, stream=stream)
        return o, bufs

    # ---- whole path from host memory --------------------------------------
    def host_workspace_bytes(self):
        n = ctypes.c_size_t()
        _check(self._lib.cpdr_host_workspace_bytes(self._h, ctypes.byref(n)))
        return n.value

    def forward_host(self, q, k, v, beta, g, o, final_state, workspace, stream=None):
        """Host tensors in (pinned for async copies), host o / final_state out."""
        self._check_inputs(q=q, k=k, v=v, beta=beta, g=g, o=o)
        _check(self._lib.cpdr_forward_host(self._h, _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(o),
                                           _ptr(final_state), _ptr(workspace),
                                           ctypes.c_size_t(workspace.numel() * workspace.element_size()),
                                           _stream(stream)))

    def forward_noalloc(self, q, k, v, beta, g, o, final_state=None, stream=None):
        """Whole path through the allocation-free entry point: the library
        keeps its exchange buffers and tables in a fixed device array and
        allocates nothing (works with a host_only context)."""
        self._check_inputs(q=q, k=k, v=v, beta=beta, g=g, o=o)
        _check(self._lib.cpdr_forward_noalloc(self._h, _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(o),
                                              _ptr(final_state), _stream(stream)))

    # ---- backward ------------------------------------------------------------
    def bwd_workspace_bytes(self):
        n = ctypes.c_size_t()
        _check(self._lib.cpdr_bwd_workspace_bytes(self._h, ctypes.byref(n)))
        return n.value

    def backward(self, q, k, v, beta, g, do, S_init, M, dht=None, workspace=None, stream=None):
        """Gradients of sum <do, o> + sum <dht, final_state> (fp32 tensors
        dq, dk, dv, dbeta, dg).  do is shaped like o ([B, T, Hq, dv]); S_init
        and M are the buffers the forward's merge and pre-process filled for
        the same inputs."""
        self._check_inputs(q=q, k=k, v=v, beta=beta, g=g)
        if tuple(do.shape) != tuple(q.shape[:3]) + (v.shape[3],) or do.dtype != v.dtype or not do.is_contiguous():
            raise ValueError("do must be shaped like o, in the dtype of v")
        dev = q.device
        f32 = torch.float32
        out = dict(dq=torch.empty(q.shape, dtype=f32, device=dev), dk=torch.empty(k.shape, dtype=f32, device=dev),
                   dv=torch.empty(v.shape, dtype=f32, device=dev),
                   dbeta=torch.empty(beta.shape, dtype=f32, device=dev), dg=torch.empty(g.shape, dtype=f32, device=dev))
        if workspace is None:
            workspace = torch.empty(self.bwd_workspace_bytes(), dtype=torch.uint8, device=dev)
        _check(self._lib.cpdr_bwd(self._h, _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(do), _ptr(dht),
                                  _ptr(S_init), _ptr(M), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
                                  _ptr(out["dbeta"]), _ptr(out["dg"]), _ptr(workspace),
                                  ctypes.c_size_t(workspace.numel()), _stream(stream)))
        return out

    # ---- causal conv1d on the same segments -------------------------------
    def conv_pre_tokens(self):
        """pre_num_conv_tokens per segment (entries: segments x rows)."""
        n = self.pieces * self.B
        out = (ctypes.c_int32 * n)()
        _check(self._lib.cpdr_plan_conv_tokens(self._h, out, n))
        return list(out)

    def conv1d_fwd(self, x, weight, bias, y, activation="silu", stream=None):
        """y = act(bias + causal depthwise conv of x), x and y [B, T, C] in the
        context's token order and input dtype; weight [C, W] and bias [C] fp32."""
        B, T = self.B, self.T
        if x.dim() != 3 or tuple(x.shape[:2]) != (B, T) or x.dtype != self.torch_dtype or not x.is_contiguous():
            raise ValueError(f"x must be a contiguous [{B}, {T}, C] {self.torch_dtype} tensor")
        C = x.shape[2]
        if tuple(y.shape) != tuple(x.shape) or y.dtype != x.dtype or not y.is_contiguous():
            raise ValueError("y must match x")
        if tuple(weight.shape) != (C, self.conv_width) or weight.dtype != torch.float32 or not weight.is_contiguous():
            raise ValueError(f"weight must be a contiguous [{C}, {self.conv_width}] float32 tensor")
        if bias is not None and (tuple(bias.shape) != (C,) or bias.dtype != torch.float32):
            raise ValueError(f"bias must be a [{C}] float32 tensor")
        act = {"silu": 1, None: 0, "none": 0}[activation]
        _check(self._lib.cpdr_conv1d_fwd(self._h, _ptr(x), _ptr(weight), _ptr(bias), C, act, _ptr(y),
                                         _stream(stream)))

    # ---- gated linear recurrence -------------------------------------------
    def glr_carry_shape(self, channels):
        """Shape of the fp32 ``carry`` that ``glr_fwd`` keeps for ``glr_bwd``:
        the state before every 16th token of each sequence."""
        n = ctypes.c_size_t()
        _check(self._lib.cpdr_glr_carry_bytes(self._h, int(channels), ctypes.byref(n)))
        return (n.value // (4 * int(channels)), int(channels))

    def glr_plan(self, channels, backward=False):
        """How the recurrence runs with that many channels: CTAs of a cluster,
        CTAs of an SM that the choice counts on, and those that the device holds."""
        out = (ctypes.c_int32 * 3)()
        _check(self._lib.cpdr_plan_glr(self._h, int(channels), int(backward), out))
        return dict(zip(("cluster", "per_sm", "resident"), out))

    def _glr_shapes(self, x):
        if x.dim() != 3 or tuple(x.shape[:2]) != (self.B, self.T):
            raise ValueError(f"x must be a [{self.B}, {self.T}, C] tensor, got {list(x.shape)}")
        C = x.shape[2]
        return C, x.shape, (self.N, C)

    def glr_fwd(self, x, g, y, h0=None, hT=None, carry=None, stream=None):
        """y_t = h_t = exp(g_t) h_{t-1} + x_t over every sequence of the
        context: x and y [B, T, C] in its token order and input dtype, g fp32;
        h0 and hT [N, C] fp32 or None; carry (``glr_carry_shape``) keeps what
        ``glr_bwd`` needs."""
        C, tok, st = self._glr_shapes(x)
        dt, dev = self.torch_dtype, self._dev
        keep = None if carry is None else _addr("carry", carry, self.glr_carry_shape(C), _F32, dev)
        _check(self._lib.cpdr_glr_fwd(self._h, _addr("x", x, tok, dt, dev), _addr("g", g, tok, _F32, dev),
                                      _addr("h0", h0, st, _F32, dev), C, _addr("y", y, tok, dt, dev),
                                      _addr("hT", hT, st, _F32, dev), keep, _raw_stream(stream, dev)))

    def glr_bwd(self, x, g, carry, dy, dhT=None, out=None, stream=None):
        """Gradients of sum <dy, y> + sum <dhT, hT>: a dict of dx (input
        dtype), dg and dh0 (fp32), written into ``out``'s tensors if given
        (dh0 may be None there)."""
        C, tok, st = self._glr_shapes(x)
        dt, dev = self.torch_dtype, self._dev
        args = (_addr("x", x, tok, dt, dev), _addr("g", g, tok, _F32, dev),
                _addr("carry", carry, self.glr_carry_shape(C), _F32, dev), _addr("dy", dy, tok, dt, dev),
                _addr("dhT", dhT, st, _F32, dev))
        if out is None:
            with _owned_by(stream):
                out = dict(dx=torch.empty_like(x), dg=torch.empty_like(g),
                           dh0=torch.empty(st, dtype=_F32, device=x.device))
        _check(self._lib.cpdr_glr_bwd(self._h, *args, C, _addr("dx", out["dx"], tok, dt, dev),
                                      _addr("dg", out["dg"], tok, _F32, dev),
                                      _addr("dh0", out.get("dh0"), st, _F32, dev),
                                      _raw_stream(stream, dev)))
        return out

    def glr_step(self, x, g, state, y, slots=None, state_out=None, stream=None):
        """One token for each row: x and y [n, C] in the input dtype, g [n, C]
        fp32; row i continues the sequence whose state is slot ``slots[i]``
        (int32; None: i) of state [S, C] fp32, updated in place or into
        ``state_out``.  Rows with a slot outside 0 .. S - 1 are left alone;
        rows of one slot are its consecutive tokens."""
        if x.dim() != 2 or state.dim() != 2:
            raise ValueError("x must be [n, C] and state [S, C]")
        rows, st = x.shape, state.shape
        dt, dev = self.torch_dtype, self._dev
        if st[1] != rows[1]:
            raise ValueError(f"state must have {rows[1]} channels, got {st[1]}")
        old = _addr("state", state, st, _F32, dev)
        _check(self._lib.cpdr_glr_step(self._h, _addr("x", x, rows, dt, dev), _addr("g", g, rows, _F32, dev), old,
                                       old if state_out is None else _addr("state_out", state_out, st, _F32, dev),
                                       _addr("slots", slots, rows[:1], torch.int32, dev), rows[0], st[0], rows[1],
                                       _addr("y", y, rows, dt, dev), _raw_stream(stream, dev)))

    # ---- RMS norm --------------------------------------------------------
    @staticmethod
    def _rows(x):
        """Rows and width of x, whose last axis is the row."""
        if x.dim() < 1:
            raise ValueError("x must have at least one dimension")
        width = x.shape[-1]
        return x.numel() // width if width else 0, width

    def rmsnorm_fwd(self, x, weight, residual=None, sum_out=None, y=None, y8=None, scale=None, eps=1e-6, stream=None):
        """RMS norm of s = x + residual over the last axis, times weight
        (fp32): s into ``sum_out``, the norm into ``y`` (input dtype) and/or
        ``y8`` (float8_e4m3fn) with ``scale`` (fp32, one per row).  |s| up to 1e17."""
        rows, width = self._rows(x)
        dt, dev, sh = self.torch_dtype, self._dev, x.shape
        _check(self._lib.cpdr_rmsnorm_fwd(self._h, rows, width, _addr("x", x, sh, dt, dev),
                                          _addr("residual", residual, sh, dt, dev),
                                          _addr("weight", weight, (width,), _F32, dev), eps,
                                          _addr("sum_out", sum_out, sh, dt, dev), _addr("y", y, sh, dt, dev),
                                          _addr("y8", y8, sh, _E4M3, dev),
                                          None if scale is None else _addr("scale", scale, sh[:-1], _F32, dev),
                                          _raw_stream(stream, dev)))

    def rmsnorm_bwd_workspace_bytes(self, rows, width):
        n = ctypes.c_size_t()
        _check(self._lib.cpdr_rmsnorm_bwd_workspace_bytes(self._h, int(rows), int(width), ctypes.byref(n)))
        return n.value

    def rmsnorm_bwd(self, s, weight, dy, dsum=None, eps=1e-6, out=None, workspace=None, stream=None):
        """Gradients of the norm from s (``sum_out``, or x), dy and the
        gradient ``dsum`` that reaches s past the norm: a dict of ds (input
        dtype; of x and residual alike) and dweight (fp32)."""
        rows, width = self._rows(s)
        dt, dev, sh = self.torch_dtype, self._dev, s.shape
        args = (_addr("s", s, sh, dt, dev), _addr("weight", weight, sh[-1:], _F32, dev), eps,
                _addr("dy", dy, sh, dt, dev), _addr("dsum", dsum, sh, dt, dev))
        with _owned_by(stream):
            if out is None:
                out = dict(ds=torch.empty_like(s), dweight=torch.empty_like(weight))
            if workspace is None:
                workspace = torch.empty(self.rmsnorm_bwd_workspace_bytes(rows, width), dtype=torch.uint8,
                                        device=s.device)
        _check(self._lib.cpdr_rmsnorm_bwd(self._h, rows, width, *args, _addr("ds", out["ds"], sh, dt, dev),
                                          _addr("dweight", out["dweight"], sh[-1:], _F32, dev), *_space(workspace, dev),
                                          _raw_stream(stream, dev)))
        return out

    # ---- matrix product with its epilogue ----------------------------------
    def linear_fwd(self, x, w, y, bias=None, activation=None, residual=None, z=None, x_scale=None, w_scale=None,
                   stream=None):
        """y = act(x w^T + bias) + residual over the last axis of x: x [.., K]
        and w [N, K] bf16, or float8_e4m3fn with ``x_scale`` [..] and
        ``w_scale`` [N]; y, residual and z (the value before the activation)
        [.., N] bf16; bias [N] fp32; activation None, "silu" or "gelu"."""
        rows, K = self._rows(x)
        dev, sh = self._dev, x.shape
        it = _BF16 if x_scale is None else _E4M3
        if w.dim() != 2:
            raise ValueError(f"w must be a [N, {K}] tensor, got {list(w.shape)}")
        N = w.shape[0]
        out, n = ((rows, N) if len(sh) == 2 else (*sh[:-1], N)), (N,)
        if (x_scale is None) != (w_scale is None):
            raise ValueError("x_scale and w_scale come together")
        _check(self._lib.cpdr_linear_fwd(self._h, rows, K, N, _addr("x", x, sh, it, dev),
                                         _addr("w", w, (N, K), it, dev),
                                         None if x_scale is None else _addr("x_scale", x_scale, sh[:-1], _F32, dev),
                                         _addr("w_scale", w_scale, n, _F32, dev), _addr("bias", bias, n, _F32, dev),
                                         ACTIVATIONS[activation], _addr("residual", residual, out, _BF16, dev),
                                         _addr("z", z, out, _BF16, dev), _addr("y", y, out, _BF16, dev),
                                         _raw_stream(stream, dev)))

    def linear_plan(self, rows, K, N, e4m3=False):
        """The form in which a product runs: (rows of x in a tile of the form for
        few rows, or 0 for the other one; CTAs that K is split over).  The input
        gradient of w [K, N] runs as a product of the same sizes."""
        out = (ctypes.c_int32 * 2)()
        _check(self._lib.cpdr_plan_linear(self._h, int(rows), int(K), int(N), int(e4m3), out))
        return tuple(out)

    def linear_bwd_workspace_bytes(self, rows, K, N, activation=None):
        n = ctypes.c_size_t()
        _check(self._lib.cpdr_linear_bwd_workspace_bytes(self._h, int(rows), int(K), int(N), ACTIVATIONS[activation],
                                                         ctypes.byref(n)))
        return n.value

    def linear_bwd(self, x, w, dy, z=None, activation=None, out=None, workspace=None, stream=None):
        """Gradients from dy [.., N] (also the residual's): a dict of dx and dw
        (bf16) and dbias (fp32).  Of a given ``out`` only the entries that it
        holds are computed."""
        rows, K = self._rows(x)
        dev, act = self._dev, ACTIVATIONS[activation]
        N = w.shape[0]
        wide = (*x.shape[:-1], N)
        if act and z is None:
            raise ValueError("z is missing: the gradient of an activation needs it")
        args = (_addr("x", x, x.shape, _BF16, dev), _addr("w", w, (N, K), _BF16, dev),
                _addr("z", z, wide, _BF16, dev), _addr("dy", dy, wide, _BF16, dev), act)
        with _owned_by(stream):
            if out is None:
                out = dict(dx=torch.empty_like(x), dw=torch.empty_like(w),
                           dbias=torch.empty(N, dtype=torch.float32, device=x.device))
            if workspace is None:
                workspace = torch.empty(self.linear_bwd_workspace_bytes(rows, K, N, activation), dtype=torch.uint8,
                                        device=x.device)
        _check(self._lib.cpdr_linear_bwd(self._h, rows, K, N, *args, _addr("dx", out.get("dx"), x.shape, _BF16, dev),
                                         _addr("dw", out.get("dw"), w.shape, _BF16, dev),
                                         _addr("dbias", out.get("dbias"), (N,), torch.float32, dev),
                                         *_space(workspace, dev), _raw_stream(stream, dev)))
        return out

    def check_device_status(self, stream=None):
        _check(self._lib.cpdr_check_device_status(self._h, _stream(stream)))

    def selftest_wait_timeout(self, max_cycles=20_000_000, stream=None):
        """Make one bounded device wait give up on purpose (see include/cpdr.h)."""
        _check(self._lib.cpdr_selftest_wait_timeout(self._h, ctypes.c_longlong(int(max_cycles)), _stream(stream)))
