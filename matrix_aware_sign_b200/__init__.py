"""Thin Python binding of libsmuon.so (the C ABI in include/smuon.h).

Argument marshalling only: every step of the optimizer runs in the library's
CUDA kernels. PyTorch supplies device memory and the current stream. There is
no fallback: if the shared library is missing, importing a function raises.

Functions keep the C names: smuon_ns, smuon_sign_pack, smuon_vote,
smuon_update, cachemuon_reuse_probe, lionmuon_step, adamw_step, adamw_convert,
smuon_grad_norm (plus the workspace queries). Matrices are 2-D torch tensors
with unit column stride; the AdamW calls take tensors of any shape.
"""
from __future__ import annotations

import ctypes
import os
import struct
from contextlib import nullcontext
from ctypes import POINTER, c_double, c_float, c_int8, c_int32, c_int64, c_size_t, c_uint32, c_void_p

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsmuon.so")

F32, BF16, I8, BITS, E4M3 = 0, 1, 2, 3, 4
NS_FP32_REF, NS_SPLIT_BF16, NS_NO_NORMALIZE, NS_EMIT_Q, NS_SIMT_BF16 = 1, 2, 4, 8, 16
NS_GRAM_ONLY = 32  # CacheMuon fresh solve iterated on the m x m Gram (with NS_EMIT_Q, one matrix)
NS_SPECTRAL = 64  # spectral-norm normalisation X_0 = M / (||M||_2 + eps) (Lanczos estimate on the device)
NS_TEST_WAIT_EXPIRY = 0x8000  # failure-detection test: the tensor-core stages' pipeline waits run out
NS_ONE_SM = 0x80  # tensor-core stages on single-SM 128 x 256 tiles instead of SM pairs (256 x 256 tiles)


def ns_plain_lead(k: int) -> int:
    """SMUON_NS_PLAIN_LEAD(k): with NS_SPLIT_BF16, the first k Newton-Schulz steps use plain BF16 operands."""
    if not 0 <= k <= 7:
        raise ValueError("k must be in 0..7")
    return k << 12
VOTE_POPCOUNT, VOTE_INT8 = 0, 1
VOTE_TEST_WAIT_EXPIRY = 0x100  # failure-detection test: the bulk-copy 1-bit vote's waits run out, W unchanged
LION_MUON_VOTE = 0x100  # lionmuon_step ns_flags: Muon steps as Sign-Muon steps (per-worker NS + vote)
DEV_NONFINITE_NORM, DEV_WAIT_TIMEOUT = 1, 2

STATUS_NAMES = {0: "OK", -1: "INVALID_ARG", -2: "SHAPE", -3: "DTYPE", -4: "UNSUPPORTED",
                -5: "WORKSPACE", -6: "CUDA"}


class SmuonError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"smuon status {code} ({STATUS_NAMES.get(code, '?')}): {msg}")
        self.code = code


class SmuonMat(ctypes.Structure):
    _fields_ = [("data", c_void_p), ("rows", c_int32), ("cols", c_int32), ("ld", c_int64),
                ("dtype", c_int32)]


class CacheMuonCounters(ctypes.Structure):
    _fields_ = [("hits", c_int64), ("misses", c_int64), ("probes", c_int64), ("reserved", c_int64)]


class TraceRec(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 40), ("kind", c_int32), ("work", ctypes.c_double),
                ("nominal", ctypes.c_double), ("ms", c_float)]


class GradStream(ctypes.Structure):
    """smuon_grad_stream: worker k's gradient of matrix j is keyed (seed_base + k, matrix_base + j)."""
    _fields_ = [("seed_base", c_uint32), ("matrix_base", c_uint32), ("sigma", c_float), ("reserved", c_uint32)]


class LionMuonState(ctypes.Structure):
    _fields_ = [("n_layers", c_int32), ("workers", c_int32), ("W", POINTER(SmuonMat)),
                ("mom", POINTER(SmuonMat)), ("t", c_int64), ("grad", POINTER(GradStream))]


class AdamWState(ctypes.Structure):
    """adamw_state (the binding's AdamW fills it)."""
    _fields_ = [("n_tensors", c_int32), ("seed", c_uint32), ("W", POINTER(SmuonMat)), ("master", POINTER(SmuonMat)),
                ("m", POINTER(SmuonMat)), ("v", POINTER(SmuonMat)), ("scales", POINTER(c_void_p)),
                ("lr_scale", POINTER(c_float)), ("weight_decay", POINTER(c_float)), ("t", c_int64),
                ("d_t", c_void_p)]


_lib = None


def lib() -> ctypes.CDLL:
    """Loads libsmuon.so once; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m matrix_aware_sign_b200.build` (there is no fallback)")
        L = ctypes.CDLL(LIB_PATH)
        M = POINTER(SmuonMat)
        sigs = {
            "smuon_last_error": (ctypes.c_char_p, []),
            "smuon_version": (c_int32, []),
            "smuon_launch_count": (c_int64, []),
            "smuon_trace_enable": (None, [c_int32]),
            "smuon_trace_read": (c_int32, [POINTER(TraceRec), c_int32]),
            "smuon_ns_workspace_bytes": (c_int32, [M, c_int32, c_int32, c_uint32, POINTER(c_size_t)]),
            "smuon_ns": (c_int32, [M, M, c_int32, M, c_float, c_float, c_float, c_float, c_int32, c_float,
                                   c_uint32, M, c_void_p, c_void_p, c_size_t, c_void_p, c_void_p]),
            "smuon_sign_pack": (c_int32, [M, c_int32, c_void_p, c_void_p, c_void_p]),
            "smuon_vote": (c_int32, [c_void_p, c_void_p, c_int32, c_int64, c_int8, c_void_p, c_void_p]),
            "smuon_update": (c_int32, [M, c_int32, M, M, M, c_int32, c_float, c_int8, c_uint32,
                                       POINTER(c_void_p), POINTER(c_void_p), c_void_p, c_void_p]),
            "smuon_ns_static": (c_int32, [M, M, c_int32, M, c_float, c_float, c_float, c_float, c_int32, c_float,
                                          c_uint32, M, c_void_p, c_void_p, c_void_p]),
            "smuon_ns_plan_create": (c_int32, [M, M, c_int32, M, c_float, c_float, c_float, c_float, c_int32,
                                               c_float, c_uint32, M, c_void_p, c_size_t, c_void_p, c_void_p,
                                               POINTER(c_void_p)]),
            "smuon_ns_execute": (c_int32, [c_void_p, c_void_p, c_void_p]),
            "smuon_update_plan_create": (c_int32, [M, c_int32, M, M, M, c_int32, c_float, c_int8, c_uint32,
                                                   POINTER(c_void_p), POINTER(c_void_p), c_void_p,
                                                   POINTER(c_void_p)]),
            "smuon_update_execute": (c_int32, [c_void_p, c_void_p]),
            "smuon_plan_destroy": (None, [c_void_p]),
            "cachemuon_workspace_bytes": (c_int32, [M, POINTER(c_size_t)]),
            "cachemuon_reuse_probe": (c_int32, [M, M, M, c_float, c_float, c_void_p, c_void_p, c_void_p,
                                                c_void_p, c_size_t, c_void_p, c_void_p]),
            "smuon_harness_gaussian": (c_int32, [M, c_int32, c_int32, POINTER(GradStream), c_uint32, c_void_p]),
            "lionmuon_workspace_bytes": (c_int32, [POINTER(LionMuonState), c_int32, c_uint32,
                                                   POINTER(c_size_t)]),
            "lionmuon_step": (c_int32, [POINTER(LionMuonState), c_int32, c_float, c_float, c_float, c_float,
                                        c_float, c_float, c_int32, c_int8, c_uint32, M, c_void_p, c_size_t,
                                        c_void_p, c_void_p]),
            "adamw_step": (c_int32, [POINTER(AdamWState), M, c_double, c_double, c_double, c_double, c_void_p,
                                     c_void_p, c_void_p, c_void_p]),
            "adamw_plan_workspace_bytes": (c_int32, [POINTER(AdamWState), POINTER(c_size_t)]),
            "adamw_plan_create": (c_int32, [POINTER(AdamWState), M, c_double, c_double, c_double, c_void_p, c_void_p,
                                            c_void_p, c_void_p, c_size_t, c_void_p, POINTER(c_void_p)]),
            "adamw_execute": (c_int32, [c_void_p, POINTER(AdamWState), c_double, c_void_p]),
            "adamw_convert": (c_int32, [POINTER(AdamWState), POINTER(AdamWState), c_void_p]),
            "smuon_grad_norm_workspace_bytes": (c_int32, [M, c_int32, POINTER(c_size_t)]),
            "smuon_grad_norm": (c_int32, [M, c_int32, c_double, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p,
                                          c_void_p]),
            "smuon_grad_norm_plan_create": (c_int32, [M, c_int32, c_double, c_void_p, c_void_p, c_void_p, c_size_t,
                                                      c_void_p, c_void_p, POINTER(c_void_p)]),
            "smuon_grad_norm_execute": (c_int32, [c_void_p, c_void_p]),
        }
        for name, (res, args) in sigs.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(code: int) -> None:
    if code != 0:
        raise SmuonError(code, lib().smuon_last_error().decode())


_DT = {torch.float32: F32, torch.bfloat16: BF16, torch.int8: I8}


class Bits:
    """The 1-bit message of a rows x cols sign matrix (SMUON_BITS): `words` is a
    contiguous int32 tensor of packed_words(rows * cols) words, entry i of the
    row-major flattening at bit i % 32 of word i // 32."""

    def __init__(self, words: torch.Tensor, rows: int, cols: int):
        if words.dtype != torch.int32 or not words.is_contiguous() or words.numel() < packed_words(rows * cols):
            raise ValueError("words must be a contiguous int32 tensor of packed_words(rows * cols) words")
        self.words, self.rows, self.cols = words, int(rows), int(cols)

    @property
    def shape(self):
        return (self.rows, self.cols)

    @property
    def device(self):
        return self.words.device

    @staticmethod
    def empty(rows: int, cols: int, device=None) -> "Bits":
        return Bits(torch.zeros(packed_words(rows * cols), dtype=torch.int32, device=device or "cuda"), rows, cols)


def mat(t) -> SmuonMat:
    """Describes a 2-D row-major tensor (unit column stride), or a Bits message."""
    if isinstance(t, Bits):
        return SmuonMat(t.words.data_ptr(), t.rows, t.cols, t.cols, BITS)
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError("matrices must be 2-D with unit column stride")
    if t.dtype not in _DT:
        raise ValueError(f"dtype {t.dtype} is not supported")
    ld = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    return SmuonMat(t.data_ptr(), t.shape[0], t.shape[1], max(ld, t.shape[1]), _DT[t.dtype])


def _mats(ts):
    if ts is None:
        return None
    arr = (SmuonMat * len(ts))(*[mat(t) for t in ts])
    return arr


def _ptr(t):
    return None if t is None else t.data_ptr()


# The current device and a device's current stream as bare numbers, by PyTorch's own short ways where it has them
# (torch.cuda.current_stream() builds a Stream object, 3 us a call).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream(stream):
    if stream is None:
        return _raw_stream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _torch_stream(handle, index):
    """The stream of a handle on device `index` (handle 0 is the default stream; ExternalStream(0) would be a new one)."""
    return torch.cuda.ExternalStream(handle, device=index) if handle else torch.cuda.default_stream(index)


def workspace(nbytes: int, device=None) -> torch.Tensor:
    """Caller-owned workspace (torch allocation, 512-byte aligned)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


# ---------------------------------------------------------------- diagnostics
WORK_FLOPS, WORK_BYTES = 0, 1


def launch_count() -> int:
    return lib().smuon_launch_count()


def trace_enable(on: bool = True) -> None:
    lib().smuon_trace_enable(1 if on else 0)


def trace_read() -> list[dict]:
    """Synchronises on the logged launch events and returns and clears them."""
    n = lib().smuon_trace_read(None, 0)
    if n == 0:
        return []
    buf = (TraceRec * n)()
    got = lib().smuon_trace_read(buf, n)
    return [dict(name=r.name.decode(), kind=r.kind, work=r.work, nominal=r.nominal, ms=r.ms) for r in buf[:got]]


# ---------------------------------------------------------------- smuon_ns
def smuon_ns_workspace_bytes(M_in, iters: int, flags: int = 0) -> int:
    arr = _mats(M_in)
    out = c_size_t(0)
    _check(lib().smuon_ns_workspace_bytes(arr, len(M_in), iters, flags, ctypes.byref(out)))
    return out.value


def smuon_ns(M_in, U_out, a, b, c, iters, G=None, beta=0.0, eps=1e-7, flags=0, Q_out=None,
             skip_if=None, ws=None, status=None, stream=None):
    """Momentum (when G is given) + Frobenius normalisation + K Newton-Schulz steps."""
    if ws is None:
        ws = workspace(smuon_ns_workspace_bytes(M_in, iters, flags), M_in[0].device)
    _check(lib().smuon_ns(_mats(M_in), _mats(U_out), len(M_in), _mats(G), beta, a, b, c, iters, eps, flags,
                          _mats(Q_out), _ptr(skip_if), ws.data_ptr(), ws.numel(), _ptr(status),
                          _stream(stream)))
    return ws


NS_STATIC_SCRATCH_BYTES = 32 << 20


def smuon_ns_static(M_in, U_out, a, b, c, iters, G=None, beta=0.0, eps=1e-7, flags=0, Q_out=None,
                    skip_if=None, status=None, stream=None):
    """smuon_ns with the library's fixed device scratch array (no workspace, no allocation)."""
    _check(lib().smuon_ns_static(_mats(M_in), _mats(U_out), len(M_in), _mats(G), beta, a, b, c, iters, eps, flags,
                                 _mats(Q_out), _ptr(skip_if), _ptr(status), _stream(stream)))


class NsPlan:
    """smuon_ns prepared once (plan uploaded into `ws`); run() enqueues only the kernels."""

    def __init__(self, M_in, U_out, a, b, c, iters, G=None, beta=0.0, eps=1e-7, flags=0, Q_out=None, ws=None,
                 status=None, stream=None):
        self.tensors = (list(M_in), list(U_out), G, Q_out, status)  # keep the buffers alive
        if ws is None:
            ws = workspace(smuon_ns_workspace_bytes(M_in, iters, flags), M_in[0].device)
        self.ws = ws
        h = c_void_p()
        _check(lib().smuon_ns_plan_create(_mats(M_in), _mats(U_out), len(M_in), _mats(G), beta, a, b, c, iters, eps,
                                          flags, _mats(Q_out), ws.data_ptr(), ws.numel(), _ptr(status),
                                          _stream(stream), ctypes.byref(h)))
        self.handle = h

    def run(self, skip_if=None, stream=None):
        _check(lib().smuon_ns_execute(self.handle, _ptr(skip_if), _stream(stream)))

    def __del__(self):
        h = getattr(self, "handle", None)
        if h and _lib is not None:
            _lib.smuon_plan_destroy(h)
            self.handle = None


class UpdatePlan:
    """smuon_update prepared once; run() enqueues only the kernels."""

    def __init__(self, W, eta, U=None, votes=None, dense=None, M=1, tie_value=0, vote_kind=VOTE_POPCOUNT,
                 packed_out=None, vote_out=None, status=None):
        Uflat = None if U is None else [u for layer in U for u in layer]
        self.tensors = (None if W is None else list(W), Uflat, votes, dense, packed_out, vote_out, status)
        n = len(U) if W is None else len(W)  # W None: signs, message and votes only
        po = None if packed_out is None else (c_void_p * n)(*[_ptr(p) for p in packed_out])
        vo = None if vote_out is None else (c_void_p * n)(*[_ptr(v) for v in vote_out])
        h = c_void_p()
        _check(lib().smuon_update_plan_create(_mats(W), n, _mats(Uflat), _mats(votes), _mats(dense), M, eta,
                                              tie_value, vote_kind, po, vo, _ptr(status), ctypes.byref(h)))
        self.handle = h

    def run(self, stream=None):
        _check(lib().smuon_update_execute(self.handle, _stream(stream)))

    def __del__(self):
        h = getattr(self, "handle", None)
        if h and _lib is not None:
            _lib.smuon_plan_destroy(h)
            self.handle = None


# ---------------------------------------------------------------- sign / vote / update
def packed_words(n: int) -> int:
    return ((n + 127) // 128) * 4


def smuon_sign_pack(U, packed=None, signs_i8=None, stream=None):
    _check(lib().smuon_sign_pack(_mats(U), len(U), _ptr(packed), _ptr(signs_i8), _stream(stream)))


def smuon_vote(M: int, N: int, vote, packed=None, signs_i8=None, tie_value: int = 0, stream=None):
    _check(lib().smuon_vote(_ptr(packed), _ptr(signs_i8), M, N, tie_value, vote.data_ptr(), _stream(stream)))


def smuon_update(W, eta: float, U=None, votes=None, dense=None, M: int = 1, tie_value: int = 0,
                 vote_kind: int = VOTE_POPCOUNT, packed_out=None, vote_out=None, status=None, stream=None):
    """U is a list over layers of lists over workers (flattened worker-minor).
    W may be None with U and packed_out / vote_out: signs, message and votes only.
    status: optional device int32 tensor for SMUON_DEV_* bits."""
    Uflat = None if U is None else [u for layer in U for u in layer]
    n = len(U) if W is None else len(W)
    po = None if packed_out is None else (c_void_p * n)(*[_ptr(p) for p in packed_out])
    vo = None if vote_out is None else (c_void_p * n)(*[_ptr(v) for v in vote_out])
    _check(lib().smuon_update(_mats(W), n, _mats(Uflat), _mats(votes), _mats(dense), M, eta, tie_value,
                              vote_kind, po, vo, _ptr(status), _stream(stream)))


# ---------------------------------------------------------------- CacheMuon
def cachemuon_workspace_bytes(M_t) -> int:
    out = c_size_t(0)
    _check(lib().cachemuon_workspace_bytes(ctypes.byref(mat(M_t)), ctypes.byref(out)))
    return out.value


def new_counters(device=None) -> torch.Tensor:
    """Device storage for cachemuon_counters (4 x int64)."""
    return torch.zeros(4, dtype=torch.int64, device=device or "cuda")


def cachemuon_reuse_probe(Q, M_t, D_hat, gamma, err, accept, counters=None, eps=1e-7, ws=None, status=None,
                          stream=None):
    if ws is None:
        ws = workspace(cachemuon_workspace_bytes(M_t), M_t.device)
    qm = None if Q is None else ctypes.byref(mat(Q))
    _check(lib().cachemuon_reuse_probe(qm, ctypes.byref(mat(M_t)), ctypes.byref(mat(D_hat)), gamma, eps,
                                       err.data_ptr(), accept.data_ptr(), _ptr(counters), ws.data_ptr(),
                                       ws.numel(), _ptr(status), _stream(stream)))
    return ws


class CacheMuon:
    """CacheMuon schedule for one matrix, kept on the device: every step probes
    the cached transform (reuse D_hat = Q X_t, residual, accept flag) and then
    enqueues the fresh solve, whose kernels return at once when the flag says
    the cached transform was accepted. The host never waits on the GPU; read
    counters() at the end."""

    def __init__(self, M_t, D_out, gamma, coeffs, iters, flags=NS_SPLIT_BF16, eps=1e-7):
        dev = M_t.device
        m = min(M_t.shape)
        self.M, self.D, self.gamma, self.eps = M_t, D_out, float(gamma), eps
        self.Q = torch.zeros((m, m), dtype=torch.bfloat16, device=dev)
        self.err = torch.zeros(1, dtype=torch.float32, device=dev)
        self.accept = torch.zeros(1, dtype=torch.int32, device=dev)
        self.cnt = new_counters(dev)
        self.ws_probe = workspace(cachemuon_workspace_bytes(M_t), dev)
        self.fresh = NsPlan([M_t], [D_out], *coeffs, iters, flags=flags | NS_EMIT_Q, Q_out=[self.Q], eps=eps)
        self.steps = 0

    def probe(self, stream=None):
        """The step's probe: D_hat = Q X_t into D, its residual and the accept flag (no cache on the first step)."""
        cachemuon_reuse_probe(self.Q if self.steps > 0 else None, self.M, self.D, self.gamma, self.err, self.accept,
                              self.cnt, eps=self.eps, ws=self.ws_probe, stream=stream)

    def refresh(self, stream=None):
        """The step's fresh solve (D and Q), whose kernels return at once when the probe accepted."""
        self.fresh.run(skip_if=self.accept, stream=stream)
        self.steps += 1

    def step(self, stream=None):
        self.probe(stream)
        self.refresh(stream)

    def counters(self) -> dict:
        h, mi, pr, _ = self.cnt.tolist()
        return {"hits": h, "misses": mi, "probes": pr}


# ---------------------------------------------------------------- LionMuon
class LionMuon:
    """Holds the C lionmuon_state for lists W[layer] and mom[layer][worker].
    With `grad` (a GradStream), lionmuon_step may be called with G=None: the
    kernels then draw the workers' gradients from the counter-based streams."""

    def __init__(self, W, mom, t: int = 0, grad: GradStream | None = None):
        self.W = list(W)
        self.mom = [list(m) for m in mom]
        self.workers = len(self.mom[0])
        self._w = _mats(self.W)
        self._m = _mats([m for layer in self.mom for m in layer])
        self.grad = grad
        self.state = LionMuonState(len(self.W), self.workers, self._w, self._m, t,
                                   None if grad is None else ctypes.pointer(grad))

    @property
    def t(self) -> int:
        return self.state.t

    def workspace_bytes(self, iters: int, ns_flags: int = 0) -> int:
        out = c_size_t(0)
        _check(lib().lionmuon_workspace_bytes(ctypes.byref(self.state), iters, ns_flags, ctypes.byref(out)))
        return out.value


def lionmuon_step(opt: LionMuon, G, P, beta1, beta2, eta, a, b, c, iters, tie_value=0, ns_flags=0, ws=None,
                  status=None, stream=None):
    """G is a list over layers of lists over workers, or None to draw the
    gradients in-kernel from opt.grad at step t + 1. Returns the workspace used."""
    if ws is None:
        ws = workspace(opt.workspace_bytes(iters, ns_flags), opt.W[0].device)
    Gflat = None if G is None else _mats([g for layer in G for g in layer])
    _check(lib().lionmuon_step(ctypes.byref(opt.state), P, beta1, beta2, eta, a, b, c, iters, tie_value, ns_flags,
                               Gflat, ws.data_ptr(), ws.numel(), _ptr(status), _stream(stream)))
    return ws


def smuon_harness_gaussian(G, workers: int, stream_desc: GradStream, step: int, stream=None):
    """G: flat list [layer * workers + worker] of float32 matrices, filled
    with the counter-based gradient streams at `step`."""
    n = len(G)
    if n % workers:
        raise ValueError("len(G) must be a multiple of workers")
    _check(lib().smuon_harness_gaussian(_mats(G), n // workers, workers, ctypes.byref(stream_desc), step,
                                        _stream(stream)))


# ---------------------------------------------------------------- AdamW and gradient norm
_DT_TENSOR = {torch.float32: F32, torch.bfloat16: BF16, torch.float8_e4m3fn: E4M3}


_NO_TENSOR = (0, 0, 0, 0, F32, 0)


def _describe(t):
    """(data, rows, cols, ld, dtype, 0) of a tensor of any shape: contiguous, or 2-D with unit column stride."""
    dt = _DT_TENSOR.get(t.dtype)
    if dt is None:
        raise ValueError(f"dtype {t.dtype} is not supported")
    shape, n = t.shape, t.numel()
    if n == 0:
        return 0, 0, 0, 0, dt, 0
    if t.is_contiguous():
        cols = shape[-1] if shape else 1
        rows = n // cols
        if cols >= 1 << 31 or rows >= 1 << 31:
            raise ValueError("at most 2^31 - 1 rows and columns: view the tensor in another shape")
        return t.data_ptr(), rows, cols, cols, dt, 0
    if len(shape) != 2 or (t.stride(1) != 1 and shape[1] > 1) or (shape[0] > 1 and t.stride(0) < shape[1]):
        raise ValueError("tensors must be contiguous, or 2-D with unit column stride and rows that do not overlap")
    return t.data_ptr(), shape[0], shape[1], t.stride(0) if shape[0] > 1 else shape[1], dt, 0


def tensor(t) -> SmuonMat:
    """Describes a tensor for the AdamW calls: contiguous of any shape, or 2-D with unit column stride."""
    ptr, rows, cols, ld, dt, _ = _describe(t)
    return SmuonMat(ptr or None, rows, cols, ld, dt)


def _tensors(ts, shapes=None, name="G"):
    ts = list(ts)
    if shapes is not None:
        if len(ts) != len(shapes):
            raise ValueError(f"{len(ts)} tensors in {name}, {len(shapes)} weights")
        for i, (t, s) in enumerate(zip(ts, shapes)):
            if t is not None and t.shape != s:
                raise ValueError(f"{name}[{i}] has shape {tuple(t.shape)}, its weight {tuple(s)}")
    arr, flat = (SmuonMat * len(ts))(), []
    for t in ts:
        flat += _describe(t) if t is not None else _NO_TENSOR
    struct.pack_into("@" + "QiiqiI" * len(ts), arr, 0, *flat)  # the fields of each SmuonMat and its padding, at once
    return arr


def _one_device(*groups) -> torch.device:
    """The CUDA device that all tensors are on; ValueError otherwise."""
    devs = {t.device for g in groups if g is not None for t in g if t is not None}
    if len(devs) != 1 or next(iter(devs)).type != "cuda":
        raise ValueError(f"tensors must be on one CUDA device, got {sorted(map(str, devs))}")
    return next(iter(devs))


def _scalar(t, dtype, name):
    if t is not None and (t.dtype != dtype or t.numel() != 1):
        raise ValueError(f"{name} must be a {dtype} tensor of one element")
    return t


class AdamW:
    """Weights, moments and step count of an AdamW run over many tensors: the
    parameters beside the matrices that the Muon-type steps take, or a whole
    model.

    W             weights, float32 or bfloat16, any shapes (contiguous, or 2-D
                  with a row stride), updated in place by adamw_step
    bits          32: float32 moments. 8: E4M3 codes with one power-of-two
                  exponent per 256 entries, stochastically rounded from `seed`
                  and the step (include/smuon.h states the format)
    m, v, scales  existing moments instead of zeros (float32, or float8_e4m3fn
                  with uint8 `scales` of shape (ceil(entries / 256), 2); v then
                  holds the second moment's square root)
    master        True: a float32 original is kept for every bfloat16 weight
                  and stepped in its place; or a list of them (None: none)
    weight_decay, lr_scale   one number, or one per tensor
    t             steps taken
    device_step   keep the count on the device: a step that is skipped does not
                  count, and replays of a captured step count on
    """

    def __init__(self, W, m=None, v=None, scales=None, master=None, bits=32, weight_decay=0.0, lr_scale=1.0, seed=0,
                 t=0, device_step=False):
        self.W = list(W)
        n = len(self.W)
        shapes = [w.shape for w in self.W]
        if (m is None) != (v is None) or (m is None and scales is not None):
            raise ValueError("give m and v together (with scales for 8-bit moments), or none of them")
        if m is None:
            if bits not in (8, 32):
                raise ValueError("bits must be 8 or 32")
            kind = torch.float32 if bits == 32 else torch.float8_e4m3fn
            zeros = lambda: [torch.zeros(w.numel() * (4 if bits == 32 else 1), dtype=torch.uint8, device=w.device)  # noqa: E731
                             .view(kind).view(w.shape) for w in self.W]
            m, v = zeros(), zeros()
            if bits == 8:
                scales = [torch.zeros((-(-w.numel() // 256), 2), dtype=torch.uint8, device=w.device) for w in self.W]
        self.m, self.v = list(m), list(v)
        self.bits = 8 if self.m and self.m[0].dtype == torch.float8_e4m3fn else 32
        if (self.bits == 8) != (scales is not None):
            raise ValueError("scales go with 8-bit moments, and only with them")
        self.scales = None if scales is None else list(scales)
        if self.scales is not None:
            if len(self.scales) != n:
                raise ValueError(f"{len(self.scales)} scales, {n} weights")
            for i, (s, w) in enumerate(zip(self.scales, self.W)):
                if s.dtype != torch.uint8 or not s.is_contiguous() or s.numel() != 2 * -(-w.numel() // 256):
                    raise ValueError(f"scales[{i}] must be a contiguous uint8 tensor of shape (ceil(entries / 256), 2)")
        if master is True:
            master = [w.detach().float().contiguous() if w.dtype == torch.bfloat16 else None for w in self.W]
        self.master = None if not master else list(master)
        self.device = _one_device(self.W, self.m, self.v, self.scales, self.master)
        self._shapes = shapes
        per = lambda x: (c_float * n)(*(x if isinstance(x, (list, tuple)) else [x] * n))  # noqa: E731
        for x, name in ((weight_decay, "weight_decay"), (lr_scale, "lr_scale")):
            if isinstance(x, (list, tuple)) and len(x) != n:
                raise ValueError(f"{len(x)} values of {name}, {n} weights")
        self._arrays = (_tensors(self.W), None if self.master is None else _tensors(self.master, shapes, "master"),
                        _tensors(self.m, shapes, "m"), _tensors(self.v, shapes, "v"),
                        None if self.scales is None else (c_void_p * n)(*[s.data_ptr() for s in self.scales]),
                        per(lr_scale), per(weight_decay))
        self.d_t = torch.tensor([t, 0], dtype=torch.int64, device=self.device) if device_step else None
        W_, master_, m_, v_, scales_, ls_, wd_ = self._arrays
        self.state = AdamWState(n, seed, W_, master_, m_, v_, scales_, ls_, wd_, t, _ptr(self.d_t))

    @property
    def t(self) -> int:
        """Steps taken (with device_step: waits for the device)."""
        return self.state.t if self.d_t is None else int(self.d_t[0])


def _adamw_args(opt, G, lr, grad_scale, skip_if):
    G = list(G)
    d_lr = _scalar(lr, torch.float32, "lr") if isinstance(lr, torch.Tensor) else None
    _scalar(grad_scale, torch.float32, "grad_scale")
    _scalar(skip_if, torch.int32, "skip_if")
    mats = _tensors(G, opt._shapes)
    if _one_device(G, [d_lr, grad_scale, skip_if]) != opt.device:
        raise ValueError("the gradients are on another device than the weights")
    return mats, d_lr


def adamw_step(opt: AdamW, G, lr, beta1=0.9, beta2=0.999, eps=1e-8, grad_scale=None, skip_if=None, stream=None):
    """One AdamW step on all tensors of `opt`. G: gradients of the weights'
    shapes, float32 or bfloat16. lr: a number, or a one-element float32 device
    tensor read when the step runs. grad_scale: one-element float32 device
    tensor that multiplies the gradients (GradNorm.coef). skip_if: one-element
    int32 device tensor; nonzero leaves everything as it was (GradNorm.skip)."""
    mats, d_lr = _adamw_args(opt, G, lr, grad_scale, skip_if)
    with torch.cuda.device(opt.device):
        _check(lib().adamw_step(ctypes.byref(opt.state), mats, 0.0 if d_lr is not None else lr, beta1, beta2, eps,
                                _ptr(d_lr), _ptr(grad_scale), _ptr(skip_if), _stream(stream)))


class _Prepared:
    """A plan with its table in device memory. Its creation returns when the table has arrived there (it waits for the
    stream that was current then), so runs need no order against it: on any stream, captured or not. A graph that
    captured a run needs the plan as long as it is replayed."""
    handle = None

    def _uploading(self, device):
        """To be entered around the creation: its device, and no capture there (the upload would be the graph's)."""
        self._index = device.index
        with torch.cuda.device(device):
            if torch.cuda.is_current_stream_capturing():
                raise ValueError("prepare the plan before the capture: its table is uploaded once")
        return torch.cuda.device(device)

    def _uploaded(self, *own):
        stream = torch.cuda.current_stream()
        stream.synchronize()
        self._own, self._seen = own, {stream.cuda_stream}

    def _here(self, stream):
        """Handle of the stream to run on. The plan's device is current."""
        s = _raw_stream(self._index) if stream is None else _stream(stream)
        if s not in self._seen:
            self._hold(s)
        return s

    def _hold(self, s):
        stream = _torch_stream(s, self._index)
        for t in self._own:  # allocated on the stream of the creation: not reused before this one is done with them
            t.record_stream(stream)
        self._seen.add(s)

    def __del__(self):
        h = self.handle
        if h and _lib is not None:
            _lib.smuon_plan_destroy(h)
            self.handle = None


class AdamWPlan(_Prepared):
    """adamw_step prepared once, for gradients that keep their addresses; run()
    enqueues only the kernels. `lr` may be a device tensor here, or a number in run()."""

    def __init__(self, opt: AdamW, G, beta1=0.9, beta2=0.999, eps=1e-8, lr=None, grad_scale=None, skip_if=None):
        if lr is not None and not isinstance(lr, torch.Tensor):
            raise ValueError("lr must be a device tensor here: give a number to run()")
        mats, d_lr = _adamw_args(opt, G, lr, grad_scale, skip_if)
        self.opt, self.tensors = opt, (list(G), d_lr, grad_scale, skip_if)  # keep the buffers alive
        h, n = c_void_p(), c_size_t(0)
        with self._uploading(opt.device):
            _check(lib().adamw_plan_workspace_bytes(ctypes.byref(opt.state), ctypes.byref(n)))
            self.ws = workspace(n.value, opt.device)
            _check(lib().adamw_plan_create(ctypes.byref(opt.state), mats, beta1, beta2, eps, _ptr(d_lr),
                                           _ptr(grad_scale), _ptr(skip_if), self.ws.data_ptr(), self.ws.numel(),
                                           _stream(None), ctypes.byref(h)))
            self._uploaded(self.ws)
        self.handle, self._state, self._device_lr = h, ctypes.byref(opt.state), d_lr is not None
        self._execute = lib().adamw_execute

    def run(self, lr=None, stream=None):
        if (lr is None) != self._device_lr:
            raise ValueError("give lr once: as a device tensor to the plan, or as a number here")
        if _current_device() != self._index:
            with torch.cuda.device(self._index):
                return self.run(lr, stream)
        code = self._execute(self.handle, self._state, 0.0 if lr is None else lr, self._here(stream))
        if code:
            _check(code)


def adamw_convert(src: AdamW, dst: AdamW, stream=None):
    """dst's moments and step count <- src's, from 32 bits to 8 (rounded to nearest) or back."""
    if src.device != dst.device:
        raise ValueError("the two states are on different devices")
    with torch.cuda.device(src.device):
        _check(lib().adamw_convert(ctypes.byref(src.state), ctypes.byref(dst.state), _stream(stream)))


def smuon_grad_norm_workspace_bytes(G) -> int:
    G = list(G)
    out = c_size_t(0)
    _check(lib().smuon_grad_norm_workspace_bytes(_tensors(G), len(G), ctypes.byref(out)))
    return out.value


class GradNorm(_Prepared):
    """Global 2-norm of many gradients that keep their addresses, prepared once;
    run() enqueues one kernel. On the device afterwards: norm, coef = min(1,
    max_norm / (norm + 1e-6)) (float32 scalars) and skip (int32: 1 where the
    norm is not finite; coef is then 0)."""

    def __init__(self, G, max_norm: float, status=None):
        G = list(G)
        self.device = _one_device(G, [status])
        self.out = torch.zeros(2, dtype=torch.float32, device=self.device)
        self.norm, self.coef = self.out[0], self.out[1]
        self.skip = torch.zeros((), dtype=torch.int32, device=self.device)
        self.tensors = (G, _scalar(status, torch.int32, "status"))  # keep the buffers alive
        h, mats, n = c_void_p(), _tensors(G), c_size_t(0)
        with self._uploading(self.device):
            _check(lib().smuon_grad_norm_workspace_bytes(mats, len(G), ctypes.byref(n)))
            self.ws = workspace(n.value, self.device)
            _check(lib().smuon_grad_norm_plan_create(mats, len(G), max_norm, self.out.data_ptr(),
                                                     self.skip.data_ptr(), self.ws.data_ptr(), self.ws.numel(),
                                                     _ptr(status), _stream(None), ctypes.byref(h)))
            self._uploaded(self.ws, self.out, self.skip)
        self.handle, self._execute = h, lib().smuon_grad_norm_execute

    def run(self, stream=None):
        if _current_device() != self._index:
            with torch.cuda.device(self._index):
                return self.run(stream)
        code = self._execute(self.handle, self._here(stream))
        if code:
            _check(code)


def smuon_grad_norm(G, max_norm: float, out, skip=None, ws=None, status=None, stream=None):
    """The norm of G into out (float32, two elements: norm, clip factor) and the
    skip flag (int32), without a plan. Returns the workspace used (a given one: keep
    it until the work on `stream` is done)."""
    G = list(G)
    if out.dtype != torch.float32 or out.numel() != 2 or not out.is_contiguous():
        raise ValueError("out must be a contiguous float32 tensor of two elements")
    _scalar(skip, torch.int32, "skip")
    _scalar(status, torch.int32, "status")
    dev = _one_device(G, [out, skip, ws, status])
    if ws is None:
        n = smuon_grad_norm_workspace_bytes(G)
        # from the memory of the stream that uses it: work queued on the current stream may still be using that stream's
        with nullcontext() if stream is None else torch.cuda.stream(_torch_stream(_stream(stream), dev.index)):
            ws = workspace(n, dev)
    with torch.cuda.device(dev):
        _check(lib().smuon_grad_norm(_tensors(G), len(G), max_norm, out.data_ptr(), _ptr(skip), ws.data_ptr(),
                                     ws.numel(), _ptr(status), _stream(stream)))
    return ws
