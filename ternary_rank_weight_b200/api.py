"""Python binding of the ExTernD C ABI (include/externd.h).

Argument marshalling only: tensors are turned into pointers, every step of the
factorization runs in the CUDA library.  PyTorch provides device memory and
streams.  Inputs may live on the GPU (device pointers) or on the host (the
library stages them through device memory inside the call).
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass, field
from typing import Optional, Sequence

import numpy as np
import torch

from . import _lib


class ExterndError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {strerror(status)} (status {status})")


STATUS = {
    "OK": 0, "EINVAL": -1, "EZERO": -2, "ENONFINITE": -3, "ENOMEM": -4,
    "ECUDA": -5, "ELAUNCH": -6, "ETIMEOUT": -7, "ELIMIT": -8,
}


def strerror(status: int) -> str:
    return _lib.load().externd_strerror(int(status)).decode()


def rank(m: int, n: int, mu: float) -> int:
    return int(_lib.load().externd_rank(int(m), int(n), float(mu)))


def trit_bytes(length: int) -> int:
    return int(_lib.load().externd_trit_bytes(int(length)))


def last_stats() -> dict:
    st = _lib.Stats()
    _lib.load().externd_last_stats(ctypes.byref(st))
    return st.as_dict()


def _check(rc: int, what: str):
    if rc != 0:
        raise ExterndError(rc, what)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        return t.data_ptr()
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    raise TypeError(type(t))


def _stream(stream, device) -> int:
    if stream is not None:
        return int(getattr(stream, "cuda_stream", stream))
    if device is not None and device.type == "cuda":
        return torch.cuda.current_stream(device).cuda_stream
    if torch.cuda.is_available():
        return torch.cuda.current_stream().cuda_stream
    return 0


def _as_matrix(A) -> torch.Tensor:
    if isinstance(A, np.ndarray):
        A = torch.from_numpy(np.ascontiguousarray(A, dtype=np.float32))
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be a 2-D float32 tensor or array")
    if A.dtype != torch.float32:
        raise ValueError("A must be float32")
    return A.contiguous()


def _empty(shape, dtype, like: torch.Tensor) -> torch.Tensor:
    if like.is_cuda:
        return torch.empty(shape, dtype=dtype, device=like.device)
    return torch.empty(shape, dtype=dtype, pin_memory=like.is_pinned())


class _on_device:
    def __init__(self, t: torch.Tensor):
        self.ctx = torch.cuda.device(t.device) if t.is_cuda else None

    def __enter__(self):
        if self.ctx:
            self.ctx.__enter__()

    def __exit__(self, *a):
        if self.ctx:
            self.ctx.__exit__(*a)


@dataclass
class Factors:
    """B diag(D) C with packed ternary rows (2 bits per trit)."""
    B: torch.Tensor                 # uint8 [k, trit_bytes(m)]  row i = column i of B
    D: torch.Tensor                 # float32 [k]
    C: torch.Tensor                 # uint8 [k, trit_bytes(n)]  row i = row i of C
    energy: Optional[torch.Tensor]  # float64 [k]
    m: int
    n: int
    k: int
    mu: float
    tau: float
    d64: Optional[torch.Tensor] = None
    stats: dict = field(default_factory=dict)
    sweep_energy: Optional[torch.Tensor] = None   # float64 [sweeps]: energy after each refinement sweep
    trace: Optional["Trace"] = None               # test hook: traced half-steps (factor(..., trace=...))

    def trits(self):
        """Unpacked (B as m x k int8, C as k x n int8) on the host."""
        Bu = unpack_trits(self.B.cpu().numpy(), self.m).T.copy()
        Cu = unpack_trits(self.C.cpu().numpy(), self.n)
        return Bu, Cu


@dataclass
class Trace:
    """Half-steps of components [first, first + count) as the kernel saw them (test hook).

    pre_v[c, t] / pre_u[c, t]: the published output of the t-th V-step (x = R^T u, length n)
    and U-step (y = R v, length m) of component first + c; thr_*: the thresholds; trit_*:
    the packed trits those half-steps produced."""
    first: int
    count: int
    pre_v: torch.Tensor
    thr_v: torch.Tensor
    trit_v: torch.Tensor
    pre_u: torch.Tensor
    thr_u: torch.Tensor
    trit_u: torch.Tensor

    @staticmethod
    def alloc(first: int, count: int, iters: int, m: int, n: int, device) -> "Trace":
        """Buffers pre-filled with NaN, so half-steps a visit did not run stay recognisable."""
        nan = dict(fill_value=float("nan"), dtype=torch.float64, device=device)
        return Trace(first, count,
                     torch.full((count, iters, n), **nan), torch.full((count, iters), **nan),
                     torch.zeros((count, iters, trit_bytes(n)), dtype=torch.uint8, device=device),
                     torch.full((count, iters, m), **nan), torch.full((count, iters), **nan),
                     torch.zeros((count, iters, trit_bytes(m)), dtype=torch.uint8, device=device))


def factor(A, mu: float, tau: float, iters: int = 15, seed: int = 0, *, grid: int = 0, pending: int = 0,
           wait_limit_s: float = 0.0, fault_skip_cta: Optional[int] = None, want_d64: bool = False,
           want_energy: bool = True, sweeps: int = 0, h=None, lam: float = 0.0, trace=None, cluster: int = 0,
           block: int = 0, async_status=None, stream=None) -> Factors:
    """Factor one matrix (externd_factor_ex).  Outputs are allocated where A lives.

    sweeps: §2.4 refinement sweeps after extraction (``energy`` keeps the extraction
    energies, ``sweep_energy`` the energy after each sweep).  h, lam: §2.5 importance
    weights (per-column second moments, n float32 values), or None for the plain objective.
    trace: (first, count) -- test hook, records the half-steps of those visits: visit
    i < k extracts component i, visit (s + 1) k + i is sweep s's refit of component i
    (``Factors.trace``; A must be on the GPU).  cluster: kernel choice (0 automatic, 1 one
    CTA per residual stripe, 2/4/8/16 the clustered kernel with that cluster size).
    block: threads per CTA (0 automatic, 256, 512 or 1024); the same grid, cluster and block
    give the same bits.
    async_status: a one-element int32 CUDA tensor: the call queues its work and returns at
    once; the tensor receives the status (0 or a negative code) when the stream gets there.
    A (and h) must then be contiguous float32 CUDA tensors, which the queued work reads until
    the stream reaches its end: keep them alive and unchanged until then (the outputs are the
    returned tensors).  ``stats`` then holds the launch plan only."""
    if async_status is not None:
        _check_async_inputs([A], h, async_status)
    A = _as_matrix(A)
    m, n = A.shape
    if h is not None:
        h = _weights(h, n)
    k = rank(m, n, mu)
    if k < 1:
        raise ExterndError(STATUS["EINVAL"], "externd_rank")
    B = _empty((k, trit_bytes(m)), torch.uint8, A)
    C = _empty((k, trit_bytes(n)), torch.uint8, A)
    D = _empty((k,), torch.float32, A)
    E = _empty((k,), torch.float64, A) if want_energy else None
    d64 = _empty((k,), torch.float64, A) if want_d64 else None
    opt = _lib.Options()
    opt.grid = int(grid)
    opt.pending = int(pending)
    opt.wait_limit_s = float(wait_limit_s)
    opt.fault_inject = 1 if fault_skip_cta is not None else 0
    opt.fault_skip_cta = int(fault_skip_cta) if fault_skip_cta is not None else -1
    opt.d64_out = _ptr(d64)
    SE = _empty((int(sweeps),), torch.float64, A) if sweeps > 0 else None
    opt.sweeps = int(sweeps)
    opt.sweep_energy_out = _ptr(SE)
    opt.h = _ptr(h)
    opt.lambda_ = float(lam)
    opt.cluster = int(cluster)
    opt.block = int(block)
    if async_status is not None:
        opt.async_status = _ptr(async_status)
    tr = None
    if trace is not None:
        if not A.is_cuda:
            raise ValueError("trace needs A on the GPU")
        tr = Trace.alloc(int(trace[0]), int(trace[1]), int(iters), m, n, A.device)
        opt.trace_first, opt.trace_count = tr.first, tr.count
        opt.trace_pre_v, opt.trace_thr_v, opt.trace_trit_v = _ptr(tr.pre_v), _ptr(tr.thr_v), _ptr(tr.trit_v)
        opt.trace_pre_u, opt.trace_thr_u, opt.trace_trit_u = _ptr(tr.pre_u), _ptr(tr.thr_u), _ptr(tr.trit_u)
    with _on_device(A):
        rc = _lib.load().externd_factor_ex(_ptr(A), m, n, float(mu), float(tau), int(iters), int(seed),
                                           _ptr(B), _ptr(D), _ptr(C), _ptr(E),
                                           _stream(stream, A.device), ctypes.byref(opt))
    _check(rc, "externd_factor")
    return Factors(B=B, D=D, C=C, energy=E, m=m, n=n, k=k, mu=float(mu), tau=float(tau), d64=d64,
                   stats=last_stats(), sweep_energy=SE, trace=tr)


def _check_async_inputs(As, h, async_status, hs=None):
    """An asynchronous call reads its inputs after it returns: they must be the caller's own
    tensors (contiguous float32 on the GPU, so no temporary copy is made) and the status an
    int32 CUDA tensor."""
    if not (isinstance(async_status, torch.Tensor) and async_status.is_cuda and async_status.dtype == torch.int32
            and async_status.numel() >= 1):
        raise ValueError("async_status must be an int32 CUDA tensor")
    ins = list(As) + ([h] if h is not None else []) + (list(hs) if hs is not None else [])
    for t in ins:
        if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == torch.float32 and t.is_contiguous()):
            raise ValueError("an asynchronous call needs contiguous float32 CUDA tensors as inputs")


def _weights(h, n: int) -> torch.Tensor:
    if isinstance(h, np.ndarray):
        h = torch.from_numpy(np.ascontiguousarray(h, dtype=np.float32))
    if not isinstance(h, torch.Tensor) or h.dtype != torch.float32 or h.numel() != n:
        raise ValueError("h must hold n float32 values")
    return h.contiguous()


def factor_weighted(A, h, mu: float, tau: float, lam: float = 0.0, iters: int = 15, seed: int = 0, *,
                    stream=None) -> Factors:
    """Importance-weighted factorization (externd_factor_weighted, §2.5).

    h: per-column second moments (n,), float32, on the host or the GPU.  The returned
    energy is the weighted energy.  (Refinement sweeps with weights: ``factor(..., h=h, sweeps=S)``.)"""
    A = _as_matrix(A)
    m, n = A.shape
    h = _weights(h, n)
    k = rank(m, n, mu)
    if k < 1:
        raise ExterndError(STATUS["EINVAL"], "externd_rank")
    B = _empty((k, trit_bytes(m)), torch.uint8, A)
    C = _empty((k, trit_bytes(n)), torch.uint8, A)
    D = _empty((k,), torch.float32, A)
    E = _empty((k,), torch.float64, A)
    with _on_device(A):
        rc = _lib.load().externd_factor_weighted(_ptr(A), m, n, float(mu), float(tau), int(iters), int(seed), _ptr(h),
                                                 float(lam), _ptr(B), _ptr(D), _ptr(C), _ptr(E),
                                                 _stream(stream, A.device))
    _check(rc, "externd_factor_weighted")
    return Factors(B=B, D=D, C=C, energy=E, m=m, n=n, k=k, mu=float(mu), tau=float(tau), stats=last_stats())


def factor_noalloc(A: torch.Tensor, mu: float, tau: float, iters: int = 15, seed: int = 0, *, out=None,
                   stream=None) -> Factors:
    """externd_factor_noalloc: the same factorization with no device allocation inside the call.

    For callers that cannot allocate device memory while the factorization runs
    (e.g. a service whose pool already reserved the GPU).  The library's scratch is
    a fixed static device array (``NOALLOC_SCRATCH_BYTES``); larger shapes are
    rejected (ELIMIT).  A and the outputs must live on the GPU; pass preallocated
    outputs as ``out=(B, D, C, energy)`` to keep this call allocation-free on the
    Python side too.  Calls share the scratch and must not overlap on the GPU."""
    if not (isinstance(A, torch.Tensor) and A.is_cuda and A.dtype == torch.float32 and A.dim() == 2):
        raise ValueError("A must be a 2-D float32 CUDA tensor")
    if not A.is_contiguous():
        # a contiguous copy would be an allocation on the caller's side
        raise ValueError("A must be contiguous (row-major): factor_noalloc makes no copies")
    m, n = A.shape
    k = rank(m, n, mu)
    if k < 1:
        raise ExterndError(STATUS["EINVAL"], "externd_rank")
    if out is None:
        out = (torch.empty((k, trit_bytes(m)), dtype=torch.uint8, device=A.device),
               torch.empty((k,), dtype=torch.float32, device=A.device),
               torch.empty((k, trit_bytes(n)), dtype=torch.uint8, device=A.device),
               torch.empty((k,), dtype=torch.float64, device=A.device))
    B, D, C, E = out
    with _on_device(A):
        rc = _lib.load().externd_factor_noalloc(_ptr(A), m, n, float(mu), float(tau), int(iters), int(seed),
                                                _ptr(B), _ptr(D), _ptr(C), _ptr(E), _stream(stream, A.device))
    _check(rc, "externd_factor_noalloc")
    return Factors(B=B, D=D, C=C, energy=E, m=m, n=n, k=k, mu=float(mu), tau=float(tau))


NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


def factor_block(A: torch.Tensor, mu: float, tau: float, iters: int = 15, seed: int = 0, *, b: int = 0,
                 want_d64: bool = False, stream=None) -> Factors:
    """§2.4 batched block ALS with decorrelated targets (externd_factor_block); b = 0 takes the
    pages' default width (256 capped at min(m, n) / 8).  A must be a float32 CUDA tensor."""
    if not (isinstance(A, torch.Tensor) and A.is_cuda and A.dtype == torch.float32 and A.dim() == 2):
        raise ValueError("A must be a 2-D float32 CUDA tensor")
    A = A.contiguous()
    m, n = A.shape
    k = rank(m, n, mu)
    if k < 1:
        raise ExterndError(STATUS["EINVAL"], "externd_rank")
    B = torch.empty((k, trit_bytes(m)), dtype=torch.uint8, device=A.device)
    C = torch.empty((k, trit_bytes(n)), dtype=torch.uint8, device=A.device)
    D = torch.empty((k,), dtype=torch.float32, device=A.device)
    E = torch.empty((k,), dtype=torch.float64, device=A.device)
    d64 = torch.empty((k,), dtype=torch.float64, device=A.device) if want_d64 else None
    with _on_device(A):
        rc = _lib.load().externd_factor_block(_ptr(A), m, n, float(mu), float(tau), int(iters), int(seed), int(b),
                                              _ptr(B), _ptr(D), _ptr(C), _ptr(E), _ptr(d64), _stream(stream, A.device))
    _check(rc, "externd_factor_block")
    return Factors(B=B, D=D, C=C, energy=E, m=m, n=n, k=k, mu=float(mu), tau=float(tau), d64=d64, stats=last_stats())


def factor_batched(As: Sequence, mus: Sequence[float], taus: Sequence[float], iters: int = 15,
                   seeds: Optional[Sequence[int]] = None, *, hs: Optional[Sequence] = None,
                   lams: Optional[Sequence[float]] = None, sweeps: int = 0, grid: int = 0, cluster: int = 0,
                   block: int = 0, plan_only: bool = False, async_status=None, stream=None):
    """Factor independent matrices in one launch (externd_factor_batched_ex).

    hs: per-matrix importance weights (§2.5; every matrix or none), lams their lambdas;
    sweeps: refinement sweeps (§2.4) for every matrix; grid, cluster, block: the launch (0:
    automatic; a matrix gets the same bits from any launch with the same three).  plan_only: return (None, stats of the plan) without device work.
    async_status: a one-element int32 CUDA tensor: queue the work and return at once; the
    tensor receives the batch's status when the stream gets there.  Every matrix (and weight
    vector) must then be a contiguous float32 CUDA tensor, kept alive and unchanged until then.
    Returns (list of Factors, list of per-matrix status codes)."""
    if async_status is not None:
        _check_async_inputs(As, None, async_status, hs)
    mats = [_as_matrix(a) for a in As]
    cnt = len(mats)
    if seeds is None:
        seeds = list(range(cnt))
    outs = []
    for A, mu, tau in zip(mats, mus, taus):
        m, n = A.shape
        k = rank(m, n, mu)
        if k < 1:
            raise ExterndError(STATUS["EINVAL"], "externd_rank")
        outs.append((_empty((k, trit_bytes(m)), torch.uint8, A), _empty((k,), torch.float32, A),
                     _empty((k, trit_bytes(n)), torch.uint8, A), _empty((k,), torch.float64, A), k))
    P = ctypes.c_void_p * cnt
    a_ptrs = P(*[_ptr(a) for a in mats])
    b_ptrs = P(*[_ptr(o[0]) for o in outs])
    d_ptrs = P(*[_ptr(o[1]) for o in outs])
    c_ptrs = P(*[_ptr(o[2]) for o in outs])
    e_ptrs = P(*[_ptr(o[3]) for o in outs])
    ms = (ctypes.c_int64 * cnt)(*[a.shape[0] for a in mats])
    ns = (ctypes.c_int64 * cnt)(*[a.shape[1] for a in mats])
    mu_a = (ctypes.c_double * cnt)(*[float(x) for x in mus])
    tau_a = (ctypes.c_double * cnt)(*[float(x) for x in taus])
    seed_a = (ctypes.c_uint64 * cnt)(*[int(s) for s in seeds])
    st = (ctypes.c_int * cnt)()
    opt = _lib.BatchOptions()
    keep = []   # ctypes arrays and tensors that must outlive the call
    if hs is not None:
        hts = [_weights(h, A.shape[1]) for h, A in zip(hs, mats)]
        harr = P(*[_ptr(h) for h in hts])
        keep += [hts, harr]
        opt.h = ctypes.cast(harr, ctypes.c_void_p)
        if lams is not None:
            larr = (ctypes.c_double * cnt)(*[float(x) for x in lams])
            keep.append(larr)
            opt.lambda_ = ctypes.cast(larr, ctypes.c_void_p)
    SEs = [_empty((int(sweeps),), torch.float64, A) if sweeps > 0 else None for A in mats]
    opt.sweeps = int(sweeps)
    opt.grid = int(grid)
    opt.cluster = int(cluster)
    opt.block = int(block)
    opt.plan_only = 1 if plan_only else 0
    if async_status is not None:
        opt.async_status = _ptr(async_status)
    if sweeps > 0:
        sarr = P(*[_ptr(x) for x in SEs])
        keep.append(sarr)
        opt.sweep_energy_out = ctypes.cast(sarr, ctypes.c_void_p)
    with _on_device(mats[0]):
        rc = _lib.load().externd_factor_batched_ex(cnt, a_ptrs, ms, ns, mu_a, tau_a, int(iters), seed_a,
                                                   b_ptrs, d_ptrs, c_ptrs, e_ptrs, st,
                                                   _stream(stream, mats[0].device), ctypes.byref(opt))
    stats = last_stats()
    if plan_only:
        _check(rc, "externd_factor_batched_ex")
        return None, stats
    res = []
    for A, mu, tau, o, se in zip(mats, mus, taus, outs, SEs):
        res.append(Factors(B=o[0], D=o[1], C=o[2], energy=o[3], m=A.shape[0], n=A.shape[1], k=o[4],
                           mu=float(mu), tau=float(tau), stats=stats, sweep_energy=se))
    statuses = list(st)
    if rc != 0 and all(s == 0 for s in statuses):
        _check(rc, "externd_factor_batched_ex")
    return res, statuses


def reconstruct(B: torch.Tensor, D: torch.Tensor, C: torch.Tensor, m: int, n: int, *, stream=None) -> torch.Tensor:
    """Ahat = B diag(D) C as an m x n float32 tensor on B's device."""
    k = D.shape[0]
    out = _empty((m, n), torch.float32, B)
    with _on_device(B):
        rc = _lib.load().externd_reconstruct(_ptr(B), _ptr(D), _ptr(C), int(m), int(n), int(k), _ptr(out),
                                             _stream(stream, B.device))
    _check(rc, "externd_reconstruct")
    return out


def debug_halfstep(R, trits_in: torch.Tensor, tau: float, transpose: bool, *, stream=None):
    """One V-step (transpose=True: x = R^T u) or U-step (y = R v) through the ALS kernel.

    Returns (pre-threshold fp64 vector, threshold, packed output trits)."""
    R = _as_matrix(R)
    m, n = R.shape
    lout = n if transpose else m
    pre = _empty((lout,), torch.float64, R)
    thr = _empty((1,), torch.float64, R)
    out = _empty((trit_bytes(lout),), torch.uint8, R)
    with _on_device(R):
        rc = _lib.load().externd_debug_halfstep(_ptr(R), m, n, 1 if transpose else 0, _ptr(trits_in), float(tau),
                                                _ptr(pre), _ptr(thr), _ptr(out), _stream(stream, R.device))
    _check(rc, "externd_debug_halfstep")
    return pre, float(thr[0].item()), out


def debug_component(R, u0: torch.Tensor, tau: float, iters: int = 15, *, pend_d=None, pend_u=None, pend_v=None,
                    grid: int = 0, stream=None):
    """One component of §2.3 on a given residual state (externd_debug_component, test hook).

    R: m x n float32 (GPU); u0: packed start trits (GPU); pend_d / pend_u / pend_v: pending
    rank-1 terms (fp64 scales, packed u rows, packed v rows, all on the GPU) that the kernel
    applies as lazy-deflation corrections.  Returns (Trace with count 1, d64, packed u, packed v)."""
    R = _as_matrix(R)
    m, n = R.shape
    dev = R.device
    tr = Trace.alloc(0, 1, int(iters), m, n, dev)
    D = torch.empty((1,), dtype=torch.float32, device=dev)
    d64 = torch.empty((1,), dtype=torch.float64, device=dev)
    uo = torch.empty((1, trit_bytes(m)), dtype=torch.uint8, device=dev)
    vo = torch.empty((1, trit_bytes(n)), dtype=torch.uint8, device=dev)
    npend = 0 if pend_d is None else int(pend_d.shape[0])
    with _on_device(R):
        rc = _lib.load().externd_debug_component(
            _ptr(R), m, n, float(tau), int(iters), _ptr(u0), npend, _ptr(pend_d), _ptr(pend_u), _ptr(pend_v),
            _ptr(tr.pre_v), _ptr(tr.thr_v), _ptr(tr.trit_v), _ptr(tr.pre_u), _ptr(tr.thr_u), _ptr(tr.trit_u),
            _ptr(D), _ptr(d64), _ptr(uo), _ptr(vo), int(grid), _stream(stream, dev))
    _check(rc, "externd_debug_component")
    return tr, float(d64[0].item()), uo[0], vo[0]


def debug_start_trits(m: int, k: int, tau: float, seed: int, device="cuda", *, stream=None) -> torch.Tensor:
    """Packed start trits of components 0..k-1 (k x trit_bytes(m)), generated on the GPU."""
    out = torch.empty((k, trit_bytes(m)), dtype=torch.uint8, device=device)
    with _on_device(out):
        rc = _lib.load().externd_debug_start_trits(int(m), int(k), float(tau), int(seed), _ptr(out),
                                                   _stream(stream, out.device))
    _check(rc, "externd_debug_start_trits")
    return out


@contextlib.contextmanager
def debug_wait_fault(withhold: int, wait_limit_s: float = 0.05):
    """Within: the gated block's and the 4-bit products' tile kernels, called from this thread, do not make the products
    of worker `withhold` (counted from 1), so that the waits for them run out (externd_debug_wait_fault)."""
    L = _lib.load()
    _check(L.externd_debug_wait_fault(float(wait_limit_s), int(withhold)), "externd_debug_wait_fault")
    try:
        yield
    finally:
        L.externd_debug_wait_fault(0.0, 0)


# ---------------------------------------------------------------------------
# host codecs of the packed 2-bit format: 00 = 0, 01 = +1, 11 = -1
# ---------------------------------------------------------------------------

def unpack_trits(packed: np.ndarray, length: int) -> np.ndarray:
    """uint8 rows (..., nbytes) -> int8 (..., length)."""
    p = np.asarray(packed, dtype=np.uint8)
    shifts = np.array([0, 2, 4, 6], dtype=np.uint8)
    codes = (p[..., :, None] >> shifts) & 3
    codes = codes.reshape(*p.shape[:-1], p.shape[-1] * 4)[..., :length]
    out = np.zeros(codes.shape, dtype=np.int8)
    out[codes == 1] = 1
    out[codes == 3] = -1
    return out


def pack_trits(t: np.ndarray) -> np.ndarray:
    """int8 (..., length) in {-1, 0, 1} -> uint8 (..., trit_bytes(length))."""
    t = np.asarray(t, dtype=np.int8)
    length = t.shape[-1]
    nb = trit_bytes(length)
    codes = np.zeros((*t.shape[:-1], nb * 4), dtype=np.uint8)
    codes[..., :length][t == 1] = 1
    codes[..., :length][t == -1] = 3
    codes = codes.reshape(*t.shape[:-1], nb, 4)
    return (codes[..., 0] | (codes[..., 1] << 2) | (codes[..., 2] << 4) | (codes[..., 3] << 6)).astype(np.uint8)


# ---------------------------------------------------------------------------
# inference with the factors and mask+sign storage (§2.6)
# ---------------------------------------------------------------------------

def transpose_trits(T: torch.Tensor, rows: int, length: int, *, stream=None) -> torch.Tensor:
    """(rows x length) packed trits -> (length x rows) packed trits, on T's device."""
    out = torch.empty((length, trit_bytes(rows)), dtype=torch.uint8, device=T.device)
    with _on_device(T):
        rc = _lib.load().externd_transpose_trits(_ptr(T), int(rows), int(length), _ptr(out), _stream(stream, T.device))
    _check(rc, "externd_transpose_trits")
    return out


def inference_layout(f: "Factors") -> torch.Tensor:
    """B laid out for inference: m rows x trit_bytes(k), row r = B[r, 0..k)."""
    return transpose_trits(f.B, f.k, f.m)


def matvec(Bt: torch.Tensor, D: torch.Tensor, C: torch.Tensor, m: int, n: int, X: torch.Tensor, *,
           out: Optional[torch.Tensor] = None, z_work: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y = B diag(D) C X for X of shape (batch, n) or (n,), fp32 on the GPU (externd_matvec)."""
    k = D.shape[0]
    squeeze = X.dim() == 1
    X2 = X.reshape(1, -1) if squeeze else X
    if X2.dtype != torch.float32 or not X2.is_cuda:
        raise ValueError("X must be a float32 CUDA tensor")
    X2 = X2.contiguous()
    batch = X2.shape[0]
    Y = out if out is not None else torch.empty((batch, m), dtype=torch.float32, device=X2.device)
    Z = z_work if z_work is not None else torch.empty((min(batch, 8), k), dtype=torch.float32, device=X2.device)
    with _on_device(X2):
        rc = _lib.load().externd_matvec(_ptr(Bt), _ptr(D), _ptr(C), int(m), int(n), int(k), _ptr(X2), int(batch),
                                        _ptr(Y), _ptr(Z), _stream(stream, X2.device))
    _check(rc, "externd_matvec")
    return Y.reshape(-1) if squeeze else Y


def pack_mask_sign(T: torch.Tensor, rows: int, length: int, *, stream=None):
    """Mask+sign storage of packed trit rows: (mask bytes rows x ceil(length/8),
    sign bit stream as int32 words, bit offsets per row (rows + 1))."""
    mask = torch.empty((rows, (length + 7) // 8), dtype=torch.uint8, device=T.device)
    words = max(1, (rows * length + 31) // 32)
    signs = torch.empty((words,), dtype=torch.int32, device=T.device)
    offs = torch.empty((rows + 1,), dtype=torch.int64, device=T.device)
    with _on_device(T):
        rc = _lib.load().externd_pack_mask_sign(_ptr(T), int(rows), int(length), _ptr(mask), _ptr(signs), int(words),
                                                _ptr(offs), _stream(stream, T.device))
    _check(rc, "externd_pack_mask_sign")
    total = int(offs[-1].item())
    return mask, signs[: (total + 31) // 32], offs


# ---------------------------------------------------------------------------
# 4-bit weights with group scales
# ---------------------------------------------------------------------------

_DTYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_SIZE = {torch.float32: 4, torch.float16: 2, torch.bfloat16: 2}
ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu2": 3}


_NOTHING = contextlib.nullcontext()


def _guard(stream, device: torch.device):
    """Make `device` current, and `stream` if one is given: the memory of temporaries and outputs must belong
    to the stream the kernels run on, for torch's allocator hands it to later work of that stream only.
    Results of a call with `stream` are ready for, and belong to, that stream."""
    if stream is None:
        return _NOTHING if device.index == torch.cuda.current_device() else torch.cuda.device(device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=device)
    if stream.device != device:
        raise ValueError("the stream and the tensors must belong to one device")
    return torch.cuda.stream(stream)


# the current stream's handle without building a Stream object (3 us of a call's 11), where torch offers it
_handle_of = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _rows_in(t, cols: int, name: str) -> torch.Tensor:
    """A 2-D CUDA tensor with `cols` columns of unit stride (copied otherwise) and one of the element
    types; rows may be strided."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or not t.is_cuda or t.dtype not in _DTYPE:
        raise ValueError(f"{name} must be a 2-D float32, float16 or bfloat16 CUDA tensor")
    rows, width = t.shape
    if width != cols:
        raise ValueError(f"{name} must have {cols} columns, not {width}")
    if rows:
        ld, step = t.stride()
        if (step != 1 and cols > 1) or (rows > 1 and ld < cols):
            return t.contiguous()
    return t


def _ld(t: torch.Tensor) -> int:
    """Leading dimension (that of a single row may be anything)."""
    rows, cols = t.shape
    return t.stride(0) if rows > 1 else max(cols, 1)


def _result(out, rows: int, cols: int, like: torch.Tensor) -> torch.Tensor:
    if out is None:
        return like.new_empty((rows, cols))
    if (not isinstance(out, torch.Tensor) or out.shape != (rows, cols) or out.dtype != like.dtype
            or out.device != like.device or (cols > 1 and out.stride(1) != 1)
            or (rows > 1 and out.stride(0) < cols)):
        raise ValueError(f"out must be a {rows} x {cols} {like.dtype} tensor on {like.device} with unit column stride")
    return out


def _overlap(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether two matrices with unit column stride may share memory.  Side by side in the rows of one buffer (equal
    row strides) they do not."""
    if a.numel() == 0 or b.numel() == 0 or a.device != b.device:
        return False
    (pa, ra, la, wa), (pb, rb, lb, wb) = ((t.data_ptr(), t.shape[0], _ld(t) * t.element_size(), t.shape[1] * t.element_size())
                                          for t in (a, b))
    if pa + (ra - 1) * la + wa <= pb or pb + (rb - 1) * lb + wb <= pa:
        return False
    if ra > 1 and rb > 1 and la == lb:
        d = (pb - pa) % la                       # where b's rows start within a's period
        return d < wa or d + wb > la
    return True


def _check_apart(out, *inputs):
    if any(_overlap(out, t) for t in inputs):
        raise ValueError("out must not share memory with the inputs: they are still read while it is written")


def _operand(t, cols: int, name: str, dtype: torch.dtype, device: torch.device):
    """A 2-D operand (copied where its columns are not of unit stride): the tensor, its address, its leading
    dimension and the workspace it takes if its rows do not start on 16-byte boundaries
    (externd_aligned_bytes)."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be a 2-D {dtype} tensor on {device}")
    rows, width = t.shape
    if width != cols:
        raise ValueError(f"{name} must have {cols} columns, not {width}")
    ld, step = t.stride()
    if rows and ((step != 1 and cols > 1) or (rows > 1 and ld < cols)):
        t = t.contiguous()
        ld = cols
    if rows < 2:
        ld = cols
    ptr, size = t.data_ptr(), _SIZE[dtype]
    if ptr & 15 or (rows > 1 and ld * size & 15):
        return t, ptr, ld, (rows * ((cols * size + 15) // 16 * 16) + 255) // 256 * 256
    return t, ptr, ld, 0


def _flat(t: torch.Tensor) -> torch.Tensor:
    return t if t.dim() == 2 else t.reshape(-1, t.shape[-1])


def _check_out(out, shape):
    if (not isinstance(out, torch.Tensor) or out.shape != shape or (out.dim() > 2 and not out.is_contiguous())):
        raise ValueError(f"out must have shape {shape} (and be contiguous with more than two dimensions)")


def _act(act: str) -> int:
    if act not in ACTS:
        raise ValueError(f"act must be one of {', '.join(ACTS)}")
    return ACTS[act]


def int4_row_bytes(n: int) -> int:
    return int(_lib.load().externd_int4_row_bytes(int(n)))


@dataclass
class Int4Weights:
    """An m x n matrix in 4 bits: w = scale (q - 8) + offset."""
    q: torch.Tensor                  # uint8 [m, int4_row_bytes(n)] (pack_int4 gives the layout)
    scale: torch.Tensor              # float16 [ceil(n / group), m]
    offset: Optional[torch.Tensor]   # float16 [ceil(n / group), m]; None: symmetric
    m: int
    n: int
    group: int                       # 32, 64 or 128 columns

    def codes(self) -> np.ndarray:
        """q on the host, m x n uint8."""
        return unpack_int4(self.q.cpu().numpy(), self.n)


def _check_int4(w: Int4Weights, device: torch.device):
    if not isinstance(w, Int4Weights):
        raise ValueError("4-bit matrices are given as Int4Weights")
    m, n, group = w.m, w.n, w.group
    if m < 1 or n < 1 or group not in (32, 64, 128):
        raise ValueError("Int4Weights need m, n >= 1 and groups of 32, 64 or 128 columns")
    q, scale, offset = w.q, w.scale, w.offset
    if not isinstance(q, torch.Tensor) or not isinstance(scale, torch.Tensor) or not (offset is None or isinstance(offset, torch.Tensor)):
        raise ValueError("q, scale and offset must be tensors (offset may be None)")
    scales = ((n + group - 1) // group, m)
    if q.dtype != torch.uint8 or q.shape != (m, (n + 127) // 128 * 64) or q.device != device or not q.is_contiguous():
        raise ValueError(f"q must be a contiguous uint8 tensor of {m} rows of int4_row_bytes({n}) on {device}")
    for t in (scale,) if offset is None else (scale, offset):
        if t.dtype != torch.float16 or t.shape != scales or t.device != device or not t.is_contiguous():
            raise ValueError(f"scale and offset must be contiguous float16 tensors of shape {scales} on {device}")


def int4_quantize(A: torch.Tensor, group: int = 128, *, affine: bool = True, async_status=None,
                  stream=None) -> Int4Weights:
    """Round a matrix to 4 bits with fp16 scales (and, affine, offsets) per row and group of columns
    (externd_int4_quantize).  A: 2-D float32, float16 or bfloat16 CUDA tensor.

    async_status: a one-element int32 CUDA tensor: the call queues its work and returns at once; the
    tensor receives the status when the stream gets there.  A must then need no copy (unit column
    stride) and stay alive and unchanged until then."""
    if not isinstance(A, torch.Tensor) or A.dim() != 2 or not A.is_cuda or A.numel() == 0:
        raise ValueError("A must be a 2-D float32, float16 or bfloat16 CUDA tensor that is not empty")
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    dev = A.device
    _check_status(async_status, dev)
    with _guard(stream, dev):
        A2 = _rows_in(A, A.shape[1], "A")
        if async_status is not None and A2 is not A:
            raise ValueError("an asynchronous call needs A with unit column stride")
        m, n = A2.shape
        groups = (n + group - 1) // group
        q = torch.empty((m, (n + 127) // 128 * 64), dtype=torch.uint8, device=dev)
        scale = torch.empty((groups, m), dtype=torch.float16, device=dev)
        offset = torch.empty((groups, m), dtype=torch.float16, device=dev) if affine else None
        rc = _lib.load().externd_int4_quantize(A2.data_ptr(), _DTYPE[A2.dtype], m, n, _ld(A2), int(group), q.data_ptr(),
                                               scale.data_ptr(), _ptr(offset), _ptr(async_status), _handle_of(dev.index))
    _check(rc, "externd_int4_quantize")
    return Int4Weights(q=q, scale=scale, offset=offset, m=m, n=n, group=int(group))


def int4_dequantize(w: Int4Weights, dtype: torch.dtype = torch.float32, *, stream=None) -> torch.Tensor:
    """The m x n matrix that the 4 bits stand for, rounded once to dtype (externd_int4_dequantize)."""
    if not isinstance(w, Int4Weights) or not isinstance(w.q, torch.Tensor) or not w.q.is_cuda:
        raise ValueError("w must be Int4Weights on the GPU")
    if dtype not in _DTYPE:
        raise ValueError("dtype must be float32, float16 or bfloat16")
    dev = w.q.device
    _check_int4(w, dev)
    with _guard(stream, dev):
        out = torch.empty((w.m, w.n), dtype=dtype, device=dev)
        rc = _lib.load().externd_int4_dequantize(w.q.data_ptr(), w.scale.data_ptr(), _ptr(w.offset), w.m, w.n, w.group,
                                                 out.data_ptr(), _DTYPE[dtype], w.n, _handle_of(dev.index))
    _check(rc, "externd_int4_dequantize")
    return out


def int4_matvec(w: Int4Weights, X: torch.Tensor, *, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y = X W^T for X of shape (..., n), in X's element type (externd_int4_matvec); out must not share memory with
    X."""
    return _int4_products((w,), X, 0, out, stream)


def int4_gated(wg: Int4Weights, wu: Int4Weights, X: torch.Tensor, act: str = "silu", *,
               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """H = act(X Wg^T) * (X Wu^T) for X of shape (..., n), in X's element type
    (externd_int4_gated); act: "silu", "gelu", "gelu_tanh" or "relu2"; out must not share memory with X."""
    if isinstance(wg, Int4Weights) and isinstance(wu, Int4Weights) and (wg.m, wg.n, wg.group) != (wu.m, wu.n, wu.group):
        raise ValueError("both matrices must have the same shape and group")
    return _int4_products((wg, wu), X, _act(act), out, stream)


def _int4_products(ws, X, act: int, out, stream) -> torch.Tensor:
    if not isinstance(X, torch.Tensor) or not X.is_cuda or X.dtype not in _DTYPE:
        raise ValueError("X must be a float32, float16 or bfloat16 CUDA tensor")
    dev, dtype, w = X.device, X.dtype, ws[0]
    mats = []
    for w in ws:
        _check_int4(w, dev)
        mats += (w.q.data_ptr(), w.scale.data_ptr(), None if w.offset is None else w.offset.data_ptr())
    two = X.dim() == 2
    if not two and (X.dim() < 1 or X.shape[-1] != w.n):
        raise ValueError(f"X's last dimension must be {w.n}")
    if out is not None:
        _check_out(out, (*X.shape[:-1], w.m))
    with _guard(stream, dev):
        X2, x, ldx, nbytes = _operand(X if two else _flat(X), w.n, "X", dtype, dev)
        batch = X2.shape[0]
        if out is None:
            Y = X2.new_empty((batch, w.m))
        else:
            Y = _result(out.view(-1, w.m), batch, w.m, X2)
            _check_apart(Y, X2)
        work = None
        if nbytes and batch > 8:
            work = torch.empty((nbytes,), dtype=torch.uint8, device=dev)
        tail = (x, _DTYPE[dtype], ldx, batch, Y.data_ptr(), w.m if out is None else _ld(Y), _ptr(work),
                0 if work is None else nbytes, _handle_of(dev.index))
        if len(ws) == 1:
            rc = _lib.load().externd_int4_matvec(*mats, w.m, w.n, w.group, *tail)
        else:
            rc = _lib.load().externd_int4_gated(*mats, w.m, w.n, w.group, act, *tail)
    _check(rc, "externd_int4_matvec" if len(ws) == 1 else "externd_int4_gated")
    return Y if two else Y.view((*X.shape[:-1], w.m))


def _int4_places(n: int):
    """Byte and shift of each column's nibble within a row."""
    j = np.arange(n)
    t, c, i, blk = j % 8, j // 8 % 4, j // 32 % 4, j // 128
    nib = 4 * (t % 2) + t // 2
    return 64 * blk + 4 * (4 * c + i) + nib // 2, (4 * (nib % 2)).astype(np.uint8)


def unpack_int4(packed: np.ndarray, n: int) -> np.ndarray:
    """uint8 rows (..., int4_row_bytes(n)) -> uint8 codes (..., n), 0..15."""
    byte, shift = _int4_places(n)
    return (np.asarray(packed, dtype=np.uint8)[..., byte] >> shift) & 15


def pack_int4(codes: np.ndarray) -> np.ndarray:
    """Codes 0..15 (..., n) -> uint8 (..., int4_row_bytes(n)); padding columns hold 8."""
    codes = np.asarray(codes, dtype=np.uint8)
    n = codes.shape[-1]
    full = np.full((*codes.shape[:-1], (n + 127) // 128 * 128), 8, dtype=np.uint8)
    full[..., :n] = codes
    byte, shift = _int4_places(full.shape[-1])
    out = np.zeros((*codes.shape[:-1], int4_row_bytes(n)), dtype=np.uint8)
    low = shift == 0
    out[..., byte[low]] = full[..., low]
    out[..., byte[~low]] |= full[..., ~low] << np.uint8(4)
    return out


# ---------------------------------------------------------------------------
# gated feed-forward block with dense weights
# ---------------------------------------------------------------------------

def _check_status(async_status, device):
    if async_status is not None and not (isinstance(async_status, torch.Tensor) and async_status.device == device
                                         and async_status.dtype == torch.int32 and async_status.numel() >= 1):
        raise ValueError("async_status must be an int32 CUDA tensor on the other tensors' device")


def _gated_inputs(X, Wg, Wu):
    if not isinstance(Wg, torch.Tensor) or Wg.dim() != 2 or Wg.numel() == 0:
        raise ValueError("Wg must be a 2-D float16 or bfloat16 CUDA tensor")
    m, n = Wg.shape
    if not isinstance(X, torch.Tensor) or not X.is_cuda or X.dim() < 1 or X.shape[-1] != n:
        raise ValueError(f"X must be a CUDA tensor whose last dimension is {n}")
    if X.dtype != torch.bfloat16 and X.dtype != torch.float16:
        raise ValueError("X, Wg and Wu must be float16 or bfloat16")
    if not isinstance(Wu, torch.Tensor) or Wu.shape != Wg.shape:
        raise ValueError("Wg and Wu must have the same shape")
    return m, n, X.device, X.dtype


def _gated(X, Wg, Wu, act, save, out, async_status, stream):
    m, n, dev, dtype = _gated_inputs(X, Wg, Wu)
    code = _act(act)
    _check_status(async_status, dev)
    two = X.dim() == 2
    shape = (X.shape[0], m) if two else (*X.shape[:-1], m)
    if out is not None:
        _check_out(out, shape)
    if save is not None and save != torch.float32 and save != dtype:
        raise ValueError("the projections can be saved in float32 or in X's type")
    with _guard(stream, dev):
        X2, x, ldx, bx = _operand(_flat(X), n, "X", dtype, dev)
        Wg, wg, ldg, bg = _operand(Wg, n, "Wg", dtype, dev)
        Wu, wu, ldu, bu = _operand(Wu, n, "Wu", dtype, dev)
        t = X2.shape[0]
        H = _result(None if out is None else out.view(-1, m), t, m, X2)
        if out is not None:
            _check_apart(H, X2, Wg, Wu)
        G = U = None
        lds = m
        if save is not None:
            # rows on 16-byte boundaries: the kernels store and load them whole
            lds = (m + 7) // 8 * 8
            G, U = X2.new_empty((t, lds), dtype=save), X2.new_empty((t, lds), dtype=save)
            if lds != m:
                G, U = G[:, :m], U[:, :m]
        nbytes = bx + bg + bu
        work = torch.empty((nbytes,), dtype=torch.uint8, device=dev) if nbytes else None
        kept = t and save is not None
        rc = _lib.load().externd_gated(x, ldx, wg, ldg, wu, ldu, _DTYPE[dtype], m, n, t, code, H.data_ptr(),
                                       m if out is None else _ld(H), G.data_ptr() if kept else None,
                                       U.data_ptr() if kept else None, _DTYPE[save or dtype], lds, _ptr(work), nbytes,
                                       _ptr(async_status), _handle_of(dev.index))
    _check(rc, "externd_gated")
    if two:
        return H, G, U
    return H.view(shape), None if G is None else G.view(shape), None if U is None else U.view(shape)


def gated(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, act: str = "silu", *, out: Optional[torch.Tensor] = None,
          async_status=None, stream=None) -> torch.Tensor:
    """H = act(X Wg^T) * (X Wu^T) for X of shape (..., n) and Wg, Wu of shape (m, n), float16 or bfloat16
    (externd_gated); act: "silu", "gelu", "gelu_tanh" or "relu2".  Operands whose rows do not start on 16-byte
    boundaries are copied first; out must not share memory with them.  The call is asynchronous; autograd does not record it (gated_forward and
    gated_backward are the training pair).  async_status: an int32 CUDA tensor that receives the status."""
    return _gated(X, Wg, Wu, act, None, out, async_status, stream)[0]


def gated_forward(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, act: str = "silu", *,
                  save_dtype: torch.dtype = torch.float32, async_status=None, stream=None):
    """(H, G, U): gated() with the projections G = X Wg^T and U = X Wu^T that gated_backward needs, in
    float32, or in X's type (half the memory; their rounding then adds to the gradients' errors).  G's and
    U's rows start on 16-byte boundaries: with m not a multiple of 8 they are not contiguous."""
    if save_dtype is None:
        raise ValueError("the projections can be saved in float32 or in X's type")
    return _gated(X, Wg, Wu, act, save_dtype, None, async_status, stream)


def gated_backward(dH: torch.Tensor, X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, G: torch.Tensor, U: torch.Tensor,
                   act: str = "silu", *, need=(True, True, True), async_status=None, stream=None):
    """(dX, dWg, dWu) from the gradient dH of gated_forward's H and the G and U it returned
    (externd_gated_backward); need: which of the three to compute (None in place of the others).  Infinite entries of
    G and U (projections past 65504 saved in float16) count as the type's largest value."""
    m, n, dev, dtype = _gated_inputs(X, Wg, Wu)
    code = _act(act)
    _check_status(async_status, dev)
    two = X.dim() == 2
    shape = (X.shape[0], m) if two else (*X.shape[:-1], m)
    for name, v in (("dH", dH), ("G", G), ("U", U)):
        if not isinstance(v, torch.Tensor) or v.shape != shape:
            raise ValueError(f"{name} must have shape {shape}")
    saved = G.dtype
    if saved != torch.float32 and saved != dtype:
        raise ValueError("G and U must both be float32 or both of X's type")
    with _guard(stream, dev):
        X2, x, ldx, bx = _operand(_flat(X), n, "X", dtype, dev)
        Wg, wg, ldg, bg = _operand(Wg, n, "Wg", dtype, dev)
        Wu, wu, ldu, bu = _operand(Wu, n, "Wu", dtype, dev)
        dH2, dh, lddh, _ = _operand(_flat(dH), m, "dH", dtype, dev)
        G2, g, lds, _ = _operand(_flat(G), m, "G", saved, dev)
        U2, u, ldu2, _ = _operand(_flat(U), m, "U", saved, dev)
        if lds != ldu2:
            G2, U2 = G2.contiguous(), U2.contiguous()
            g, u, lds = G2.data_ptr(), U2.data_ptr(), m
        t = X2.shape[0]
        dX = X2.new_empty((t, n)) if need[0] else None
        dWg = X2.new_empty((m, n)) if need[1] else None
        dWu = X2.new_empty((m, n)) if need[2] else None
        nbytes = 0
        if t and (need[0] or need[1] or need[2]):
            nbytes = (_lib.load().externd_gated_backward_work(m, n, t) + (bg + bu if need[0] else 0)
                      + (bx if need[1] or need[2] else 0))
        work = torch.empty((nbytes,), dtype=torch.uint8, device=dev) if nbytes else None
        rc = _lib.load().externd_gated_backward(dh, lddh, x, ldx, wg, ldg, wu, ldu, g, u, _DTYPE[saved], lds, _DTYPE[dtype], m, n,
                                                t, code, _ptr(dX), n, _ptr(dWg), _ptr(dWu), n, _ptr(work), nbytes,
                                                _ptr(async_status), _handle_of(dev.index))
    _check(rc, "externd_gated_backward")
    return (dX if two or dX is None else dX.view(X.shape)), dWg, dWu
