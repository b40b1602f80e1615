"""ctypes binding of ``libcce.so`` (declared in ``include/cce.h``).

Argument marshalling only: every step of the head runs in the library's CUDA
kernels.  Tensors are torch CUDA tensors (used for device memory and
streams); the functions keep the C names and raise ``CCEError`` for a
synchronous error status.  The library is loaded on first use; if it is
missing the call raises instead of falling back to anything else.
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libcce.so")

CCE_F32, CCE_BF16 = 0, 1
CCE_W_DENSE, CCE_W_AFFINE_Q4_G64, CCE_W_AFFINE_Q8_G64 = 0, 1, 2
SCOPE = {"full": 0, "response": 1}
VOCAB_BLOCK = 256

STATUS_NAMES = {
    0: "CCE_OK", 1: "CCE_ERR_INVALID_ARGUMENT", 2: "CCE_ERR_UNSUPPORTED",
    3: "CCE_ERR_CUDA", 4: "CCE_ERR_WORKSPACE_TOO_SMALL",
    5: "CCE_ERR_LABEL_OUT_OF_RANGE", 6: "CCE_ERR_DEVICE_TIMEOUT",
    7: "CCE_ERR_EMPTY_SEGMENT", 8: "CCE_ERR_DOMAIN", 9: "CCE_ERR_FP16_RANGE",
}


class CCEError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")
        self.status = status


class _Head(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int), ("dtype", ctypes.c_int),
                ("V", ctypes.c_int64), ("D", ctypes.c_int64),
                ("w", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("biases", ctypes.c_void_p), ("softcap", ctypes.c_float)]


class _Objective(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("lam", ctypes.c_double), ("beta", ctypes.c_double),
                ("gamma", ctypes.c_double), ("sft_scope", ctypes.c_int)]


OBJECTIVES = {"orpo": 0, "simpo": 1, "orpo_margin": 2}


class _Layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "prompt_begin", "prompt_end", "chosen_begin", "chosen_end",
        "rejected_begin", "rejected_end")]


class _Plan(ctypes.Structure):
    _fields_ = [("fwd_ok", ctypes.c_int), ("bwd_ok", ctypes.c_int),
                ("fwd_chunk", ctypes.c_int64), ("bwd_chunk", ctypes.c_int64),
                ("bwd_ksplit", ctypes.c_int),
                ("fwd_staged", ctypes.c_int), ("bwd_staged", ctypes.c_int),
                ("fwd_cta_pairs", ctypes.c_int), ("bwd_cta_pairs", ctypes.c_int),
                ("bwd_fused", ctypes.c_int), ("bwd_fused_groups", ctypes.c_int),
                ("bwd_fused_members", ctypes.c_int), ("bwd_fused_buffers", ctypes.c_int),
                ("bwd_sliced", ctypes.c_int), ("bwd_sliced_clusters", ctypes.c_int),
                ("bwd_sliced_ctas", ctypes.c_int), ("fwd_q_small_m", ctypes.c_int)]


_lib = None

_SIGS = {
    "cce_blockmax_cols": (ctypes.c_int64, [ctypes.c_int64]),
    "cce_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int, ctypes.POINTER(_Head)]),
    "cce_workspace_min_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int, ctypes.POINTER(_Head)]),
    "cce_forward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.POINTER(_Head),
                                   ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                   ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "orpo_loss_from_logps": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                            ctypes.POINTER(_Layout), ctypes.c_double, ctypes.c_int,
                                            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                            ctypes.c_void_p]),
    "orpo_grad_coeffs": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                        ctypes.POINTER(_Layout), ctypes.c_double, ctypes.c_int,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                        ctypes.c_void_p]),
    "orpo_partial_sums": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                         ctypes.POINTER(_Layout), ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_size_t, ctypes.c_void_p]),
    "orpo_from_sums": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                      ctypes.POINTER(_Layout), ctypes.c_double, ctypes.c_int,
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_size_t, ctypes.c_void_p]),
    "cce_backward_dh": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.POINTER(_Head),
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_size_t, ctypes.c_void_p]),
    "cce_backward_dh_dw": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                          ctypes.POINTER(_Head), ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p,
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "cce_device_status": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "cce_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "cce_set_wait_limit_ns": (None, [ctypes.c_uint64]),
    "cce_set_cta_pairs": (None, [ctypes.c_int]),
    "cce_set_quant_staging": (None, [ctypes.c_int]),
    "cce_set_backward_mode": (None, [ctypes.c_int]),
    "cce_set_forward_mode": (None, [ctypes.c_int]),
    "cce_query_fused_schedule": (ctypes.c_int64, [ctypes.c_int64, ctypes.c_int,
                                                  ctypes.POINTER(_Head), ctypes.c_void_p,
                                                  ctypes.c_int64]),
    "cce_query_plan": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int, ctypes.POINTER(_Head),
                                      ctypes.c_size_t, ctypes.POINTER(_Plan)]),
    "cce_selftest_wait_timeout": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "pref_loss_from_logps": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                            ctypes.POINTER(_Layout), ctypes.POINTER(_Objective),
                                            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                            ctypes.c_void_p]),
    "pref_grad_coeffs": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                        ctypes.POINTER(_Layout), ctypes.POINTER(_Objective),
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                        ctypes.c_void_p]),
    "cce_prefix_gather": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                         ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                         ctypes.c_void_p, ctypes.c_void_p]),
    "cce_prefix_scatter": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                          ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                          ctypes.c_void_p]),
    "cce_fp8_quant_rows": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                          ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                          ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p]),
    "cce_fp8_quant_blocks": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                            ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                            ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p]),
    "cce_fp8_matmul": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                      ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                      ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                      ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "cce_sample_rows": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                       ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_void_p]),
    "cce_norm_forward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                        ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                        ctypes.c_int, ctypes.c_double, ctypes.c_void_p,
                                        ctypes.c_int, ctypes.c_int64, ctypes.c_void_p,
                                        ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p]),
    "cce_norm_backward_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    "cce_norm_backward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                         ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                         ctypes.c_int, ctypes.c_int64, ctypes.c_void_p,
                                         ctypes.c_int, ctypes.c_int64, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "cce_profile_enable": (None, [ctypes.c_int]),
    "cce_profile_read": (ctypes.c_int, [ctypes.POINTER(ctypes.c_double),
                                        ctypes.POINTER(ctypes.c_longlong), ctypes.c_int]),
    "cce_profile_kind_name": (ctypes.c_char_p, [ctypes.c_int]),
    "cce_forward_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(_Head),
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_void_p]),
}

NOALLOC_SCRATCH_BYTES = 32 << 20


def cce_forward_noalloc(H, head: "Head", labels, logp, lse, tgt_logit=None, blockmax=None,
                        status=None, stream=None):
    """Forward for callers that cannot allocate device memory: the library's
    fixed scratch array (NOALLOC_SCRATCH_BYTES) replaces the workspace.
    Calls share that array, so calls that overlap on the GPU race."""
    st = lib().cce_forward_noalloc(_p(H), H.shape[0], ctypes.byref(head.c()), _p(labels),
                                   _p(logp), _p(lse), _p(tgt_logit), _p(blockmax), _p(status),
                                   _stream(stream))
    _check(st, "cce_forward_noalloc")

PROFILE_KINDS = 32


def cce_profile_enable(on: bool):
    lib().cce_profile_enable(1 if on else 0)


def cce_profile_read() -> dict:
    """{kind name: (total ms, launches)} of the kernels recorded since
    ``cce_profile_enable(True)``; clears the records."""
    ms = (ctypes.c_double * PROFILE_KINDS)()
    n = (ctypes.c_longlong * PROFILE_KINDS)()
    k = lib().cce_profile_read(ms, n, PROFILE_KINDS)
    return {lib().cce_profile_kind_name(i).decode(): (ms[i], n[i])
            for i in range(min(k, PROFILE_KINDS))}


def lib():
    """Load ``libcce.so`` once; raise if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m lm_head_cross_flash_b200.build` (no fallback exists)")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _lib = l
    return _lib


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(st: int, where: str):
    if st != 0:
        raise CCEError(st, where)


@dataclass
class Head:
    """The frozen head: dense ``w`` [V, D] (f32 or bf16), or a 4-bit affine
    head (``w`` uint32 [V, D/8] stored as int32, ``scales``/``biases`` bf16
    [V, D/64])."""

    w: torch.Tensor
    V: int
    D: int
    fmt: int = CCE_W_DENSE
    scales: torch.Tensor | None = None
    biases: torch.Tensor | None = None
    softcap: float = 0.0

    @property
    def dtype(self) -> int:
        if self.fmt in (CCE_W_AFFINE_Q4_G64, CCE_W_AFFINE_Q8_G64):
            return CCE_BF16
        return CCE_F32 if self.w.dtype == torch.float32 else CCE_BF16

    def c(self) -> _Head:
        return _Head(self.fmt, self.dtype, self.V, self.D, self.w.data_ptr(),
                     None if self.scales is None else self.scales.data_ptr(),
                     None if self.biases is None else self.biases.data_ptr(),
                     float(self.softcap))


def h_dtype(H: torch.Tensor) -> int:
    return CCE_F32 if H.dtype == torch.float32 else CCE_BF16


def blockmax_cols(V: int) -> int:
    return int(lib().cce_blockmax_cols(V))


def workspace_bytes(M: int, H_dtype: int, head: Head) -> int:
    return int(lib().cce_workspace_bytes(M, H_dtype, ctypes.byref(head.c())))


def workspace_min_bytes(M: int, H_dtype: int, head: Head) -> int:
    return int(lib().cce_workspace_min_bytes(M, H_dtype, ctypes.byref(head.c())))


def alloc_workspace(M: int, H_dtype: int, head: Head, device="cuda", nbytes=None):
    """Caller-side workspace (torch allocation) with a zeroed status word."""
    n = workspace_bytes(M, H_dtype, head) if nbytes is None else nbytes
    if n == 0:
        raise CCEError(1, "cce_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def cce_forward(H, head: Head, labels, logp, lse, tgt_logit=None, blockmax=None,
                ws=None, stream=None):
    st = lib().cce_forward(_p(H), h_dtype(H), H.shape[0], ctypes.byref(head.c()),
                           _p(labels), _p(logp), _p(lse), _p(tgt_logit), _p(blockmax),
                           _p(ws), ws.numel(), _stream(stream))
    _check(st, "cce_forward")


def _layout(layout):
    return _Layout(*[int(x) for x in layout])


def orpo_loss_from_logps(logp, labels, layout, lam, sft_scope, out8, ws, stream=None):
    st = lib().orpo_loss_from_logps(_p(logp), _p(labels), logp.shape[0],
                                    ctypes.byref(_layout(layout)), float(lam),
                                    SCOPE.get(sft_scope, sft_scope), _p(out8), _p(ws),
                                    ws.numel(), _stream(stream))
    _check(st, "orpo_loss_from_logps")


def orpo_grad_coeffs(logp, labels, layout, lam, sft_scope, coeff, ws, stream=None):
    st = lib().orpo_grad_coeffs(_p(logp), _p(labels), logp.shape[0],
                                ctypes.byref(_layout(layout)), float(lam),
                                SCOPE.get(sft_scope, sft_scope), _p(coeff), _p(ws),
                                ws.numel(), _stream(stream))
    _check(st, "orpo_grad_coeffs")


def orpo_partial_sums(logp, labels, layout, sums6, ws, stream=None):
    """This shard's segment sums and counts (fp64 [6] on the device)."""
    st = lib().orpo_partial_sums(_p(logp), _p(labels), logp.shape[0],
                                 ctypes.byref(_layout(layout)), _p(sums6), _p(ws), ws.numel(),
                                 _stream(stream))
    _check(st, "orpo_partial_sums")


def orpo_from_sums(sums6, labels, layout, lam, sft_scope, out8, coeff, ws, stream=None):
    """Loss and this shard's dL/dlogp from the all-reduced segment sums."""
    st = lib().orpo_from_sums(_p(sums6), _p(labels), labels.shape[0],
                              ctypes.byref(_layout(layout)), float(lam),
                              SCOPE.get(sft_scope, sft_scope), _p(out8), _p(coeff), _p(ws),
                              ws.numel(), _stream(stream))
    _check(st, "orpo_from_sums")


def cce_backward_dh(H, head: Head, labels, lse, coeff, filter_eps, blockmax, dH,
                    skip_stats=None, ws=None, stream=None):
    st = lib().cce_backward_dh(_p(H), h_dtype(H), H.shape[0], ctypes.byref(head.c()),
                               _p(labels), _p(lse), _p(coeff), float(filter_eps),
                               _p(blockmax), _p(dH), _p(skip_stats), _p(ws), ws.numel(),
                               _stream(stream))
    _check(st, "cce_backward_dh")


def cce_device_status(ws, stream=None) -> int:
    return int(lib().cce_device_status(_p(ws), _stream(stream)))


def cce_set_wait_limit_ns(ns: int):
    lib().cce_set_wait_limit_ns(int(ns))


def cce_selftest_wait_timeout(ws, stream=None):
    _check(lib().cce_selftest_wait_timeout(_p(ws), ws.numel(), _stream(stream)),
           "cce_selftest_wait_timeout")


# ----------------------------------------------------------------------------
# one pass of the whole head
# ----------------------------------------------------------------------------

@dataclass
class HeadBuffers:
    """Device buffers of one head pass (outputs and the workspace)."""

    logp: torch.Tensor
    lse: torch.Tensor
    tgt: torch.Tensor
    blockmax: torch.Tensor
    out8: torch.Tensor
    coeff: torch.Tensor
    dH: torch.Tensor
    skip: torch.Tensor
    ws: torch.Tensor

    @staticmethod
    def alloc(M: int, D: int, V: int, H_dtype: int, head: Head, device="cuda",
              ws_bytes=None):
        f = dict(device=device, dtype=torch.float32)
        return HeadBuffers(
            logp=torch.empty(M, **f), lse=torch.empty(M, **f), tgt=torch.zeros(M, **f),
            blockmax=torch.empty(blockmax_cols(V), M, **f),
            out8=torch.empty(8, device=device, dtype=torch.float64),
            coeff=torch.empty(M, **f), dH=torch.empty(M, D, **f),
            skip=torch.zeros(2, device=device, dtype=torch.int64),
            ws=alloc_workspace(M, H_dtype, head, device, ws_bytes))


def orpo_head_pass(H, head: Head, labels, layout, lam, sft_scope, filter_eps,
                   block_skip: bool, buf: HeadBuffers, stream=None):
    """Forward, ORPO loss, cotangent and dH, all enqueued on one stream."""
    cce_forward(H, head, labels, buf.logp, buf.lse, buf.tgt, buf.blockmax, buf.ws, stream)
    orpo_loss_from_logps(buf.logp, labels, layout, lam, sft_scope, buf.out8, buf.ws, stream)
    orpo_grad_coeffs(buf.logp, labels, layout, lam, sft_scope, buf.coeff, buf.ws, stream)
    cce_backward_dh(H, head, labels, buf.lse, buf.coeff, filter_eps,
                    buf.blockmax if block_skip else None, buf.dH, buf.skip, buf.ws, stream)


def orpo_head_pass_sharded(H, head: Head, labels, layout, lam, sft_scope, filter_eps,
                           block_skip: bool, buf: HeadBuffers, group=None, stream=None):
    """One pair split by rows over the processes of ``group`` (one per GPU):
    this process holds some rows of each segment (``layout`` in its own row
    numbering).  Forward, then one all-reduce of the six segment sums, then
    the loss, this shard's cotangent and its dH rows.  The all-reduce runs on
    the device for NCCL and through host memory for gloo."""
    import torch.distributed as dist
    s = torch.cuda.current_stream() if stream is None else stream
    cce_forward(H, head, labels, buf.logp, buf.lse, buf.tgt, buf.blockmax, buf.ws, s)
    sums = torch.zeros(6, dtype=torch.float64, device=H.device)
    orpo_partial_sums(buf.logp, labels, layout, sums, buf.ws, s)
    if dist.get_backend(group) == "nccl":
        with torch.cuda.stream(s):
            dist.all_reduce(sums, group=group)
    else:
        s.synchronize()
        host = sums.cpu()
        dist.all_reduce(host, group=group)
        with torch.cuda.stream(s):
            sums.copy_(host)
    orpo_from_sums(sums, labels, layout, lam, sft_scope, buf.out8, buf.coeff, buf.ws, s)
    cce_backward_dh(H, head, labels, buf.lse, buf.coeff, filter_eps,
                    buf.blockmax if block_skip else None, buf.dH, buf.skip, buf.ws, s)


class HeadPassGraph:
    """``orpo_head_pass`` captured once into a CUDA graph and replayed.

    The library allocates nothing and never synchronises inside a call, and
    every launch goes to the stream it is given, so the whole pass (forward,
    merge, loss, cotangent, backward) is one graph.  The graph keeps the
    addresses of ``H``, ``labels`` and ``buf``: copy each step's inputs into
    those tensors, then ``replay()``.  The settings read at capture time
    (CTA pairs, quantised-head staging, the wait limit) are frozen into the
    graph.  Profiling must be off while capturing.
    """

    def __init__(self, H, head: Head, labels, layout, lam, sft_scope, filter_eps,
                 block_skip: bool, buf: HeadBuffers):
        self.args = (H, head, labels, layout, lam, sft_scope, filter_eps, block_skip, buf)
        side = torch.cuda.Stream(device=H.device)
        side.wait_stream(torch.cuda.current_stream(H.device))
        with torch.cuda.stream(side):  # first call outside the capture: one-time setup
            orpo_head_pass(*self.args, stream=side)
        torch.cuda.current_stream(H.device).wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            orpo_head_pass(*self.args, stream=torch.cuda.current_stream(H.device))

    def replay(self):
        self.graph.replay()


def upload_workload(wl, device="cuda"):
    """Device tensors (H, Head, labels) of a ``synthetic.Workload``."""
    import numpy as np
    if wl.dtype == "bf16":
        H = torch.from_numpy(wl.H_bits.view(np.int16)).to(device).view(torch.bfloat16)
    else:
        H = torch.from_numpy(wl.H).to(device)
    if wl.wformat in ("q4g64", "q8g64"):
        head = Head(w=torch.from_numpy(wl.q_packed.view(np.int32)).to(device), V=wl.V, D=wl.D,
                    fmt=CCE_W_AFFINE_Q4_G64 if wl.wformat == "q4g64" else CCE_W_AFFINE_Q8_G64,
                    scales=torch.from_numpy(wl.q_scales.view(np.int16)).to(device).view(torch.bfloat16),
                    biases=torch.from_numpy(wl.q_biases.view(np.int16)).to(device).view(torch.bfloat16))
    elif wl.dtype == "bf16":
        head = Head(w=torch.from_numpy(wl.W_bits.view(np.int16)).to(device).view(torch.bfloat16),
                    V=wl.V, D=wl.D)
    else:
        head = Head(w=torch.from_numpy(wl.W).to(device), V=wl.V, D=wl.D)
    labels = torch.from_numpy(wl.labels).to(device)
    return H, head, labels


def _objective(kind, lam, beta, gamma, sft_scope):
    return _Objective(OBJECTIVES.get(kind, kind), float(lam), float(beta), float(gamma),
                      SCOPE.get(sft_scope, sft_scope))


def pref_loss_from_logps(logp, labels, layout, kind, lam, beta, gamma, sft_scope, out8, ws,
                         stream=None):
    st = lib().pref_loss_from_logps(_p(logp), _p(labels), logp.shape[0],
                                    ctypes.byref(_layout(layout)),
                                    ctypes.byref(_objective(kind, lam, beta, gamma, sft_scope)),
                                    _p(out8), _p(ws), ws.numel(), _stream(stream))
    _check(st, "pref_loss_from_logps")


def pref_grad_coeffs(logp, labels, layout, kind, lam, beta, gamma, sft_scope, coeff, ws,
                     stream=None):
    st = lib().pref_grad_coeffs(_p(logp), _p(labels), logp.shape[0],
                                ctypes.byref(_layout(layout)),
                                ctypes.byref(_objective(kind, lam, beta, gamma, sft_scope)),
                                _p(coeff), _p(ws), ws.numel(), _stream(stream))
    _check(st, "pref_grad_coeffs")


def cce_prefix_gather(H_cat, P, Rc, Rr, H_head, stream=None):
    _check(lib().cce_prefix_gather(_p(H_cat), h_dtype(H_cat), P, Rc, Rr, H_cat.shape[1],
                                   _p(H_head), _stream(stream)), "cce_prefix_gather")


def cce_prefix_scatter(dH_head, P, Rc, Rr, dH_cat, stream=None):
    _check(lib().cce_prefix_scatter(_p(dH_head), P, Rc, Rr, dH_head.shape[1], _p(dH_cat),
                                    _stream(stream)), "cce_prefix_scatter")


def cce_backward_dh_dw(H, head: Head, labels, lse, coeff, filter_eps, blockmax, dH, dW,
                       skip_stats=None, ws=None, stream=None):
    st = lib().cce_backward_dh_dw(_p(H), h_dtype(H), H.shape[0], ctypes.byref(head.c()),
                                  _p(labels), _p(lse), _p(coeff), float(filter_eps),
                                  _p(blockmax), _p(dH), _p(dW), _p(skip_stats), _p(ws),
                                  ws.numel(), _stream(stream))
    _check(st, "cce_backward_dh_dw")


def cce_set_cta_pairs(on: bool):
    lib().cce_set_cta_pairs(1 if on else 0)


def cce_set_quant_staging(mode: int):
    """0: choose; 1: dequantise inside the GEMMs; 2: staged fp16 chunks."""
    lib().cce_set_quant_staging(int(mode))


def cce_set_backward_mode(mode: int):
    """Dense bf16 heads: 0 choose; 1 the grouped fused backward kernel; 2 two
    GEMMs per vocab chunk; 3 the sliced fused kernel (M <= 64, D <= 2048)."""
    lib().cce_set_backward_mode(int(mode))


def cce_set_forward_mode(mode: int):
    """4/8-bit heads: 0 choose (a transposed small-M kernel up to 240 head
    rows); 1 the tiled GEMM with in-kernel dequantisation at every M; 2 the
    transposed form of 129-240 rows for 1 to 256 rows."""
    lib().cce_set_forward_mode(int(mode))


def cce_query_fused_schedule(M: int, H_dtype: int, head: "Head | _Head"):
    """The fused backward's units as an int32 array [n, 6] (group, row tile,
    round, first, last, dH buffer), or None when the fused kernel does not
    take the problem (host-only)."""
    import numpy as np
    h = head.c() if isinstance(head, Head) else head
    n = lib().cce_query_fused_schedule(M, H_dtype, ctypes.byref(h), None, 0)
    if n < 0:
        return None
    out = np.zeros((max(n, 1), 6), dtype=np.int32)
    lib().cce_query_fused_schedule(M, H_dtype, ctypes.byref(h),
                                   out.ctypes.data_as(ctypes.c_void_p), n)
    return out[:n]


def cce_query_plan(M: int, H_dtype: int, head: "Head | _Head", ws_bytes: int) -> dict:
    """The chunking, K split, staging and CTA-pair plan the forward and
    backward would take with a workspace of ``ws_bytes`` (host-only)."""
    out = _Plan()
    h = head.c() if isinstance(head, Head) else head
    _check(lib().cce_query_plan(M, H_dtype, ctypes.byref(h), ws_bytes, ctypes.byref(out)),
           "cce_query_plan")
    return {n: getattr(out, n) for n, _ in _Plan._fields_}


# ----------------------------------------------------------------------------
# operators around the head
# ----------------------------------------------------------------------------
#
# Tensors: matrices may have any row stride (the columns are contiguous);
# 8-bit codes are torch.float8_e4m3fn; scales and per-row vectors are dense
# fp32.  A shape, type or stride the library would misread raises ValueError
# before the call; everything else is left to the library's own checks.  The
# call is made on the tensors' device and, without ``stream``, on that device's
# current stream.

QGROUP = 128


def fp8_groups(n: int) -> int:
    """Number of groups of 128 that ``n`` columns (or rows) fall into."""
    return -(-int(n) // QGROUP)


def fp8_empty(rows: int, cols: int, device="cuda"):
    """Room for 8-bit codes [rows, cols] with rows on 16-byte boundaries, as
    cce_fp8_matmul wants them."""
    return torch.empty(rows, -(-cols // 16) * 16, dtype=torch.float8_e4m3fn,
                       device=device)[:, :cols]


_MAT_TYPES = {torch.float32: CCE_F32, torch.bfloat16: CCE_BF16}
_CODES = {torch.float8_e4m3fn: 0}
_F32 = {torch.float32: CCE_F32}


def _bad(name, t, types, shape, dev):
    if not t.is_cuda:
        raise ValueError(f"{name}: not a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, the others on cuda:{dev}")
    if t.dtype not in types:
        raise ValueError(f"{name}: {t.dtype} not supported")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
    raise ValueError(f"{name}: strides {t.stride()} not supported")


def _mat(name, t, types, rows, cols, dev):
    """Address, type code and row stride of a matrix with contiguous rows."""
    if t.get_device() != dev or dev < 0 or t.dtype not in types or t.shape != (rows, cols):
        _bad(name, t, types, (rows, cols), dev)
    s0, s1 = t.stride()
    if (s1 != 1 and cols > 1) or (s0 < cols and rows > 1):
        _bad(name, t, types, (rows, cols), dev)
    return t.data_ptr(), types[t.dtype], (s0 if rows > 1 else cols)


def _dense(name, t, types, shape, dev):
    """Address of a contiguous tensor of this shape."""
    if (t.get_device() != dev or dev < 0 or t.dtype not in types or t.shape != shape
            or not t.is_contiguous()):
        _bad(name, t, types, shape, dev)
    return t.data_ptr()


def _workspace(ws, dev):
    if ws.get_device() != dev or dev < 0 or not ws.is_contiguous() or ws.dtype is not torch.uint8:
        _bad("ws", ws, {torch.uint8: 0}, tuple(ws.shape), dev)
    return ws.data_ptr(), ws.numel()


def _run(name, dev, stream, *args):
    """The library's call with the tensors' device current."""
    cur = torch._C._cuda_getDevice()
    if cur != dev:
        torch.cuda.set_device(dev)
    try:
        s = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
        st = getattr(lib(), name)(*args, s)
    finally:
        if cur != dev:
            torch.cuda.set_device(cur)
    if st != 0:
        raise CCEError(st, name)


def cce_fp8_quant_rows(X, Q, S, stream=None):
    """8-bit codes Q [M, D] and scales S [M, ceil(D/128)] of the rows of X
    (f32 or bf16), one scale for each 128 columns."""
    (M, D), dev = X.shape, X.get_device()
    x, xt, ldx = _mat("X", X, _MAT_TYPES, M, D, dev)
    q, _, ldq = _mat("Q", Q, _CODES, M, D, dev)
    _run("cce_fp8_quant_rows", dev, stream, x, xt, M, D, ldx, q, ldq,
         _dense("S", S, _F32, (M, fp8_groups(D)), dev))


def cce_fp8_quant_blocks(W, Q, S, stream=None):
    """8-bit codes Q [N, K] and scales S [ceil(N/128), ceil(K/128)] of the
    128 x 128 blocks of W (f32 or bf16)."""
    (N, K), dev = W.shape, W.get_device()
    x, xt, ldx = _mat("W", W, _MAT_TYPES, N, K, dev)
    q, _, ldq = _mat("Q", Q, _CODES, N, K, dev)
    _run("cce_fp8_quant_blocks", dev, stream, x, xt, N, K, ldx, q, ldq,
         _dense("S", S, _F32, (fp8_groups(N), fp8_groups(K)), dev))


def cce_fp8_matmul(A, SA, B, SB, C, ws, stream=None):
    """C [M, N] (f32 or bf16) = rows A [M, K] (scales SA, one for each 128
    columns) times head B [N, K] (scales SB, one for each 128 x 128 block),
    transposed.  A and B: rows on 16-byte boundaries (``fp8_empty``); ``ws``:
    uint8, 256 bytes for the status word, zeroed once."""
    (M, N), K, dev = C.shape, A.shape[1], C.get_device()
    c, ct, ldc = _mat("C", C, _MAT_TYPES, M, N, dev)
    a, _, lda = _mat("A", A, _CODES, M, K, dev)
    b, _, ldb = _mat("B", B, _CODES, N, K, dev)
    G = fp8_groups(K)
    _run("cce_fp8_matmul", dev, stream, a, lda, _dense("SA", SA, _F32, (M, G), dev), b, ldb,
         _dense("SB", SB, _F32, (fp8_groups(N), G), dev), M, N, K, c, ct, ldc,
         *_workspace(ws, dev))


def _codes_of(name, q, s, M, D, dev):
    if q is None and s is None:
        return None, 0, None
    if q is None or s is None:
        raise ValueError(f"{name}: codes and scales go together")
    p, _, ld = _mat(name, q, _CODES, M, D, dev)
    return p, ld, _dense(name + " scales", s, _F32, (M, fp8_groups(D)), dev)


def cce_norm_forward(X, w, eps, H=None, H8=None, Hs=None, X8=None, Xs=None, rstd=None,
                     stream=None):
    """Final norm H = X / sqrt(mean(X^2) + eps) * w, row by row, with its
    optional outputs: H (f32 or bf16), its 8-bit form (H8, Hs) and the
    checkpoint (X8, Xs, rstd) that cce_norm_backward reads."""
    (M, D), dev = X.shape, X.get_device()
    x, xt, ldx = _mat("X", X, _MAT_TYPES, M, D, dev)
    h, ht, ldh = (None, CCE_BF16, 0) if H is None else _mat("H", H, _MAT_TYPES, M, D, dev)
    h8, ldh8, hs = _codes_of("H8", H8, Hs, M, D, dev)
    x8, ldx8, xs = _codes_of("X8", X8, Xs, M, D, dev)
    _run("cce_norm_forward", dev, stream, x, xt, M, D, ldx,
         _dense("w", w, _MAT_TYPES, (D,), dev), _MAT_TYPES[w.dtype], eps, h, ht, ldh, h8, ldh8, hs,
         x8, ldx8, xs, None if rstd is None else _dense("rstd", rstd, _F32, (M,), dev))


def cce_norm_backward_workspace_bytes(M: int, D: int) -> int:
    return int(lib().cce_norm_backward_workspace_bytes(M, D))


def cce_norm_backward(X8, Xs, rstd, w, dH, dX, dW=None, ws=None, stream=None):
    """Gradient of the final norm from its checkpoint: dX [M, D] (f32 or bf16)
    and, unless the norm is frozen, dW fp32 [D]; ``ws``: uint8, at least
    cce_norm_backward_workspace_bytes(M, D) long, needed for dW only."""
    (M, D), dev = dH.shape, dH.get_device()
    dh, dht, lddh = _mat("dH", dH, _MAT_TYPES, M, D, dev)
    dx, dxt, lddx = _mat("dX", dX, _MAT_TYPES, M, D, dev)
    x8, ldx8, xs = _codes_of("X8", X8, Xs, M, D, dev)
    p, n = (None, 0) if ws is None else _workspace(ws, dev)
    _run("cce_norm_backward", dev, stream, x8, ldx8, xs, _dense("rstd", rstd, _F32, (M,), dev),
         M, D, _dense("w", w, _MAT_TYPES, (D,), dev), _MAT_TYPES[w.dtype], dh, dht, lddh, dx, dxt,
         lddx, None if dW is None else _dense("dW", dW, _F32, (D,), dev), p, n)


_I32 = {torch.int32: 0}


def cce_sample_rows(logits, temperature, top_k, top_p, min_p, u, tokens, logp=None, stream=None):
    """One token for each row of ``logits`` [B, V] (f32 or bf16) from the
    uniform numbers ``u`` [B]: ``temperature``, ``top_p``, ``min_p`` fp32 [B]
    and ``top_k`` int32 [B], each of the four None for none.  ``tokens`` int32
    [B] (-1 for a row that is masked throughout); ``logp`` fp32 [B], the
    tokens' log-softmax at temperature 1."""
    (B, V), dev = logits.shape, logits.get_device()
    l, lt, ld = _mat("logits", logits, _MAT_TYPES, B, V, dev)
    row = (B,)
    _run("cce_sample_rows", dev, stream, l, lt, B, V, ld,
         None if temperature is None else _dense("temperature", temperature, _F32, row, dev),
         None if top_k is None else _dense("top_k", top_k, _I32, row, dev),
         None if top_p is None else _dense("top_p", top_p, _F32, row, dev),
         None if min_p is None else _dense("min_p", min_p, _F32, row, dev),
         _dense("u", u, _F32, row, dev), _dense("tokens", tokens, _I32, row, dev),
         None if logp is None else _dense("logp", logp, _F32, row, dev))


# ----------------------------------------------------------------------------
# the operators in use: training behind a final norm, and decoding
# ----------------------------------------------------------------------------

@dataclass
class NormBuffers:
    """Device buffers of the final norm in a training pass: the head's rows,
    the 8-bit checkpoint that stands for X until the backward, the gradients
    (``dW`` None for a frozen norm) and the workspace."""

    H: torch.Tensor
    X8: torch.Tensor
    Xs: torch.Tensor
    rstd: torch.Tensor
    dX: torch.Tensor
    dW: torch.Tensor | None
    ws: torch.Tensor | None

    @staticmethod
    def alloc(M: int, D: int, H_dtype: int = CCE_BF16, dX_dtype=torch.bfloat16, frozen=False,
              device="cuda"):
        f = dict(device=device, dtype=torch.float32)
        return NormBuffers(
            H=torch.empty(M, D, device=device,
                          dtype=torch.float32 if H_dtype == CCE_F32 else torch.bfloat16),
            X8=fp8_empty(M, D, device), Xs=torch.empty(M, fp8_groups(D), **f),
            rstd=torch.empty(M, **f), dX=torch.empty(M, D, device=device, dtype=dX_dtype),
            dW=None if frozen else torch.empty(D, **f),
            ws=None if frozen else torch.zeros(cce_norm_backward_workspace_bytes(M, D),
                                               dtype=torch.uint8, device=device))


def orpo_norm_head_pass(X, norm_w, eps, head: Head, labels, layout, lam, sft_scope, filter_eps,
                        block_skip: bool, norm: NormBuffers, buf: HeadBuffers, stream=None):
    """``orpo_head_pass`` from the residual stream X [M, D] on: the final norm
    with its 8-bit checkpoint, the head's pass, and the norm's gradient from
    the checkpoint (``norm.dX``, ``norm.dW``).  X is read by the first kernel
    only; its memory may be reused once that has run.  The whole pass is made
    on X's device and, without ``stream``, on that device's current stream."""
    with torch.cuda.device(X.device):  # the head's own calls go to the current device
        cce_norm_forward(X, norm_w, eps, H=norm.H, X8=norm.X8, Xs=norm.Xs, rstd=norm.rstd,
                         stream=stream)
        orpo_head_pass(norm.H, head, labels, layout, lam, sft_scope, filter_eps, block_skip, buf,
                       stream)
        cce_norm_backward(norm.X8, norm.Xs, norm.rstd, norm_w, buf.dH, norm.dX, norm.dW, norm.ws,
                          stream)


@dataclass
class Fp8Head:
    """A dense head in 8 bits for decoding (``cce_forward`` and the backward do
    not take it): codes [V, D] and one scale for each 128 x 128 block."""

    q: torch.Tensor
    s: torch.Tensor

    @staticmethod
    def from_dense(w, stream=None):
        """The 8-bit form of ``w`` [V, D], made on ``stream`` behind what the
        current stream has been given so far (``w`` may be its work, and the
        new tensors' memory may still be in use there)."""
        V, D = w.shape
        h = Fp8Head(fp8_empty(V, D, w.device),
                    torch.empty(fp8_groups(V), fp8_groups(D), dtype=torch.float32,
                                device=w.device))
        if stream is not None:
            now = torch.cuda.current_stream(w.device)
            if stream != now:
                stream.wait_stream(now)
                h.q.record_stream(stream)
                h.s.record_stream(stream)
        cce_fp8_quant_blocks(w, h.q, h.s, stream)
        return h


@dataclass
class DecodeBuffers:
    """Device buffers of one decoding step of B rows."""

    H8: torch.Tensor
    Hs: torch.Tensor
    logits: torch.Tensor
    tokens: torch.Tensor
    logp: torch.Tensor
    ws: torch.Tensor

    @staticmethod
    def alloc(B: int, head: Fp8Head, logits_dtype=torch.float32):
        (V, D), dev = head.q.shape, head.q.device
        f = dict(device=dev, dtype=torch.float32)
        return DecodeBuffers(
            H8=fp8_empty(B, D, dev), Hs=torch.empty(B, fp8_groups(D), **f),
            logits=torch.empty(B, V, device=dev, dtype=logits_dtype),
            tokens=torch.empty(B, dtype=torch.int32, device=dev), logp=torch.empty(B, **f),
            ws=torch.zeros(256, dtype=torch.uint8, device=dev))


def decode_step(X, norm_w, eps, head: Fp8Head, u, buf: DecodeBuffers, temperature=None,
                top_k=None, top_p=None, min_p=None, stream=None):
    """The last step of decoding for B rows of the residual stream: final norm
    into 8 bits, logits, one sampled token a row (``buf.tokens``, and
    ``buf.logp``, the log-prob that the ORPO loss takes for that label)."""
    cce_norm_forward(X, norm_w, eps, H8=buf.H8, Hs=buf.Hs, stream=stream)
    cce_fp8_matmul(buf.H8, buf.Hs, head.q, head.s, buf.logits, buf.ws, stream)
    cce_sample_rows(buf.logits, temperature, top_k, top_p, min_p, u, buf.tokens, buf.logp, stream)
