"""Python binding of the C ABI in include/axon_ssm.h (ctypes, argument marshalling only).

Every step of the layer core runs in the CUDA library ``libaxon_ssm.so`` built
in-tree by ``selective_state_space_52_b200.build``.  There is no CPU or PyTorch
fallback: importing this module raises if the library is missing, and every
call raises ``AxonError`` on a non-OK status.  PyTorch provides device memory
and the current stream.

Functions named like the C entry points take torch tensors (device, contiguous)
and pass their pointers through; ``scan_fwd`` and ``step`` additionally allocate
outputs / workspace with torch for convenience.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libaxon_ssm.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"CUDA library not built: {LIB_PATH} is missing. "
        "Run `python -m selective_state_space_52_b200.build` (nvcc, sm_100a).")

_lib = ctypes.CDLL(LIB_PATH)

AXON_F32 = 0
AXON_BF16 = 1
STATUS = {0: "AXON_OK", 1: "AXON_ERR_INVALID_ARG", 2: "AXON_ERR_UNSUPPORTED",
          3: "AXON_ERR_ALIGNMENT", 4: "AXON_ERR_WORKSPACE", 5: "AXON_ERR_CUDA",
          6: "AXON_ERR_TIMEOUT"}

_vp = ctypes.c_void_p
_i = ctypes.c_int
_sz = ctypes.c_size_t

_lib.axon_ssm_abi_version.restype = _i
_lib.axon_ssm_abi_version.argtypes = []
_lib.axon_status_string.restype = ctypes.c_char_p
_lib.axon_status_string.argtypes = [_i]
_lib.axon_ssm_scan_workspace_bytes.restype = _sz
_lib.axon_ssm_scan_workspace_bytes.argtypes = [_i] * 6
_lib.axon_ssm_scan_launch_count.restype = _i
_lib.axon_ssm_scan_launch_count.argtypes = [_i] * 6
_SCAN_ARGS = [_i] * 6 + [_vp] * 15 + [_vp, _sz]
_lib.axon_ssm_scan_fwd.restype = _i
_lib.axon_ssm_scan_fwd.argtypes = _SCAN_ARGS + [_vp]
_lib.axon_ssm_scan_fwd_segments.restype = _i
_lib.axon_ssm_scan_fwd_segments.argtypes = _SCAN_ARGS + [_i, _vp]
_lib.axon_ssm_scan_fwd_noalloc.restype = _i
_lib.axon_ssm_scan_fwd_noalloc.argtypes = [_i] * 6 + [_vp] * 15 + [_i, _vp]
NOALLOC_SCRATCH_BYTES = 16 << 20
_lib.axon_ssm_scan_fwd_qsplit.restype = _i
_lib.axon_ssm_scan_fwd_qsplit.argtypes = [_i] * 8 + [_vp] * 15 + [_vp]
_lib.axon_ssm_scan_fwd_ex.restype = _i
_lib.axon_ssm_scan_fwd_ex.argtypes = [_i] * 7 + [_vp] * 15 + [_vp, _sz, _i, _vp]
_lib.axon_ssm_step_ex.restype = _i
_lib.axon_ssm_step_ex.argtypes = [_i] * 6 + [_vp] * 13 + [_vp]
AXON_DISC_FIRST_ORDER = 0
AXON_DISC_ZOH = 1
_DISC = {"first_order": AXON_DISC_FIRST_ORDER, "zoh": AXON_DISC_ZOH}
_lib.axon_ssm_step.restype = _i
_lib.axon_ssm_step.argtypes = [_i] * 5 + [_vp] * 13 + [_vp]
_lib.axon_ssm_dt_sum.restype = _i
_lib.axon_ssm_dt_sum.argtypes = [_i] * 4 + [_vp] * 3 + [_vp]
_lib.axon_ssm_carry_fold.restype = _i
_lib.axon_ssm_carry_fold.argtypes = [_i] * 5 + [_vp] * 4 + [_vp]
_lib.axon_ssm_scan_state.restype = _i
_lib.axon_ssm_scan_state.argtypes = [_i] * 6 + [_vp] * 12 + [_vp]
_lib.axon_ssd_wait_probe.restype = _i
_lib.axon_ssd_wait_probe.argtypes = [_vp, _i, _vp]
_lib.axon_ssd_workspace_bytes.restype = _sz
_lib.axon_ssd_workspace_bytes.argtypes = [_i] * 6
_lib.axon_ssd_scan_fwd.restype = _i
_lib.axon_ssd_scan_fwd.argtypes = [_i] * 6 + [_vp] * 10 + [_i, _vp, _sz, _vp]
_lib.axon_delta_workspace_bytes.restype = _sz
_lib.axon_delta_workspace_bytes.argtypes = [_i] * 8
_lib.axon_delta_scan_fwd.restype = _i
_lib.axon_delta_scan_fwd.argtypes = ([_i] * 7 + [_vp, _i] * 3 + [_vp] * 6 + [ctypes.c_float, _i] +
                                     [_vp] * 2 + [_i, _vp, _sz, _vp])
_lib.axon_delta_wait_probe.restype = _i
_lib.axon_delta_wait_probe.argtypes = [_vp, _i, _vp]
_lib.axon_delta_step.restype = _i
_lib.axon_delta_step.argtypes = [_i] * 6 + [_vp, _i] * 3 + [_vp] * 4 + [ctypes.c_float, _i] + [_vp] * 3
_lib.axon_gated_norm_fwd.restype = _i
_lib.axon_gated_norm_fwd.argtypes = [_i] * 7 + [_vp, _i] * 2 + [_vp] * 2 + [_i, ctypes.c_float, _vp, _i, _vp]
_lib.axon_gemm_bf16.restype = _i
_lib.axon_exp2_fma.restype = _i
_lib.axon_peak_probe.restype = _i
_lib.axon_peak_probe.argtypes = [_i, _vp, _i, ctypes.c_longlong, _vp]
_lib.axon_exp2_fma.argtypes = [_vp, _vp, ctypes.c_longlong, _vp]
_lib.axon_gemm_bf16.argtypes = [_i] * 3 + [_vp, _i, _vp, _i, _vp, _i, _vp, _vp]
_lib.axon_gemm_bf16_plan.restype = _i
_lib.axon_gemm_bf16_plan.argtypes = [_i] * 3 + [_vp, _i, _vp, _i, _vp, _i, _vp, _i, _vp, _sz, _vp]
_lib.axon_gemm_workspace_bytes.restype = _sz
_lib.axon_gemm_workspace_bytes.argtypes = []
_lib.axon_ssm_block_workspace_bytes.restype = _sz
_lib.axon_ssm_block_workspace_bytes.argtypes = [_i] * 7
_lib.axon_ssm_block_fwd.restype = _i
_lib.axon_ssm_block_fwd.argtypes = [_i] * 7 + [_vp] * 14 + [_vp, _sz, _vp]


class AxonError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return AXON_F32
    if t == torch.bfloat16:
        return AXON_BF16
    raise TypeError(f"unsupported io dtype {t}; use float32 or bfloat16")


def _p(t):
    """Device pointer of a tensor (None -> NULL).  Tensors must be contiguous."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors passed to the C ABI must be contiguous")
    return t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, where: str):
    if rc != 0:
        raise AxonError(rc, where)


# ------------------------------------------------------------ C entry points
def axon_ssm_abi_version() -> int:
    return _lib.axon_ssm_abi_version()


def axon_status_string(status: int) -> str:
    return _lib.axon_status_string(int(status)).decode()


def axon_ssm_scan_workspace_bytes(B, L, E, N=16, K=4, io=AXON_BF16) -> int:
    return int(_lib.axon_ssm_scan_workspace_bytes(B, L, E, N, K, io))


def axon_ssm_scan_launch_count(B, L, E, N=16, K=4, io=AXON_BF16) -> int:
    return int(_lib.axon_ssm_scan_launch_count(B, L, E, N, K, io))


def axon_ssm_scan_fwd(B, L, E, N, K, io, x, z, dt_raw, Bm, Cm, conv_w, conv_b, dt_bias,
                      A_log, D, conv_cache_in, ssm_state_in, y, conv_cache_out,
                      ssm_state_out, workspace, workspace_bytes, stream=None, *,
                      raise_on_error=True) -> int:
    rc = _lib.axon_ssm_scan_fwd(B, L, E, N, K, io, _p(x), _p(z), _p(dt_raw), _p(Bm), _p(Cm),
                                _p(conv_w), _p(conv_b), _p(dt_bias), _p(A_log), _p(D),
                                _p(conv_cache_in), _p(ssm_state_in), _p(y),
                                _p(conv_cache_out), _p(ssm_state_out), _p(workspace),
                                int(workspace_bytes), _stream(stream))
    if raise_on_error:
        _check(rc, "axon_ssm_scan_fwd")
    return rc


def axon_ssm_scan_fwd_segments(B, L, E, N, K, io, x, z, dt_raw, Bm, Cm, conv_w, conv_b,
                               dt_bias, A_log, D, conv_cache_in, ssm_state_in, y,
                               conv_cache_out, ssm_state_out, workspace, workspace_bytes,
                               num_segments, stream=None, *, raise_on_error=True) -> int:
    rc = _lib.axon_ssm_scan_fwd_segments(B, L, E, N, K, io, _p(x), _p(z), _p(dt_raw), _p(Bm),
                                         _p(Cm), _p(conv_w), _p(conv_b), _p(dt_bias),
                                         _p(A_log), _p(D), _p(conv_cache_in),
                                         _p(ssm_state_in), _p(y), _p(conv_cache_out),
                                         _p(ssm_state_out), _p(workspace),
                                         int(workspace_bytes), int(num_segments),
                                         _stream(stream))
    if raise_on_error:
        _check(rc, "axon_ssm_scan_fwd_segments")
    return rc


def axon_ssm_scan_fwd_noalloc(B, L, E, N, K, io, x, z, dt_raw, Bm, Cm, conv_w, conv_b,
                              dt_bias, A_log, D, conv_cache_in, ssm_state_in, y,
                              conv_cache_out, ssm_state_out, num_segments=0, stream=None, *,
                              raise_on_error=True) -> int:
    """The prefill with its time-split scratch in the library's own 16 MiB device
    array, for callers that cannot provide a workspace (see include/axon_ssm.h)."""
    rc = _lib.axon_ssm_scan_fwd_noalloc(B, L, E, N, K, io, _p(x), _p(z), _p(dt_raw), _p(Bm),
                                        _p(Cm), _p(conv_w), _p(conv_b), _p(dt_bias),
                                        _p(A_log), _p(D), _p(conv_cache_in),
                                        _p(ssm_state_in), _p(y), _p(conv_cache_out),
                                        _p(ssm_state_out), int(num_segments), _stream(stream))
    if raise_on_error:
        _check(rc, "axon_ssm_scan_fwd_noalloc")
    return rc


def axon_ssm_scan_fwd_qsplit(B, L, E, N, K, io, disc, runs, x, z, dt_raw, Bm, Cm, conv_w, conv_b,
                             dt_bias, A_log, D, conv_cache_in, ssm_state_in, y, conv_cache_out,
                             ssm_state_out, stream=None, *, raise_on_error=True) -> int:
    """The prefill on the split-chunk quadrant scan with `runs` warps per 8
    channels (1, 2, 4 or 8), for tests and tuning."""
    rc = _lib.axon_ssm_scan_fwd_qsplit(B, L, E, N, K, io, int(disc), int(runs), _p(x), _p(z),
                                       _p(dt_raw), _p(Bm), _p(Cm), _p(conv_w), _p(conv_b),
                                       _p(dt_bias), _p(A_log), _p(D), _p(conv_cache_in),
                                       _p(ssm_state_in), _p(y), _p(conv_cache_out),
                                       _p(ssm_state_out), _stream(stream))
    if raise_on_error:
        _check(rc, "axon_ssm_scan_fwd_qsplit")
    return rc


def axon_ssm_scan_fwd_ex(B, L, E, N, K, io, disc, x, z, dt_raw, Bm, Cm, conv_w, conv_b,
                         dt_bias, A_log, D, conv_cache_in, ssm_state_in, y, conv_cache_out,
                         ssm_state_out, workspace, workspace_bytes, num_segments=0, stream=None, *,
                         raise_on_error=True) -> int:
    rc = _lib.axon_ssm_scan_fwd_ex(B, L, E, N, K, io, int(disc), _p(x), _p(z), _p(dt_raw),
                                   _p(Bm), _p(Cm), _p(conv_w), _p(conv_b), _p(dt_bias),
                                   _p(A_log), _p(D), _p(conv_cache_in), _p(ssm_state_in), _p(y),
                                   _p(conv_cache_out), _p(ssm_state_out), _p(workspace),
                                   int(workspace_bytes), int(num_segments), _stream(stream))
    if raise_on_error:
        _check(rc, "axon_ssm_scan_fwd_ex")
    return rc


def axon_ssm_step_ex(B, E, N, K, io, disc, x, z, dt_raw, Bm, Cm, conv_w, conv_b, dt_bias,
                     A_log, D, conv_cache, ssm_state, y, stream=None, *, raise_on_error=True) -> int:
    rc = _lib.axon_ssm_step_ex(B, E, N, K, io, int(disc), _p(x), _p(z), _p(dt_raw), _p(Bm),
                               _p(Cm), _p(conv_w), _p(conv_b), _p(dt_bias), _p(A_log), _p(D),
                               _p(conv_cache), _p(ssm_state), _p(y), _stream(stream))
    if raise_on_error:
        _check(rc, "axon_ssm_step_ex")
    return rc


def axon_ssm_step(B, E, N, K, io, x, z, dt_raw, Bm, Cm, conv_w, conv_b, dt_bias, A_log, D,
                  conv_cache, ssm_state, y, stream=None, *, raise_on_error=True) -> int:
    rc = _lib.axon_ssm_step(B, E, N, K, io, _p(x), _p(z), _p(dt_raw), _p(Bm), _p(Cm),
                            _p(conv_w), _p(conv_b), _p(dt_bias), _p(A_log), _p(D),
                            _p(conv_cache), _p(ssm_state), _p(y), _stream(stream))
    if raise_on_error:
        _check(rc, "axon_ssm_step")
    return rc


def axon_ssm_dt_sum(B, L, E, io, dt_raw, dt_bias, dt_sum, stream=None, *, raise_on_error=True) -> int:
    rc = _lib.axon_ssm_dt_sum(B, L, E, io, _p(dt_raw), _p(dt_bias), _p(dt_sum), _stream(stream))
    if raise_on_error:
        _check(rc, "axon_ssm_dt_sum")
    return rc


def axon_ssm_carry_fold(P, r, B, E, N, A_log, h_loc, dt_sum, h_in, stream=None, *,
                        raise_on_error=True) -> int:
    rc = _lib.axon_ssm_carry_fold(P, r, B, E, N, _p(A_log), _p(h_loc), _p(dt_sum), _p(h_in),
                                  _stream(stream))
    if raise_on_error:
        _check(rc, "axon_ssm_carry_fold")
    return rc


def axon_ssm_scan_state(B, L, E, N, K, io, x, dt_raw, Bm, conv_w, conv_b, dt_bias, A_log,
                        conv_cache_in, ssm_state_in, conv_cache_out, ssm_state_out, dt_sum, stream=None, *,
                        raise_on_error=True) -> int:
    rc = _lib.axon_ssm_scan_state(B, L, E, N, K, io, _p(x), _p(dt_raw), _p(Bm), _p(conv_w), _p(conv_b),
                                  _p(dt_bias), _p(A_log), _p(conv_cache_in), _p(ssm_state_in),
                                  _p(conv_cache_out), _p(ssm_state_out), _p(dt_sum), _stream(stream))
    if raise_on_error:
        _check(rc, "axon_ssm_scan_state")
    return rc


def axon_ssd_wait_probe(status, limit, stream=None, *, raise_on_error=True) -> int:
    rc = _lib.axon_ssd_wait_probe(_p(status), int(limit), _stream(stream))
    if raise_on_error:
        _check(rc, "axon_ssd_wait_probe")
    return rc


def axon_ssd_workspace_bytes(B, L, H, P=64, N=128, segments=0) -> int:
    return int(_lib.axon_ssd_workspace_bytes(B, L, H, P, N, segments))


def axon_ssd_scan_fwd(B, L, H, P, N, io, x, dt_raw, dt_bias, A_log, Bm, Cm, D, h0, y, h_out, segments,
                      workspace, workspace_bytes, stream=None, *, raise_on_error=True) -> int:
    rc = _lib.axon_ssd_scan_fwd(B, L, H, P, N, io, _p(x), _p(dt_raw), _p(dt_bias), _p(A_log), _p(Bm),
                                _p(Cm), _p(D), _p(h0), _p(y), _p(h_out), int(segments), _p(workspace),
                                int(workspace_bytes), _stream(stream))
    if raise_on_error:
        _check(rc, "axon_ssd_scan_fwd")
    return rc


def axon_delta_workspace_bytes(B, L, H, G, P=128, N=128, io=AXON_BF16, segments=0) -> int:
    return int(_lib.axon_delta_workspace_bytes(B, L, H, G, P, N, io, segments))


def _v(t):
    """Device pointer of a tensor that may be a view with a row stride."""
    return t if t is None or isinstance(t, int) else t.data_ptr()


def axon_delta_scan_fwd(B, L, H, G, P, N, io, q, ldq, k, ldk, v, ldv, dt_raw, b_raw, dt_bias, A_log, lengths, h0,
                        scale, qk_norm, y, h_out, segments, workspace, workspace_bytes, stream=None, *,
                        raise_on_error=True) -> int:
    rc = _lib.axon_delta_scan_fwd(B, L, H, G, P, N, io, _v(q), ldq, _v(k), ldk, _v(v), ldv, _p(dt_raw), _p(b_raw),
                                  _p(dt_bias), _p(A_log), _p(lengths), _p(h0), scale, qk_norm, _p(y), _p(h_out),
                                  segments, _p(workspace), int(workspace_bytes), _stream(stream))
    if raise_on_error:
        _check(rc, "axon_delta_scan_fwd")
    return rc


def axon_delta_step(B, H, G, P, N, io, q, ldq, k, ldk, v, ldv, dt_raw, b_raw, dt_bias, A_log, scale, qk_norm, state,
                    y, stream=None, *, raise_on_error=True) -> int:
    rc = _lib.axon_delta_step(B, H, G, P, N, io, _v(q), ldq, _v(k), ldk, _v(v), ldv, _p(dt_raw), _p(b_raw),
                              _p(dt_bias), _p(A_log), scale, qk_norm, _p(state), _p(y), _stream(stream))
    if raise_on_error:
        _check(rc, "axon_delta_step")
    return rc


def axon_gated_norm_fwd(rows, C, D, io, kind, gate, act, x, ldx, z, ldz, weight, bias, per_channel, eps, y, ldy,
                        stream=None, *, raise_on_error=True) -> int:
    rc = _lib.axon_gated_norm_fwd(rows, C, D, io, kind, gate, act, _v(x), ldx, _v(z), ldz, _p(weight), _p(bias),
                                  per_channel, eps, _v(y), ldy, _stream(stream))
    if raise_on_error:
        _check(rc, "axon_gated_norm_fwd")
    return rc


def axon_delta_wait_probe(status, limit, stream=None, *, raise_on_error=True) -> int:
    rc = _lib.axon_delta_wait_probe(_p(status), int(limit), _stream(stream))
    if raise_on_error:
        _check(rc, "axon_delta_wait_probe")
    return rc


def axon_ssm_block_workspace_bytes(B, L, Dm, E, N=16, K=4, io=AXON_BF16) -> int:
    return int(_lib.axon_ssm_block_workspace_bytes(B, L, Dm, E, N, K, io))


def axon_ssm_block_fwd(B, L, Dm, E, N, K, io, X, W_in, W_x, W_out, conv_w, conv_b, dt_bias,
                       A_log, D, conv_cache_in, ssm_state_in, out, conv_cache_out, ssm_state_out,
                       workspace, workspace_bytes, stream=None, *, raise_on_error=True) -> int:
    rc = _lib.axon_ssm_block_fwd(B, L, Dm, E, N, K, io, _p(X), _p(W_in), _p(W_x), _p(W_out),
                                 _p(conv_w), _p(conv_b), _p(dt_bias), _p(A_log), _p(D),
                                 _p(conv_cache_in), _p(ssm_state_in), _p(out), _p(conv_cache_out),
                                 _p(ssm_state_out), _p(workspace), int(workspace_bytes),
                                 _stream(stream))
    if raise_on_error:
        _check(rc, "axon_ssm_block_fwd")
    return rc


def axon_gemm_bf16(M, N, K, A, lda, W, ldw, C, ldc, err=None, stream=None, *, raise_on_error=True) -> int:
    rc = _lib.axon_gemm_bf16(M, N, K, _p(A), int(lda), _p(W), int(ldw), _p(C), int(ldc), _p(err),
                             _stream(stream))
    if raise_on_error:
        _check(rc, "axon_gemm_bf16")
    return rc


# tilings of axon_gemm_bf16_plan (include/axon_ssm.h)
GEMM_AUTO, GEMM_SINGLE_256, GEMM_SINGLE_192, GEMM_PAIR, GEMM_PAIR_STREAMK = 0, 1, 2, 3, 4


def axon_gemm_workspace_bytes() -> int:
    return int(_lib.axon_gemm_workspace_bytes())


def axon_gemm_bf16_plan(M, N, K, A, lda, W, ldw, C, ldc, err=None, plan=GEMM_AUTO, workspace=None,
                        workspace_bytes=0, stream=None, *, raise_on_error=True) -> int:
    rc = _lib.axon_gemm_bf16_plan(M, N, K, _p(A), int(lda), _p(W), int(ldw), _p(C), int(ldc), _p(err),
                                  int(plan), _p(workspace), int(workspace_bytes), _stream(stream))
    if raise_on_error:
        _check(rc, "axon_gemm_bf16_plan")
    return rc


def axon_exp2_fma(x, y, n, stream=None, *, raise_on_error=True) -> int:
    rc = _lib.axon_exp2_fma(_p(x), _p(y), int(n), _stream(stream))
    if raise_on_error:
        _check(rc, "axon_exp2_fma")
    return rc


def axon_peak_probe(kind, out, blocks, iters, stream=None, *, raise_on_error=True) -> int:
    rc = _lib.axon_peak_probe(int(kind), _p(out), int(blocks), int(iters), _stream(stream))
    if raise_on_error:
        _check(rc, "axon_peak_probe")
    return rc


def exp2_fma(x, *, out=None, stream=None):
    """2^x of a contiguous float32 CUDA tensor through the FMA-pipe exp2."""
    import torch
    if x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("exp2_fma: x must be a contiguous float32 CUDA tensor")
    y = torch.empty_like(x) if out is None else out
    axon_exp2_fma(x.data_ptr(), y.data_ptr(), x.numel(), stream=stream)
    return y


def gemm_bf16(A, W, *, out=None, stream=None, check=True, plan=GEMM_AUTO, workspace=None):
    """C = A @ W for row-major bf16 A (M x K) and W (K x N) on the library's
    tcgen05 GEMM (float32 accumulation; ``plan``: one of the GEMM_* tilings,
    ``workspace``: a uint8 CUDA tensor of axon_gemm_workspace_bytes() bytes,
    needed by GEMM_PAIR_STREAMK).  With ``check`` the call waits for the
    device and raises AxonError (AXON_ERR_TIMEOUT) if a wait of the kernel
    gave up."""
    M, K = A.shape
    N = W.shape[1]
    C = torch.empty(M, N, dtype=torch.bfloat16, device=A.device) if out is None else out
    err = torch.zeros(1, dtype=torch.int32, device=A.device)
    nws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    axon_gemm_bf16_plan(M, N, K, A, A.stride(0), W, W.stride(0), C, C.stride(0), err, plan, workspace, nws,
                        stream=stream)
    if check and int(err.item()) != 0:
        raise AxonError(6, "axon_gemm_bf16 (a wait for a copy or a tensor-core product gave up)")
    return C


# ------------------------------------------------------------ conveniences
PARAM_KEYS = ("conv_w", "conv_b", "dt_bias", "A_log", "D")
WEIGHT_KEYS = ("W_in", "W_x", "W_out")


def scan_fwd(x, z, dt_raw, Bm, Cm, params: dict, cache=None, *, num_segments=None,
             out=None, workspace=None, stream=None, discretization="first_order", runs=None):
    """Prefill over (B, L, E) inputs on the GPU.

    ``params`` holds conv_w, conv_b, dt_bias, A_log, D (float32, on the device);
    ``cache`` is None or (conv_cache, ssm_state).  Returns
    ``(y, (conv_cache, ssm_state))`` -- the cache pair of the Axon-SSM page's
    "Autoregressive decoding" section, ready for the next call or for ``step``.
    ``runs`` (tests and tuning) forces the split-chunk quadrant scan with that
    many warps per 8 channels.
    """
    Bsz, L, E = x.shape
    K = params["conv_w"].shape[1]
    N = params["A_log"].shape[1]
    io = _dtype_code(x.dtype)
    dev = x.device
    cc_in, ss_in = (None, None) if cache is None else cache
    if out is None:
        y = torch.empty_like(x)
        cc_out = torch.empty(Bsz, K - 1, E, dtype=x.dtype, device=dev)
        ss_out = torch.empty(Bsz, E, N, dtype=torch.float32, device=dev)
    else:
        y, cc_out, ss_out = out
    if workspace is None:
        if num_segments is None:
            nbytes = axon_ssm_scan_workspace_bytes(Bsz, L, E, N, K, io)
        else:
            nbytes = max(num_segments - 1, 0) * Bsz * E * (N + 1) * 4
        if nbytes > 0:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    wsz = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = (Bsz, L, E, N, K, io, x, z, dt_raw, Bm, Cm, *(params[k] for k in PARAM_KEYS),
            cc_in, ss_in, y, cc_out, ss_out, workspace, wsz)
    if runs is not None:
        axon_ssm_scan_fwd_qsplit(Bsz, L, E, N, K, io, _DISC[discretization], runs, *args[6:-2],
                                 stream=stream)
    elif discretization != "first_order":
        axon_ssm_scan_fwd_ex(Bsz, L, E, N, K, io, _DISC[discretization], *args[6:],
                             num_segments or 0, stream=stream)
    elif num_segments is None:
        axon_ssm_scan_fwd(*args, stream=stream)
    else:
        axon_ssm_scan_fwd_segments(*args, num_segments, stream=stream)
    return y, (cc_out, ss_out)


def step(x, z, dt_raw, Bm, Cm, params: dict, cache, *, y=None, stream=None,
         discretization="first_order"):
    """One cached decode step; ``cache = (conv_cache, ssm_state)`` is updated in place."""
    Bsz, E = x.shape
    K = params["conv_w"].shape[1]
    N = params["A_log"].shape[1]
    conv_cache, ssm_state = cache
    if y is None:
        y = torch.empty_like(x)
    args = (x, z, dt_raw, Bm, Cm, *(params[k] for k in PARAM_KEYS), conv_cache, ssm_state, y)
    if discretization != "first_order":
        axon_ssm_step_ex(Bsz, E, N, K, _dtype_code(x.dtype), _DISC[discretization], *args,
                         stream=stream)
    else:
        axon_ssm_step(Bsz, E, N, K, _dtype_code(x.dtype), *args, stream=stream)
    return y


def block_error_flag(workspace) -> int:
    """The whole layer's GEMM error flag (the workspace's first int) after the
    call that used ``workspace`` has completed.  Synchronises the device."""
    torch.cuda.synchronize(workspace.device)
    return int(workspace[:4].view(torch.int32).item())


def block_fwd(X, weights: dict, params: dict, cache=None, *, out=None, workspace=None, stream=None,
              check=True):
    """The whole Axon-SSM layer on (B, L, Dm) bf16 input ``X``.

    ``weights`` holds W_in (Dm, 2E), W_x (E, E+2N), W_out (E, Dm) in bf16;
    ``params`` and ``cache`` as for ``scan_fwd``.  Returns
    ``(out, (conv_cache, ssm_state))``.  With ``check`` (the default) the call
    waits for the device and raises AxonError (AXON_ERR_TIMEOUT) if a wait of
    a projection GEMM gave up; ``check=False`` returns at once (read the flag
    with ``block_error_flag(workspace)``).
    """
    Bsz, L, Dm = X.shape
    E = weights["W_in"].shape[1] // 2
    K = params["conv_w"].shape[1]
    N = params["A_log"].shape[1]
    dev = X.device
    cc_in, ss_in = (None, None) if cache is None else cache
    if out is None:
        y = torch.empty_like(X)
        cc_out = torch.empty(Bsz, K - 1, E, dtype=X.dtype, device=dev)
        ss_out = torch.empty(Bsz, E, N, dtype=torch.float32, device=dev)
    else:
        y, cc_out, ss_out = out
    io = _dtype_code(X.dtype)
    nbytes = axon_ssm_block_workspace_bytes(Bsz, L, Dm, E, N, K, io)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    wsz = workspace.numel() * workspace.element_size()
    axon_ssm_block_fwd(Bsz, L, Dm, E, N, K, io, X, weights["W_in"], weights["W_x"], weights["W_out"],
                       *(params[k] for k in PARAM_KEYS), cc_in, ss_in, y, cc_out, ss_out,
                       workspace, wsz, stream=stream)
    if check and Bsz * E > 0 and block_error_flag(workspace) != 0:
        raise AxonError(6, "axon_ssm_block_fwd (a wait of a projection GEMM gave up)")
    return y, (cc_out, ss_out)


def dt_sum(dt_raw, dt_bias, *, stream=None):
    """(B, E) float32: the sum over the sequence of clip(softplus(dt_raw + dt_bias))."""
    Bsz, L, E = dt_raw.shape
    out = torch.empty(Bsz, E, dtype=torch.float32, device=dt_raw.device)
    axon_ssm_dt_sum(Bsz, L, E, _dtype_code(dt_raw.dtype), dt_raw, dt_bias, out, stream=stream)
    return out


def scan_state(x, dt_raw, Bm, params: dict, cache=None, *, stream=None):
    """The state-only prefill (first order): returns ((conv_cache, ssm_state),
    dt_sum) -- the final caches and the (B, E) float32 sum of the step sizes --
    without z, C, D or y."""
    Bsz, L, E = x.shape
    K = params["conv_w"].shape[1]
    N = params["A_log"].shape[1]
    cc_in, ss_in = (None, None) if cache is None else cache
    dev = x.device
    cc_out = torch.empty(Bsz, K - 1, E, dtype=x.dtype, device=dev)
    ss_out = torch.empty(Bsz, E, N, dtype=torch.float32, device=dev)
    dts = torch.empty(Bsz, E, dtype=torch.float32, device=dev)
    axon_ssm_scan_state(Bsz, L, E, N, K, _dtype_code(x.dtype), x, dt_raw, Bm, params["conv_w"], params["conv_b"],
                        params["dt_bias"], params["A_log"], cc_in, ss_in, cc_out, ss_out, dts, stream=stream)
    return (cc_out, ss_out), dts


def carry_fold(r, A_log, h_loc_all, dt_sum_all, *, stream=None):
    """The state entering slice r of a time-split sequence from the stacked
    (P,B,E,N) end states and (P,B,E) dt sums of all slices."""
    P, Bsz, E, N = h_loc_all.shape
    out = torch.empty(Bsz, E, N, dtype=torch.float32, device=h_loc_all.device)
    axon_ssm_carry_fold(P, r, Bsz, E, N, A_log, h_loc_all, dt_sum_all, out, stream=stream)
    return out


def ssd_error_flag(workspace) -> int:
    """The SSD walk's error flag (the workspace's first int) after the call
    that used ``workspace`` has completed: 1 if a wait for a tensor-core
    product gave up.  Synchronises the device."""
    torch.cuda.synchronize(workspace.device)
    return int(workspace[:4].view(torch.int32).item())


def ssd_scan(x, dt_raw, Bm, Cm, params: dict, h0=None, *, out=None, workspace=None, stream=None, segments=0,
             check=True):
    """The Mamba-2 (SSD) layer core on x (B,L,H,P) bf16; ``params`` holds
    dt_bias, A_log, D (H,) float32; ``segments`` = 0 lets the library cut the
    sequence for the current device.  Returns (y, h_out (B,H,P,N)).

    With ``check`` (the default) the call waits for the device and reads the
    walk's error flag from the workspace, raising ``AxonError``
    (AXON_ERR_TIMEOUT) if a wait for a tensor-core product gave up, in which
    case y and h_out are undefined.  ``check=False`` returns without waiting;
    the caller then reads the flag with ``ssd_error_flag(workspace)``."""
    Bsz, L, H, P = x.shape
    N = Bm.shape[2]
    if out is None:
        y = torch.empty_like(x)
        h_out = torch.empty(Bsz, H, P, N, dtype=torch.float32, device=x.device)
    else:
        y, h_out = out
    if workspace is None:
        with torch.cuda.device(x.device):
            nbytes = axon_ssd_workspace_bytes(Bsz, L, H, P, N, segments)
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=x.device)
    axon_ssd_scan_fwd(Bsz, L, H, P, N, _dtype_code(x.dtype), x, dt_raw, params["dt_bias"], params["A_log"],
                      Bm, Cm, params["D"], h0, y, h_out, segments, workspace,
                      workspace.numel() * workspace.element_size(), stream=stream)
    if check and L > 0 and Bsz * H > 0 and ssd_error_flag(workspace) != 0:
        raise AxonError(6, "axon_ssd_scan_fwd (a wait for a tensor-core product gave up)")
    return y, h_out


# ------------------------------------------------------------ gated delta rule, grouped norm
def _same_device(what, dev, **tensors):
    if dev.type != "cuda":
        raise ValueError(f"{what}: the inputs are on {dev}; a CUDA device is needed")
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{what}: {name} is on {t.device}, not on {dev}")


def _like(what, dtype, **tensors):
    for name, (t, shape, *kind) in tensors.items():
        if t is None:
            continue
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{what}: {name} has shape {tuple(t.shape)}, not {tuple(shape)}")
        want = kind[0] if kind else dtype
        if t.dtype != want:
            raise TypeError(f"{what}: {name} is {t.dtype}, not {want}")


_INT_MAX = 2 ** 31 - 1         # of a count or stride: ctypes would keep the low 32 bits of more without a word


def _stride_fits(what, name, ld):
    if ld > _INT_MAX:
        raise ValueError(f"{what}: the stride of {name} is {ld} elements, more than 2^31 - 1")
    return ld


def _token_stride(what, name, t):
    """Elements between consecutive tokens of a (B, L, heads, D) or (B, heads,
    D) tensor whose heads are dense and whose tokens lie at one stride (a slice
    of a projected row, say)."""
    heads, d = t.shape[-2:]
    ld, n = heads * d, 1
    for i in range(t.dim() - 3, -1, -1):
        if t.shape[i] > 1 and n == 1:
            ld, n = t.stride(i), t.shape[i]
        elif t.shape[i] > 1:
            if t.stride(i) != ld * n:
                raise ValueError(f"{what}: the tokens of {name} do not lie at one stride")
            n *= t.shape[i]
    if (d > 1 and t.stride(-1) != 1) or (heads > 1 and t.stride(-2) != d):
        raise ValueError(f"{what}: the heads of {name} must be dense")
    return _stride_fits(what, name, ld)


def _empty(stream, dev, *specs):
    """Tensors ((shape, dtype), ...) for a call on `stream`.  Another stream
    than the current one gets memory of its own pool (a block of the current
    stream's might still be in use there), marked as used on the current one
    too, where the caller reads it."""
    if stream is None:
        return [torch.empty(shape, dtype=dtype, device=dev) for shape, dtype in specs]
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=dev)
    with torch.cuda.stream(s):
        made = [torch.empty(shape, dtype=dtype, device=dev) for shape, dtype in specs]
    for t in made:
        t.record_stream(torch.cuda.current_stream(dev))
    return made


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_on(stream, index):
    """The raw stream handle; the current one of the (current) device `index` by default."""
    return _raw_stream(index) if stream is None and _raw_stream is not None else _stream(stream)


def _all_as(dtype, index, *tensors):
    """Whether all tensors are of this dtype on this device, and dense."""
    for t in tensors:
        if t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
            return False
    return True


def _delta_args(what, lead_dims, q, k, v, dt_raw, b_raw, params):
    """Sizes and pointer arguments, checked (small calls are bound by this code:
    the common case is looked over in one go, the rest explains itself).
    ``lead_dims``: dimensions before the heads, (B, L) or (B,); with others the
    sizes below would be read off the wrong ones."""
    bias, a_log = params["dt_bias"], params["A_log"]
    if v.dim() != lead_dims + 2:
        raise ValueError(f"{what}: v has {v.dim()} dimensions, not {lead_dims + 2}")
    dt, i = v.dtype, v.get_device()
    *lead, H, P = v.shape
    G, N = k.shape[-2:]
    rates = (*lead, H)
    fine = (i >= 0 and q.shape == k.shape == (*lead, G, N) and dt_raw.shape == b_raw.shape == rates and
            bias.shape == a_log.shape == (H,) and _all_as(torch.float32, i, bias, a_log) and _all_as(dt, i, dt_raw, b_raw))
    if fine and _all_as(dt, i, q, k, v):
        ldq = ldk = G * N
        ldv = H * P
    else:
        dev = v.device
        _same_device(what, dev, q=q, k=k, dt_raw=dt_raw, b_raw=b_raw, dt_bias=bias, A_log=a_log)
        f32 = torch.float32
        _like(what, dt, q=(q, (*lead, G, N)), k=(k, (*lead, G, N)), dt_raw=(dt_raw, rates), b_raw=(b_raw, rates),
              dt_bias=(bias, (H,), f32), A_log=(a_log, (H,), f32))
        for t in (dt_raw, b_raw, bias, a_log):
            if not t.is_contiguous():
                raise ValueError(f"{what}: the rates and parameters must be contiguous")
        ldq, ldk, ldv = (_token_stride(what, n, t) for n, t in (("q", q), ("k", k), ("v", v)))
    return i, H, P, G, N, _dtype_code(dt), (q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, dt_raw.data_ptr(),
                                            b_raw.data_ptr(), bias.data_ptr(), a_log.data_ptr())


def delta_error_flag(workspace) -> int:
    """The delta rule's error flag (the workspace's first int) after the call
    that used ``workspace`` has completed: bit 0 a wait gave up, bit 1 with raw
    keys y or the state is not finite.  Synchronises the device."""
    torch.cuda.synchronize(workspace.device)
    return int(workspace.view(-1).view(torch.uint8)[:4].view(torch.int32).item())


def _finite_tokens(lengths, values, gates, params, h0) -> bool:
    """Whether the rows' tokens, the parameters and the state are numbers (a gate may be infinite)."""
    L = values[0].shape[1]
    behind = None if lengths is None else torch.arange(L, device=lengths.device) >= lengths[:, None]
    for t in (*values, *gates):
        bad = t.isnan() if t.dim() == 3 else ~t.isfinite()
        bad = bad.flatten(2).any(-1)
        if bool((bad if behind is None else bad & ~behind).any()):
            return False
    return not any(bool(t.isnan().any()) for t in params.values()) and (h0 is None or bool(h0.isfinite().all()))


def delta_scan(q, k, v, dt_raw, b_raw, params: dict, h0=None, *, lengths=None, scale=None, qk_norm=True, out=None,
               workspace=None, stream=None, segments=0, check=True):
    """Gated delta rule prefill: q, k (B,L,G,N), v (B,L,H,P), dt_raw, b_raw
    (B,L,H); ``params`` holds dt_bias, A_log (H,) float32.  Returns
    ``(y (B,L,H,P), h_out (B,H,P,N))``, h_out ready for the next call or for
    ``delta_step``.

    q, k and v may be slices of one projected row (dense heads, tokens at one
    stride).  ``lengths`` ((B,) int32 on the device) ends rows early: y behind
    a row's end is left as it was (undefined where y is allocated here).
    ``scale`` defaults to N^(-1/2); ``segments`` = 0 lets the library cut the
    sequence for the current device.  ``out`` = (y, h_out); h_out may be h0.
    bf16 sequences but short ones go in chunks on the tensor cores, which need
    ``workspace`` and may fail; float32 and short ones go token by token.  In
    chunks the call waits, with ``check``, for the device and raises AxonError:
    AXON_ERR_TIMEOUT if a wait of a kernel gave up, AXON_ERR_UNSUPPORTED if with
    ``qk_norm=False`` an operand left fp16's range (keys longer than about 4 can
    do that).  ``check=False``, and every call token by token, returns at once
    (read the flag with ``delta_error_flag(workspace)``).
    """
    i, H, P, G, N, io, args = _delta_args("delta_scan", 2, q, k, v, dt_raw, b_raw, params)
    if i != _current_device():
        with torch.cuda.device(i):
            return delta_scan(q, k, v, dt_raw, b_raw, params, h0, lengths=lengths, scale=scale, qk_norm=qk_norm,
                              out=out, workspace=workspace, stream=stream, segments=segments, check=check)
    Bsz, L = v.shape[:2]
    dev, f32 = v.device, torch.float32
    nbytes = _lib.axon_delta_workspace_bytes(Bsz, L, H, G, P, N, io, segments)
    state = (Bsz, H, P, N)
    made = _empty(stream, dev, *(((v.shape, v.dtype), (state, f32)) if out is None else ()),
                  *(((nbytes,), torch.uint8),) * (workspace is None and nbytes > 0))
    y, h_out = out if out is not None else made[:2]
    given = workspace is not None
    if not given and nbytes > 0:
        workspace = made[-1]
    if given or out is not None or h0 is not None or lengths is not None:
        _same_device("delta_scan", dev, h0=h0, lengths=lengths, y=y, h_out=h_out, workspace=workspace)
        _like("delta_scan", f32, h0=(h0, state), h_out=(h_out, state), y=(y, v.shape, v.dtype),
              lengths=(lengths, (Bsz,), torch.int32))
    wsz = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.axon_delta_scan_fwd(Bsz, L, H, G, P, N, io, *args, _p(lengths), _p(h0),
                                    N ** -0.5 if scale is None else scale, qk_norm, _p(y), _p(h_out), segments,
                                    _p(workspace), wsz, _stream_on(stream, i)), "axon_delta_scan_fwd")
    if check and nbytes > 0:
        flag = delta_error_flag(workspace)
        if flag & 1:
            raise AxonError(6, "axon_delta_scan_fwd (a wait for a copy or a tensor-core product gave up)")
        if flag and _finite_tokens(lengths, (q, k, v), (dt_raw, b_raw), params, None if h0 is h_out else h0):
            raise AxonError(2, "axon_delta_scan_fwd (not finite: keys too long for the products' fp16 range)")
    return y, h_out


def delta_step(q, k, v, dt_raw, b_raw, params: dict, state, *, scale=None, qk_norm=True, y=None, stream=None):
    """One cached step of the gated delta rule: q, k (B,G,N), v (B,H,P),
    dt_raw, b_raw (B,H); ``state`` (B,H,P,N) float32 is updated in place.
    Returns y (B,H,P)."""
    i, H, P, G, N, io, args = _delta_args("delta_step", 1, q, k, v, dt_raw, b_raw, params)
    if i != _current_device():
        with torch.cuda.device(i):
            return delta_step(q, k, v, dt_raw, b_raw, params, state, scale=scale, qk_norm=qk_norm, y=y, stream=stream)
    Bsz = v.shape[0]
    if y is None:
        y = _empty(stream, v.device, (v.shape, v.dtype))[0]
    elif y.shape != v.shape or y.dtype is not v.dtype or y.get_device() != i:
        _same_device("delta_step", v.device, y=y)
        _like("delta_step", v.dtype, y=(y, v.shape))
    if state.shape != (Bsz, H, P, N) or state.dtype is not torch.float32 or state.get_device() != i:
        _same_device("delta_step", v.device, state=state)
        _like("delta_step", torch.float32, state=(state, (Bsz, H, P, N)))
    _check(_lib.axon_delta_step(Bsz, H, G, P, N, io, *args, N ** -0.5 if scale is None else scale, qk_norm, _p(state),
                                _p(y), _stream_on(stream, i)), "axon_delta_step")
    return y


NORM_KINDS = {"rms": 0, "group": 1}
NORM_GATES = {"after": 1, "before": 2}


def _row_stride(what, name, t, rows, C):
    """(elements between the rows) of a (..., C) tensor whose rows lie at one stride."""
    t2 = t.view(rows, C) if t.is_contiguous() or t.dim() == 2 else None
    if t2 is None:
        ld, n = C, 1
        for i in range(t.dim() - 2, -1, -1):
            if t.shape[i] > 1 and n == 1:
                ld, n = t.stride(i), t.shape[i]
            elif t.shape[i] > 1:
                if t.stride(i) != ld * n:
                    raise ValueError(f"{what}: the rows of {name} do not lie at one stride")
                n *= t.shape[i]
    else:
        ld = t2.stride(0) if rows > 1 else C
    if C > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what}: the channels of {name} must be dense")
    return _stride_fits(what, name, ld)


def gated_norm(x, weight=None, z=None, *, bias=None, group=None, kind="rms", gate="after", act=True, eps=1e-6,
               out=None, stream=None):
    """Grouped norm of channels-last rows x (..., C) with a SiLU gate or
    activation: statistics per row and ``group`` channels (default C).

    ``kind``: "rms" or "group" (mean and variance).  With z (same shape):
    ``gate`` "after" gives norm(x) f(z), "before" the norm of x f(z); without
    z the result is f(norm(x)).  f is SiLU with ``act``, else the identity.
    weight, bias: float32, (group,) shared by the groups or (C,); both of one
    form.  x, z and out may be slices with a row stride; out may be x or z.
    """
    C = x.shape[-1]
    D = C if group is None else group
    i = x.get_device()
    if i < 0:
        _same_device("gated_norm", x.device)
    if i != _current_device():
        with torch.cuda.device(i):
            return gated_norm(x, weight, z, bias=bias, group=group, kind=kind, gate=gate, act=act, eps=eps, out=out,
                              stream=stream)
    y = _empty(stream, x.device, (x.shape, x.dtype))[0] if out is None else out
    n = D if weight is None and bias is None else (bias if weight is None else weight).shape[0]
    if n != D and n != C:
        raise ValueError(f"gated_norm: weight and bias need {D} or {C} values, not {n}")
    rows = x.numel() // C if C else 0
    if rows > _INT_MAX or C > _INT_MAX or D > _INT_MAX:
        raise AxonError(2, "axon_gated_norm_fwd")
    params = [t for t in (weight, bias) if t is not None]
    data = [x, y] if z is None else [x, y, z]
    if (_all_as(torch.float32, i, *params) and all(t.shape == (n,) for t in params) and _all_as(x.dtype, i, *data) and
            all(t.shape == x.shape for t in data)):
        ldx = ldy = ldz = C
    else:
        _same_device("gated_norm", x.device, weight=weight, bias=bias, z=z, out=y)
        _like("gated_norm", torch.float32, weight=(weight, (n,)), bias=(bias, (n,)), z=(z, x.shape, x.dtype),
              out=(y, x.shape, x.dtype))
        for t in params:
            if not t.is_contiguous():
                raise ValueError("gated_norm: weight and bias must be contiguous")
        ldx, ldy, ldz = (0 if t is None else _row_stride("gated_norm", name, t, rows, C)
                         for name, t in (("x", x), ("out", y), ("z", z)))
    _check(_lib.axon_gated_norm_fwd(rows, C, D, _dtype_code(x.dtype), NORM_KINDS[kind], 0 if z is None else NORM_GATES[gate],
                                    act, x.data_ptr(), ldx, _v(z), ldz, _p(weight), _p(bias),
                                    n == C and n != D, eps, y.data_ptr(), ldy, _stream_on(stream, i)), "axon_gated_norm_fwd")
    return y
