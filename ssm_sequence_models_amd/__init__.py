"""Thin Python binding of libssm_mi355x.so (the C ABI in include/ssm_mi355x.h).

Argument marshalling only: this module checks devices / dtypes / shapes of torch tensors,
allocates outputs and workspaces with torch (device memory and streams are PyTorch's
plumbing), and calls the C entry point of the same name on the current HIP stream.  Every
step of the computation runs in the library's HIP kernels; there is no fallback, and the
import fails loudly if the library has not been built.

Sources of the operations (page title and section): the length-generalization reading
notes on arXiv:2507.02782v2, Sec. 2.1 Eq. (1), Sec. 2.5 Eq. (4), Sec. 2.6 (scan with
initial / final state); the causal-conv1d tutorial ch. 7 (conv state S / F, decode update,
cache_seqlens, conv_state_indices, seq_idx, and the backward with state gradients).  The
scan's complete backward, the gated norm, the per-channel gated recurrence, the gated delta rule
and the norm of queries and keys are formed from the same equations; their formulas stand with
the declarations in the header.
"""
from __future__ import annotations

import contextlib
import ctypes
import operator
import os

import torch  # must precede the library load: it binds the process's HIP runtime

_HERE = os.path.dirname(os.path.abspath(__file__))
# SSM_LIB_PATH selects another build of the same sources (the host-sanitizer build of the
# argument checks runs the ABI tests against one)
LIB_PATH = os.environ.get("SSM_LIB_PATH") or os.path.join(_HERE, "libssm_mi355x.so")

SSM_F32, SSM_BF16 = 0, 1
ACT = {None: 0, "none": 0, "silu": 1}
_STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "misaligned pointer",
           4: "workspace", 5: "HIP error"}


# Debug checks of caller contracts the kernels do not verify (they cost a device-to-host
# copy): with SSM_DEBUG_CHECKS=1 in the environment (or DEBUG_CHECKS = True), the calls that
# update state pools refuse two active rows on one slot (causal-conv1d ch. 7, state indices
# for continuous batching: a duplicate is a caller error, undefined in the kernels).
DEBUG_CHECKS = os.environ.get("SSM_DEBUG_CHECKS", "") == "1"


def check_distinct_slots(indices, n_slots: int, name: str = "indices") -> None:
    """Raise ValueError if two entries of `indices` inside [0, n_slots) are equal (rows
    outside that range are skipped by the kernels and may repeat)."""
    if indices is None:
        return
    v = indices.detach().to("cpu").to(torch.int64)
    v = v[(v >= 0) & (v < n_slots)]
    if v.numel() != torch.unique(v).numel():
        vals, counts = torch.unique(v, return_counts=True)
        raise ValueError(f"{name}: slot(s) {vals[counts > 1].tolist()} used by more than one "
                         "active row")


class SSMError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str):
        super().__init__(f"{fn}: {_STATUS.get(status, status)}: {detail}")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it first (python ssm_sequence_models_amd/build.py "
            "or __graft_entry__.build()); there is no non-HIP fallback")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, i32p, fp = ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p
    ci = ctypes.c_int
    lib.ssm_abi_version.restype = ci
    lib.ssm_last_error.restype = ctypes.c_char_p
    lib.ssm_status_string.restype = ctypes.c_char_p
    lib.ssm_status_string.argtypes = [ci]
    lib.ssm_conv1d_fwd.argtypes = [vp, fp, fp, vp, vp, i32p, vp, i64, i64, i64, i64, ci, ci, vp]
    lib.ssm_conv1d_update.argtypes = [vp, vp, fp, fp, i32p, i32p, vp, i64, i64, i64, i64, i64,
                                      i64, ci, ci, vp]
    lib.ssm_scan_workspace_size.restype = ctypes.c_size_t
    lib.ssm_scan_workspace_size.argtypes = [i64, i64, i64, i64, i64, i64, ci]
    lib.ssm_scan_fwd.argtypes = [vp, fp, fp, vp, vp, fp, fp, i32p, vp, i64, i64, i64, i64, i64,
                                 i64, ci, vp, ctypes.c_size_t, vp]
    lib.ssm_conv_scan_fwd.argtypes = [vp, fp, fp, vp, vp, fp, fp, fp, fp, i32p, vp, i64, i64, i64,
                                      i64, i64, i64, i64, ci, ci, vp, ctypes.c_size_t, vp]
    lib.ssm_conv_scan_fwd_noalloc.argtypes = [vp, fp, fp, vp, vp, fp, fp, fp, fp, i32p, vp, i64,
                                              i64, i64, i64, i64, i64, i64, ci, ci, vp]
    lib.ssm_noalloc_scratch_bytes.restype = ctypes.c_size_t
    lib.ssm_noalloc_scratch_bytes.argtypes = []
    lib.ssm_step.argtypes = [vp, i64, i64, i64, fp, fp, vp, i64, i64, i64, vp, i64, i64, i64, fp,
                             i32p, vp, i64, i64, i64, i64, i64, i64, i64, ci, vp]
    lib.ssm_decode_step.argtypes = [vp, vp, fp, fp, i32p, i32p, fp, fp, fp, i32p, vp, vp, i64,
                                    i64, i64, i64, i64, i64, i64, i64, i64, i64, ci, ci, vp]
    lib.ssm_conv1d_bwd_workspace_size.restype = ctypes.c_size_t
    lib.ssm_conv1d_bwd_workspace_size.argtypes = [i64, i64, i64, i64]
    lib.ssm_conv1d_bwd.argtypes = [vp, fp, fp, vp, i32p, vp, vp, vp, vp, fp, fp, vp,
                                   ctypes.c_size_t, i64, i64, i64, i64, ci, ci, vp]
    lib.ssm_scan_bwd_initial_state.argtypes = [fp, fp, vp, vp, i32p, fp, fp, i64, i64, i64, i64,
                                               i64, i64, ci, vp]
    lib.ssm_conv_scan_fwd_pooled_workspace_size.restype = ctypes.c_size_t
    lib.ssm_conv_scan_fwd_pooled_workspace_size.argtypes = [i64, i64, i64, i64, i64, i64, i64, ci]
    lib.ssm_conv_scan_fwd_pooled.argtypes = [vp, fp, fp, fp, fp, vp, fp, i32p, i32p, i32p, vp,
                                             i64, i64, i64, i64, i64, i64, i64, i64, i64, ci, ci,
                                             vp, ctypes.c_size_t, vp]
    lib.ssm_scan_fwd_vector_decay.argtypes = [vp, fp, fp, fp, vp, vp, fp, fp, i32p, vp, i64, i64,
                                              i64, i64, i64, i64, ci, vp]
    u64 = ctypes.c_uint64
    lib.ssm_state_stats_update.argtypes = [fp, i64, i64, i64, i64, ctypes.c_float, fp, fp, vp]
    lib.ssm_initial_state_noise.argtypes = [fp, i64, i64, i64, i64, fp, fp, ctypes.c_float, u64,
                                            u64, vp]
    lib.ssm_state_reset.argtypes = [vp, vp, vp, i64, i64, ctypes.c_double, u64, u64, vp]
    cf, sz = ctypes.c_float, ctypes.c_size_t
    lib.ssm_norm_fwd.argtypes = [vp, i64, vp, i64, fp, fp, vp, i64, i64, i64, i64, cf, ci, ci, ci,
                                 vp]
    lib.ssm_norm_bwd_workspace_size.restype = sz
    lib.ssm_norm_bwd_workspace_size.argtypes = [i64, i64, i64]
    lib.ssm_norm_bwd.argtypes = [vp, i64, vp, i64, vp, i64, fp, fp, vp, i64, vp, i64, fp, fp, vp,
                                 sz, i64, i64, i64, cf, ci, ci, ci, vp]
    lib.ssm_scan_bwd_workspace_size.restype = sz
    lib.ssm_scan_bwd_workspace_size.argtypes = [i64, i64, i64, i64, i64, i64, ci]
    lib.ssm_scan_bwd.argtypes = [vp, fp, fp, vp, vp, vp, fp, fp, i32p, vp, fp, fp, vp, vp, fp, i64,
                                 i64, i64, i64, i64, i64, ci, vp, sz, vp]
    lib.ssm_gated_scan_fwd_workspace_size.restype = sz
    lib.ssm_gated_scan_fwd_workspace_size.argtypes = [i64, i64, i64]
    lib.ssm_gated_scan_fwd.argtypes = [vp, i64, vp, i64, fp, fp, i32p, vp, i64, i64, i64, i64, ci,
                                       ci, vp, sz, vp]
    lib.ssm_gated_scan_bwd_workspace_size.restype = sz
    lib.ssm_gated_scan_bwd_workspace_size.argtypes = [i64, i64, i64]
    lib.ssm_gated_scan_bwd.argtypes = [vp, i64, vp, i64, vp, i64, fp, fp, i32p, vp, i64, vp, i64,
                                       fp, i64, i64, i64, ci, ci, vp, sz, vp]
    lib.ssm_gated_scan_step.argtypes = [vp, i64, vp, i64, fp, i32p, vp, i64, i64, i64, i64, i64,
                                        ci, ci, vp]
    sizes = [i64, i64, i64, i64, i64, i64, ci]
    for f in (lib.ssm_delta_scan_fwd_workspace_size, lib.ssm_delta_scan_bwd_workspace_size):
        f.restype = sz
        f.argtypes = sizes
    qkv = [vp, i64, vp, i64, vp, i64, fp, fp, cf]
    lib.ssm_delta_scan_fwd.argtypes = qkv + [fp, fp, i32p, vp, i64] + sizes + [vp, sz, vp]
    lib.ssm_delta_scan_bwd.argtypes = qkv + [vp, i64, fp, fp, i32p, vp, i64, vp, i64, vp, i64, fp, fp,
                                             fp] + sizes + [vp, sz, vp]
    lib.ssm_delta_scan_step.argtypes = qkv + [fp, i32p, vp, i64, i64, i64, i64, i64, i64, i64, i64, ci,
                                              vp]
    qk = [vp, i64, vp, i64, fp, fp, fp, i32p]
    how = [i64, i64, i64, i64, i64, i64, ci, cf, ci, ci, vp]
    lib.ssm_qk_norm_fwd.argtypes = qk + [vp, i64, vp, i64] + how
    lib.ssm_qk_norm_bwd_workspace_size.restype = sz
    lib.ssm_qk_norm_bwd_workspace_size.argtypes = [i64, i64, i64]
    lib.ssm_qk_norm_bwd.argtypes = qk + [vp, i64, vp, i64, vp, i64, vp, i64, fp, fp, vp, sz] + how
    lib.ssm_stream_copy.argtypes = [vp, vp, i64, vp]
    lib.ssm_timing_enable.argtypes = [ci]
    lib.ssm_timing_read.argtypes = [ctypes.POINTER(ctypes.c_double),
                                    ctypes.POINTER(ctypes.c_int64)]
    for f in ("ssm_conv1d_fwd", "ssm_conv1d_update", "ssm_scan_fwd", "ssm_conv_scan_fwd",
              "ssm_conv_scan_fwd_noalloc", "ssm_step", "ssm_decode_step", "ssm_conv1d_bwd", "ssm_scan_bwd_initial_state",
              "ssm_conv_scan_fwd_pooled", "ssm_state_stats_update", "ssm_scan_fwd_vector_decay",
              "ssm_initial_state_noise", "ssm_state_reset", "ssm_stream_copy", "ssm_norm_fwd",
              "ssm_norm_bwd", "ssm_scan_bwd", "ssm_gated_scan_fwd", "ssm_gated_scan_bwd", "ssm_gated_scan_step",
              "ssm_delta_scan_fwd", "ssm_delta_scan_bwd", "ssm_delta_scan_step", "ssm_qk_norm_fwd",
              "ssm_qk_norm_bwd",
              "ssm_timing_enable", "ssm_timing_read"):
        getattr(lib, f).restype = ci
    return lib


_lib = _load()


def abi_version() -> int:
    return int(_lib.ssm_abi_version())


def _check(fn: str, status: int):
    if status != 0:
        raise SSMError(fn, status, _lib.ssm_last_error().decode())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SSM_BF16
    if t.dtype == torch.float32:
        return SSM_F32
    raise TypeError(f"activations must be bfloat16 or float32, got {t.dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    # the current stream's handle without a Stream object around it (2.9 us of a 15 us call)
    return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))


_CURRENT = contextlib.nullcontext()


def _on(device):
    """The device of a call's tensors made the current one; nothing to do where it is already."""
    return _CURRENT if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _need(t, name, dtype=None, shape=None, contiguous=True):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need_device(ref, **tensors):
    """Every given tensor lives on ref's device (the call is made on that device's current
    stream)."""
    for name, t in tensors.items():
        if t is not None and t.device != ref.device:
            raise ValueError(f"{name} must be on {ref.device}, got {t.device}")


def _rows(t, name, channels):
    """(rows, row stride) of t [..., channels]: its last dimension consecutive, the leading
    ones at one stride."""
    if t.dim() < 1 or t.shape[-1] != channels:
        raise ValueError(f"{name} must have {channels} channels, got shape {tuple(t.shape)}")
    if t.is_contiguous():
        return t.numel() // channels, channels
    if channels > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have consecutive channels")
    rows, row = 1, None
    for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if row is None:
            row = s
        elif s != row * rows:
            raise ValueError(f"{name} must have its rows at one stride")
        rows *= n
    return rows, channels if row is None else row


def workspace_size(batch, seqlen, nheads, headdim, ngroups, dstate, dtype=torch.bfloat16) -> int:
    code = SSM_BF16 if dtype == torch.bfloat16 else SSM_F32
    return int(_lib.ssm_scan_workspace_size(batch, seqlen, nheads, headdim, ngroups, dstate,
                                            code))


def _workspace(ws, nbytes, device):
    if nbytes == 0:
        return None, 0
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    # the kernels write nbytes from its first element on: repeated or skipped elements do not count
    if ws.device != device or not ws.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {device}")
    if ws.numel() * ws.element_size() < nbytes:
        raise ValueError(f"workspace must hold {nbytes} bytes")
    return ws, ws.numel() * ws.element_size()


def conv1d_fwd(x, weight, bias=None, initial_state=None, seq_idx=None, activation=None,
               return_final_state=True, final_state=None, out=None):
    """x [B, L, C] (bf16 / fp32, channel-last); weight [C, K] fp32; bias [C] fp32;
    initial_state [B, C, K-1]; seq_idx [B, L] int32.  Returns (out, final_state)."""
    B, L, C = x.shape
    K = weight.shape[1]
    _need(x, "x")
    _need(weight, "weight", torch.float32, (C, K))
    _need(bias, "bias", torch.float32, (C,))
    _need(initial_state, "initial_state", x.dtype, (B, C, K - 1))
    _need(seq_idx, "seq_idx", torch.int32, (B, L))
    if out is None:
        out = torch.empty_like(x)
    _need(out, "out", x.dtype, (B, L, C))
    if final_state is None and return_final_state:
        final_state = torch.empty((B, C, K - 1), dtype=x.dtype, device=x.device)
    _need(final_state, "final_state", x.dtype, (B, C, K - 1))
    _check("ssm_conv1d_fwd", _lib.ssm_conv1d_fwd(
        _ptr(x), _ptr(weight), _ptr(bias), _ptr(initial_state), _ptr(final_state), _ptr(seq_idx),
        _ptr(out), B, L, C, K, _dtype_code(x), ACT[activation], _stream()))
    return out, final_state


def conv_scan_fwd_pooled(xBC, conv_weight, conv_bias, dt, A, conv_state, ssm_state, nheads,
                         headdim, ngroups, dstate, state_indices=None, cache_seqlens=None,
                         seq_idx=None, activation="silu", y=None, workspace=None):
    """The fused prefill on the decode pools: row b's initial conv history and SSM state come
    from slot state_indices[b] (ring position cache_seqlens[b], or the linear layout), and its
    new raw inputs and final state go back there.  conv_state [n_slots, C_conv, state_len]
    (xBC's dtype) and ssm_state [n_slots, H, P, N] fp32 update in place; cache_seqlens is not
    advanced.  Returns y [b, L, H, P]."""
    b, L, C_conv = xBC.shape
    K = conv_weight.shape[1]
    n_slots, _, state_len = conv_state.shape
    H, P, G, N = nheads, headdim, ngroups, dstate
    _need(xBC, "xBC")
    _need(conv_weight, "conv_weight", torch.float32, (C_conv, K))
    _need(conv_bias, "conv_bias", torch.float32, (C_conv,))
    _need(dt, "dt", torch.float32, (b, L, H))
    _need(A, "A", torch.float32, (H,))
    _need(conv_state, "conv_state", xBC.dtype, (n_slots, C_conv, state_len))
    _need(ssm_state, "ssm_state", torch.float32, (n_slots, H, P, N))
    _need(state_indices, "state_indices", torch.int32, (b,))
    if DEBUG_CHECKS:
        check_distinct_slots(state_indices, ssm_state.shape[0], "state_indices")
    _need(cache_seqlens, "cache_seqlens", torch.int32, (b,))
    _need(seq_idx, "seq_idx", torch.int32, (b, L))
    if y is None:
        y = torch.empty((b, L, H, P), dtype=xBC.dtype, device=xBC.device)
    _need(y, "y", xBC.dtype, (b, L, H, P))
    nbytes = int(_lib.ssm_conv_scan_fwd_pooled_workspace_size(b, L, H, P, G, N, K, _dtype_code(xBC)))
    if workspace is None:
        workspace = torch.empty(nbytes + 256, dtype=torch.uint8, device=xBC.device)
    off = (-workspace.data_ptr()) % 256
    if workspace.numel() - off < nbytes:
        raise ValueError(f"workspace must hold {nbytes} bytes past a 256-byte boundary")
    _check("ssm_conv_scan_fwd_pooled", _lib.ssm_conv_scan_fwd_pooled(
        _ptr(xBC), _ptr(conv_weight), _ptr(conv_bias), _ptr(dt), _ptr(A), _ptr(conv_state),
        _ptr(ssm_state), _ptr(state_indices), _ptr(cache_seqlens), _ptr(seq_idx), _ptr(y), b, L,
        H, P, G, N, K, state_len, n_slots, _dtype_code(xBC), ACT[activation],
        ctypes.c_void_p(workspace.data_ptr() + off), workspace.numel() - off, _stream()))
    return y


def conv_scan_fwd_pooled_workspace_size(batch, seqlen, nheads, headdim, ngroups, dstate, width,
                                        dtype=torch.bfloat16) -> int:
    code = SSM_BF16 if dtype == torch.bfloat16 else SSM_F32
    return int(_lib.ssm_conv_scan_fwd_pooled_workspace_size(batch, seqlen, nheads, headdim, ngroups,
                                                            dstate, width, code))


def scan_fwd_vector_decay(x, B, C, log_decay=None, A_vec=None, dt=None, initial_state=None,
                          seq_idx=None, return_final_state=True, final_state=None, y=None):
    """The scan with a diagonal transition, one decay per state dimension (length-
    generalization notes Sec. 2.1 Eq. (1) with A_t = diag(a_t), Sec. 2.5): log a_t[n] from
    log_decay [b, L, H, N] fp32, or dt * A_vec [H, N].  x [b, L, H, P]; B, C [b, L, G, N];
    dt [b, L, H] fp32 or None (= 1).  Returns (y [b, L, H, P], final_state or None)."""
    bsz, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    _need(x, "x")
    _need(B, "B", x.dtype, (bsz, L, G, N))
    _need(C, "C", x.dtype, (bsz, L, G, N))
    _need(log_decay, "log_decay", torch.float32, (bsz, L, H, N))
    _need(A_vec, "A_vec", torch.float32, (H, N))
    _need(dt, "dt", torch.float32, (bsz, L, H))
    _need(initial_state, "initial_state", torch.float32, (bsz, H, P, N))
    _need(seq_idx, "seq_idx", torch.int32, (bsz, L))
    if y is None:
        y = torch.empty((bsz, L, H, P), dtype=x.dtype, device=x.device)
    _need(y, "y", x.dtype, (bsz, L, H, P))
    if return_final_state and final_state is None:
        final_state = torch.empty((bsz, H, P, N), dtype=torch.float32, device=x.device)
    _need(final_state, "final_state", torch.float32, (bsz, H, P, N))
    _check("ssm_scan_fwd_vector_decay", _lib.ssm_scan_fwd_vector_decay(
        _ptr(x), _ptr(dt), _ptr(log_decay), _ptr(A_vec), _ptr(B), _ptr(C), _ptr(initial_state),
        _ptr(final_state), _ptr(seq_idx), _ptr(y), bsz, L, H, P, G, N, _dtype_code(x),
        _stream()))
    return y, final_state

def state_stats_update(final_state, mean, var, beta=0.1):
    """Fitted Noise statistics (length-generalization notes Sec. 2.6, Eqs. (5)-(6)): per head,
    mean <- (1 - beta) Mean(final_state) + beta mean, var likewise with the population
    variance, over batch rows, channels and state dimension.  final_state [b, H, P, N] fp32;
    mean, var [H] fp32, updated in place and returned."""
    b, H, P, N = final_state.shape
    _need(final_state, "final_state", torch.float32)
    _need(mean, "mean", torch.float32, (H,))
    _need(var, "var", torch.float32, (H,))
    _check("ssm_state_stats_update", _lib.ssm_state_stats_update(
        _ptr(final_state), b, H, P, N, float(beta), _ptr(mean), _ptr(var), _stream()))
    return mean, var


def initial_state_noise(batch, nheads, headdim, dstate, mean=None, var=None, sigma=1.0, seed=0,
                        offset=0, out=None, device="cuda"):
    """Noise initial states (Sec. 2.6): Fitted Noise N(mean[h], var[h]) per head when mean and
    var [H] are given, Random Noise N(0, sigma^2) otherwise, drawn from Philox4x64-10 with
    (seed, offset).  Returns out [batch, H, P, N] fp32."""
    shape = (batch, nheads, headdim, dstate)
    if out is None:
        out = torch.empty(shape, dtype=torch.float32, device=device)
    _need(out, "out", torch.float32, shape)
    _need(mean, "mean", torch.float32, (nheads,))
    _need(var, "var", torch.float32, (nheads,))
    _check("ssm_initial_state_noise", _lib.ssm_initial_state_noise(
        _ptr(out), batch, nheads, headdim, dstate, _ptr(mean), _ptr(var), float(sigma),
        int(seed) & (2**64 - 1), int(offset) & (2**64 - 1), _stream()))
    return out


def state_reset(state, p=0.1, seed=0, offset=0, out=None, mask=None):
    """State Passing's occasional reset (Sec. 2.6): each row of state [b, ...] (any dtype) is
    zeroed with probability p, decided by (seed, offset, row) alone.  out may be state itself.
    Returns (out, mask [b] uint8, 1 = zeroed)."""
    b = state.shape[0]
    _need(state, "state")
    if out is None:
        out = torch.empty_like(state)
    _need(out, "out", state.dtype, tuple(state.shape))
    if mask is None:
        mask = torch.empty(b, dtype=torch.uint8, device=state.device)
    _need(mask, "mask", torch.uint8, (b,))
    row_bytes = state[0].numel() * state.element_size() if b > 0 else 0
    _check("ssm_state_reset", _lib.ssm_state_reset(
        _ptr(state), _ptr(out), _ptr(mask), b, row_bytes, float(p), int(seed) & (2**64 - 1),
        int(offset) & (2**64 - 1), _stream()))
    return out, mask

def conv1d_bwd(x, weight, bias, dout, initial_state=None, dfinal_state=None, seq_idx=None,
               activation=None, dx=None, dinitial_state=None, dweight=None, dbias=None,
               workspace=None):
    """Backward of conv1d_fwd with state gradients.  x, dout [B, L, C]; weight [C, K] fp32;
    bias [C] fp32 or None; initial_state, dfinal_state [B, C, K-1] (None = zero); seq_idx
    [B, L] int32.  Returns (dx [B, L, C], dinitial_state [B, C, K-1], dweight [C, K] fp32,
    dbias [C] fp32)."""
    B, L, C = x.shape
    K = weight.shape[1]
    _need(x, "x")
    _need(weight, "weight", torch.float32, (C, K))
    _need(bias, "bias", torch.float32, (C,))
    _need(dout, "dout", x.dtype, (B, L, C))
    _need(initial_state, "initial_state", x.dtype, (B, C, K - 1))
    _need(dfinal_state, "dfinal_state", x.dtype, (B, C, K - 1))
    _need(seq_idx, "seq_idx", torch.int32, (B, L))
    if dx is None:
        dx = torch.empty_like(x)
    if dinitial_state is None:
        dinitial_state = torch.empty((B, C, K - 1), dtype=x.dtype, device=x.device)
    if dweight is None:
        dweight = torch.empty((C, K), dtype=torch.float32, device=x.device)
    if dbias is None:
        dbias = torch.empty((C,), dtype=torch.float32, device=x.device)
    _need(dx, "dx", x.dtype, (B, L, C))
    _need(dinitial_state, "dinitial_state", x.dtype, (B, C, K - 1))
    _need(dweight, "dweight", torch.float32, (C, K))
    _need(dbias, "dbias", torch.float32, (C,))
    nbytes = int(_lib.ssm_conv1d_bwd_workspace_size(B, L, C, K))
    ws, wsb = _workspace(workspace, nbytes, x.device)
    _check("ssm_conv1d_bwd", _lib.ssm_conv1d_bwd(
        _ptr(x), _ptr(weight), _ptr(bias), _ptr(initial_state), _ptr(seq_idx), _ptr(dout),
        _ptr(dfinal_state), _ptr(dx), _ptr(dinitial_state), _ptr(dweight), _ptr(dbias),
        _ptr(ws), wsb, B, L, C, K, _dtype_code(x), ACT[activation], _stream()))
    return dx, dinitial_state, dweight, dbias


def conv1d_bwd_workspace_size(batch, seqlen, channels, width) -> int:
    return int(_lib.ssm_conv1d_bwd_workspace_size(batch, seqlen, channels, width))


def scan_bwd_initial_state(dt, A, C, dy, dfinal_state=None, seq_idx=None, out=None):
    """Gradient of the scan's initial state.  dt [b, L, H] fp32; A [H] fp32; C [b, L, G, N];
    dy [b, L, H, P] (C's dtype); dfinal_state [b, H, P, N] fp32 or None; seq_idx [b, L]
    int32.  Returns dinitial_state [b, H, P, N] fp32 (out may be dfinal_state itself)."""
    b, L, H, P = dy.shape
    G, N = C.shape[2], C.shape[3]
    _need(dt, "dt", torch.float32, (b, L, H))
    _need(A, "A", torch.float32, (H,))
    _need(C, "C", dy.dtype, (b, L, G, N))
    _need(dy, "dy")
    _need(dfinal_state, "dfinal_state", torch.float32, (b, H, P, N))
    _need(seq_idx, "seq_idx", torch.int32, (b, L))
    if out is None:
        out = torch.empty((b, H, P, N), dtype=torch.float32, device=dy.device)
    _need(out, "out", torch.float32, (b, H, P, N))
    _check("ssm_scan_bwd_initial_state", _lib.ssm_scan_bwd_initial_state(
        _ptr(dt), _ptr(A), _ptr(C), _ptr(dy), _ptr(seq_idx), _ptr(dfinal_state), _ptr(out),
        b, L, H, P, G, N, _dtype_code(dy), _stream()))
    return out


def conv1d_update(x, conv_state, weight, bias=None, conv_state_indices=None,
                  cache_seqlens=None, activation=None, out=None):
    """x [B, C, L_new]; conv_state [n_slots, C, state_len] (updated in place);
    conv_state_indices, cache_seqlens [B] int32 (cache_seqlens is not advanced).
    Returns out [B, C, L_new]."""
    B, C, L_new = x.shape
    n_slots, _, state_len = conv_state.shape
    K = weight.shape[1]
    _need(x, "x")
    _need(conv_state, "conv_state", x.dtype, (n_slots, C, state_len))
    _need(weight, "weight", torch.float32, (C, K))
    _need(bias, "bias", torch.float32, (C,))
    _need(conv_state_indices, "conv_state_indices", torch.int32, (B,))
    if DEBUG_CHECKS:
        check_distinct_slots(conv_state_indices, conv_state.shape[0], "conv_state_indices")
    _need(cache_seqlens, "cache_seqlens", torch.int32, (B,))
    if out is None:
        out = torch.empty_like(x)
    _need(out, "out", x.dtype, (B, C, L_new))
    _check("ssm_conv1d_update", _lib.ssm_conv1d_update(
        _ptr(x), _ptr(conv_state), _ptr(weight), _ptr(bias), _ptr(conv_state_indices),
        _ptr(cache_seqlens), _ptr(out), B, C, L_new, K, state_len, n_slots, _dtype_code(x),
        ACT[activation], _stream()))
    return out


def scan_fwd(x, dt, A, B, C, initial_state=None, seq_idx=None, return_final_state=True,
             final_state=None, y=None, workspace=None):
    """x [b, L, H, P]; dt [b, L, H] fp32; A [H] fp32; B, C [b, L, G, N]; initial_state
    [b, H, P, N] fp32 (may be the same tensor as final_state).  Returns (y, final_state)."""
    bsz, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    _need(x, "x")
    _need(dt, "dt", torch.float32, (bsz, L, H))
    _need(A, "A", torch.float32, (H,))
    _need(B, "B", x.dtype, (bsz, L, G, N))
    _need(C, "C", x.dtype, (bsz, L, G, N))
    _need(initial_state, "initial_state", torch.float32, (bsz, H, P, N))
    _need(seq_idx, "seq_idx", torch.int32, (bsz, L))
    if y is None:
        y = torch.empty_like(x)
    _need(y, "y", x.dtype, (bsz, L, H, P))
    if final_state is None and return_final_state:
        final_state = torch.empty((bsz, H, P, N), dtype=torch.float32, device=x.device)
    _need(final_state, "final_state", torch.float32, (bsz, H, P, N))
    ws, nbytes = _workspace(workspace, workspace_size(bsz, L, H, P, G, N, x.dtype), x.device)
    _check("ssm_scan_fwd", _lib.ssm_scan_fwd(
        _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(initial_state), _ptr(final_state),
        _ptr(seq_idx), _ptr(y), bsz, L, H, P, G, N, _dtype_code(x), _ptr(ws), nbytes, _stream()))
    return y, final_state


def conv_scan_fwd(xBC, conv_weight, conv_bias, dt, A, nheads, headdim, ngroups, dstate,
                  conv_initial_state=None, initial_state=None, seq_idx=None,
                  activation="silu", return_final_states=True, conv_final_state=None,
                  final_state=None, y=None, workspace=None, norm=None):
    """The fused prefill.  xBC [b, L, H*P + 2*G*N] (x | B | C channels); conv_weight
    [C_conv, K] fp32; conv_bias [C_conv]; dt [b, L, H]; A [H]; conv states [b, C_conv, K-1];
    SSM states [b, H, P, N] fp32.  Returns (y [b, L, H, P], conv_final_state, final_state); with
    norm (a dict of norm_fwd's keyword arguments) y normed and gated over its H*P channels,
    [b, L, H*P], in y's place."""
    bsz, L, Cc = xBC.shape
    H, P, G, N = nheads, headdim, ngroups, dstate
    if Cc != H * P + 2 * G * N:
        raise ValueError("xBC channel count must be nheads*headdim + 2*ngroups*dstate")
    K = conv_weight.shape[1]
    _need(xBC, "xBC")
    _need(conv_weight, "conv_weight", torch.float32, (Cc, K))
    _need(conv_bias, "conv_bias", torch.float32, (Cc,))
    _need(conv_initial_state, "conv_initial_state", xBC.dtype, (bsz, Cc, K - 1))
    _need(dt, "dt", torch.float32, (bsz, L, H))
    _need(A, "A", torch.float32, (H,))
    _need(initial_state, "initial_state", torch.float32, (bsz, H, P, N))
    _need(seq_idx, "seq_idx", torch.int32, (bsz, L))
    if y is None:
        y = torch.empty((bsz, L, H, P), dtype=xBC.dtype, device=xBC.device)
    _need(y, "y", xBC.dtype, (bsz, L, H, P))
    if return_final_states:
        if conv_final_state is None:
            conv_final_state = torch.empty((bsz, Cc, K - 1), dtype=xBC.dtype, device=xBC.device)
        if final_state is None:
            final_state = torch.empty((bsz, H, P, N), dtype=torch.float32, device=xBC.device)
    _need(conv_final_state, "conv_final_state", xBC.dtype, (bsz, Cc, K - 1))
    _need(final_state, "final_state", torch.float32, (bsz, H, P, N))
    ws, nbytes = _workspace(workspace, workspace_size(bsz, L, H, P, G, N, xBC.dtype), xBC.device)
    normed = None if norm is None else _norm_plan(y.view(bsz, L, H * P), **norm)[1]
    with _on(xBC.device):  # the norm reads y on the same stream
        _check("ssm_conv_scan_fwd", _lib.ssm_conv_scan_fwd(
            _ptr(xBC), _ptr(conv_weight), _ptr(conv_bias), _ptr(conv_initial_state),
            _ptr(conv_final_state), _ptr(dt), _ptr(A), _ptr(initial_state), _ptr(final_state),
            _ptr(seq_idx), _ptr(y), bsz, L, H, P, G, N, K, _dtype_code(xBC), ACT[activation],
            _ptr(ws), nbytes, _stream()))
        return y if normed is None else normed(), conv_final_state, final_state


def noalloc_scratch_bytes() -> int:
    """Bytes of the library's static per-GPU scratch that conv_scan_fwd_noalloc works in."""
    return int(_lib.ssm_noalloc_scratch_bytes())


def conv_scan_fwd_noalloc(xBC, conv_weight, conv_bias, dt, A, nheads, headdim, ngroups, dstate,
                          y, conv_final_state=None, final_state=None, conv_initial_state=None,
                          initial_state=None, seq_idx=None, activation="silu"):
    """conv_scan_fwd without a workspace: the library works in its static per-GPU scratch
    (noalloc_scratch_bytes()), so nothing is allocated; the caller passes y and the final-state
    buffers it wants (None: not written).  Calls that may overlap on one GPU race on the
    scratch; sizes needing more scratch raise SSMError (status SSM_ERR_WORKSPACE)."""
    bsz, L, Cc = xBC.shape
    H, P, G, N = nheads, headdim, ngroups, dstate
    if Cc != H * P + 2 * G * N:
        raise ValueError("xBC channel count must be nheads*headdim + 2*ngroups*dstate")
    K = conv_weight.shape[1]
    if y is None:
        raise ValueError("y is required: this call allocates nothing")
    _need(xBC, "xBC")
    _need(conv_weight, "conv_weight", torch.float32, (Cc, K))
    _need(conv_bias, "conv_bias", torch.float32, (Cc,))
    _need(conv_initial_state, "conv_initial_state", xBC.dtype, (bsz, Cc, K - 1))
    _need(dt, "dt", torch.float32, (bsz, L, H))
    _need(A, "A", torch.float32, (H,))
    _need(initial_state, "initial_state", torch.float32, (bsz, H, P, N))
    _need(seq_idx, "seq_idx", torch.int32, (bsz, L))
    _need(y, "y", xBC.dtype, (bsz, L, H, P))
    _need(conv_final_state, "conv_final_state", xBC.dtype, (bsz, Cc, K - 1))
    _need(final_state, "final_state", torch.float32, (bsz, H, P, N))
    _check("ssm_conv_scan_fwd_noalloc", _lib.ssm_conv_scan_fwd_noalloc(
        _ptr(xBC), _ptr(conv_weight), _ptr(conv_bias), _ptr(conv_initial_state),
        _ptr(conv_final_state), _ptr(dt), _ptr(A), _ptr(initial_state), _ptr(final_state),
        _ptr(seq_idx), _ptr(y), bsz, L, H, P, G, N, K, _dtype_code(xBC), ACT[activation],
        _stream()))
    return y, conv_final_state, final_state


def step(x, dt, A, B, C, state, state_indices=None, y=None, nheads=None, ngroups=None):
    """Decode update of a state pool.  x [b, n_new, H*P], B / C [b, n_new, G*N] -- any
    strides (e.g. channel ranges of the [b, C_conv, n_new] conv-update output, transposed);
    dt [b, n_new, H] fp32; state [n_slots, H, P, N] fp32 (updated in place);
    state_indices [b] int32.  Returns y [b, n_new, H, P]."""
    n_slots, H, P, N = state.shape
    bsz, n_new, HP = x.shape
    if B.dim() != 3 or B.shape[2] % N != 0:
        raise ValueError(f"B must be [b, n_new, G*N] with N = {N} (the state's last dimension)")
    G = B.shape[2] // N
    if HP != H * P or C.shape != B.shape or B.shape[:2] != x.shape[:2]:
        raise ValueError("x must be [b, n_new, H*P] and B, C [b, n_new, G*N]")
    if nheads is not None and nheads != H:
        raise ValueError(f"nheads {nheads} does not match the state's {H} heads")
    if ngroups is not None and ngroups != G:
        raise ValueError(f"ngroups {ngroups} does not match B's width {B.shape[2]} / N {N}")
    if H % G != 0:
        raise ValueError(f"nheads {H} must be a multiple of ngroups {G}")
    for t, name in ((x, "x"), (B, "B"), (C, "C")):
        _need(t, name, contiguous=False)
    _need(dt, "dt", torch.float32, (bsz, n_new, H))
    _need(A, "A", torch.float32, (H,))
    _need(state, "state", torch.float32)
    _need(state_indices, "state_indices", torch.int32, (bsz,))
    if DEBUG_CHECKS:
        check_distinct_slots(state_indices, n_slots, "state_indices")
    if y is None:
        y = torch.empty((bsz, n_new, H, P), dtype=x.dtype, device=x.device)
    _need(y, "y", x.dtype, (bsz, n_new, H, P))
    sx, sb, sc = x.stride(), B.stride(), C.stride()
    _check("ssm_step", _lib.ssm_step(
        _ptr(x), sx[0], sx[1], sx[2], _ptr(dt), _ptr(A), _ptr(B), sb[0], sb[1], sb[2], _ptr(C),
        sc[0], sc[1], sc[2], _ptr(state), _ptr(state_indices), _ptr(y), bsz, n_new, H, P, G, N,
        n_slots, _dtype_code(x), _stream()))
    return y


def decode_step(x_new, conv_state, conv_weight, conv_bias, dt, A, ssm_state, nheads, headdim,
                ngroups, dstate, conv_state_indices=None, cache_seqlens=None,
                state_indices=None, activation="silu", conv_out=None, y=None, norm=None):
    """One decode step on the pools (ssm_decode_step): the conv update over x_new
    [b, C_conv, n_new], then the SSM step reading the x | B | C channel ranges of its output.
    Both pools update in place; cache_seqlens is not advanced.  state_indices defaults to
    conv_state_indices.  Returns y [b, n_new, H, P], or with norm (a dict of norm_fwd's keyword
    arguments) y normed and gated over its H*P channels, [b, n_new, H*P]."""
    bsz, C, n_new = x_new.shape
    H, P, G, N = nheads, headdim, ngroups, dstate
    if C != H * P + 2 * G * N:
        raise ValueError("x_new channel count must be nheads*headdim + 2*ngroups*dstate")
    n_cslots, _, state_len = conv_state.shape
    K = conv_weight.shape[1]
    _need(x_new, "x_new")
    _need(conv_state, "conv_state", x_new.dtype, (n_cslots, C, state_len))
    _need(conv_weight, "conv_weight", torch.float32, (C, K))
    _need(conv_bias, "conv_bias", torch.float32, (C,))
    _need(dt, "dt", torch.float32, (bsz, n_new, H))
    _need(A, "A", torch.float32, (H,))
    if ssm_state.dim() != 4 or tuple(ssm_state.shape[1:]) != (H, P, N):
        raise ValueError(f"ssm_state must be [n_slots, {H}, {P}, {N}]")
    _need(ssm_state, "ssm_state", torch.float32)
    _need(conv_state_indices, "conv_state_indices", torch.int32, (bsz,))
    _need(cache_seqlens, "cache_seqlens", torch.int32, (bsz,))
    _need(state_indices, "state_indices", torch.int32, (bsz,))
    if DEBUG_CHECKS:
        check_distinct_slots(conv_state_indices, n_cslots, "conv_state_indices")
        check_distinct_slots(state_indices if state_indices is not None else conv_state_indices,
                             ssm_state.shape[0], "state_indices")
    if conv_out is None:
        conv_out = torch.empty_like(x_new)
    _need(conv_out, "conv_out", x_new.dtype, (bsz, C, n_new))
    if y is None:
        y = torch.empty((bsz, n_new, H, P), dtype=x_new.dtype, device=x_new.device)
    _need(y, "y", x_new.dtype, (bsz, n_new, H, P))
    normed = None if norm is None else _norm_plan(y.view(bsz, n_new, H * P), **norm)[1]
    with _on(x_new.device):  # the norm reads y on the same stream
        _check("ssm_decode_step", _lib.ssm_decode_step(
            _ptr(x_new), _ptr(conv_state), _ptr(conv_weight), _ptr(conv_bias),
            _ptr(conv_state_indices), _ptr(cache_seqlens), _ptr(dt), _ptr(A), _ptr(ssm_state),
            _ptr(state_indices), _ptr(conv_out), _ptr(y), bsz, n_new, H, P, G, N, K, state_len,
            n_cslots, ssm_state.shape[0], _dtype_code(x_new), ACT[activation], _stream()))
        return y if normed is None else normed()


def scan_bwd_workspace_size(batch, seqlen, nheads, headdim, ngroups, dstate,
                            dtype=torch.bfloat16) -> int:
    code = SSM_BF16 if dtype == torch.bfloat16 else SSM_F32
    return int(_lib.ssm_scan_bwd_workspace_size(batch, seqlen, nheads, headdim, ngroups, dstate,
                                                code))


def scan_bwd(x, dt, A, B, C, dy, initial_state=None, dfinal_state=None, seq_idx=None, dx=None,
             ddt=None, dA=None, dB=None, dC=None, dinitial_state=None, workspace=None):
    """The complete backward of scan_fwd (length-generalization notes Sec. 2.1 Eq. (1), Sec. 2.5
    Eq. (4)) from dy [b, L, H, P] and dfinal_state [b, H, P, N] fp32 (None = zero); the other
    inputs as scan_fwd's.  Returns (dx [b, L, H, P], ddt [b, L, H] fp32, dA [H] fp32, dB, dC
    [b, L, G, N], dinitial_state [b, H, P, N] fp32)."""
    bsz, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    dev = x.device
    _need(x, "x")
    _need(dt, "dt", torch.float32, (bsz, L, H))
    _need(A, "A", torch.float32, (H,))
    _need(B, "B", x.dtype, (bsz, L, G, N))
    _need(C, "C", x.dtype, (bsz, L, G, N))
    _need(dy, "dy", x.dtype, (bsz, L, H, P))
    _need(initial_state, "initial_state", torch.float32, (bsz, H, P, N))
    _need(dfinal_state, "dfinal_state", torch.float32, (bsz, H, P, N))
    _need(seq_idx, "seq_idx", torch.int32, (bsz, L))
    if dx is None:
        dx = torch.empty_like(x)
    if ddt is None:
        ddt = torch.empty_like(dt)
    if dA is None:
        dA = torch.empty_like(A)
    if dB is None:
        dB = torch.empty_like(B)
    if dC is None:
        dC = torch.empty_like(C)
    if dinitial_state is None:
        dinitial_state = torch.empty((bsz, H, P, N), dtype=torch.float32, device=dev)
    _need(dx, "dx", x.dtype, (bsz, L, H, P))
    _need(ddt, "ddt", torch.float32, (bsz, L, H))
    _need(dA, "dA", torch.float32, (H,))
    _need(dB, "dB", x.dtype, (bsz, L, G, N))
    _need(dC, "dC", x.dtype, (bsz, L, G, N))
    _need(dinitial_state, "dinitial_state", torch.float32, (bsz, H, P, N))
    _need_device(x, dt=dt, A=A, B=B, C=C, dy=dy, initial_state=initial_state,
                 dfinal_state=dfinal_state, seq_idx=seq_idx, dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC,
                 dinitial_state=dinitial_state, workspace=workspace)
    ws, wsb = _workspace(workspace, scan_bwd_workspace_size(bsz, L, H, P, G, N, x.dtype), dev)
    with _on(dev):
        _check("ssm_scan_bwd", _lib.ssm_scan_bwd(
            _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(dy), _ptr(initial_state),
            _ptr(dfinal_state), _ptr(seq_idx), _ptr(dx), _ptr(ddt), _ptr(dA), _ptr(dB), _ptr(dC),
            _ptr(dinitial_state), bsz, L, H, P, G, N, _dtype_code(x), _ptr(ws), wsb, _stream()))
    return dx, ddt, dA, dB, dC, dinitial_state


GATE = {"log": 0, "sigmoid": 1}


def _gated_args(x, gate, form):
    """Checks shared by the gated scans; returns (batch, tokens, channels, x_row, gate_row)."""
    if form not in GATE:
        raise ValueError(f"form must be one of {sorted(GATE)}, got {form!r}")
    if x.dim() != 3:
        raise ValueError(f"x must be [batch, tokens, channels], got shape {tuple(x.shape)}")
    B, L, C = x.shape
    if C < 1:
        raise ValueError("x must have at least one channel")
    _need(x, "x", contiguous=False)
    _need(gate, "gate", x.dtype, x.shape, contiguous=False)
    _need_device(x, gate=gate)
    return B, L, C, _rows(x, "x", C)[1], _rows(gate, "gate", C)[1]


def gated_scan_fwd_workspace_size(batch, seqlen, channels) -> int:
    return int(_lib.ssm_gated_scan_fwd_workspace_size(batch, seqlen, channels))


def gated_scan_bwd_workspace_size(batch, seqlen, channels) -> int:
    return int(_lib.ssm_gated_scan_bwd_workspace_size(batch, seqlen, channels))


def gated_scan_fwd(x, gate, form="sigmoid", initial_state=None, seq_idx=None,
                   return_final_state=True, final_state=None, y=None, workspace=None):
    """The per-channel gated recurrence h_t = a_t h_{t-1} + i_t x_t (length-generalization notes
    Sec. 2.1 Eq. (1), a state of one value per channel): a = exp(gate), i = 1 (form "log"; exp of
    the gates' sum over any consecutive tokens finite in fp32) or a = sigmoid(gate), i = 1 - a
    (form "sigmoid").  x, gate [b, L, C] (consecutive channels,
    tokens at any one stride); initial_state [b, C] fp32 (may be the same tensor as
    final_state; y must not overlap an input); seq_idx [b, L] int32.  Returns (y [b, L, C],
    final_state or None)."""
    B, L, C, x_row, gate_row = _gated_args(x, gate, form)
    _need(initial_state, "initial_state", torch.float32, (B, C))
    _need(seq_idx, "seq_idx", torch.int32, (B, L))
    if y is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
    _need(y, "y", x.dtype, x.shape, contiguous=False)
    if final_state is None and return_final_state:
        final_state = torch.empty((B, C), dtype=torch.float32, device=x.device)
    _need(final_state, "final_state", torch.float32, (B, C))
    _need_device(x, initial_state=initial_state, seq_idx=seq_idx, y=y, final_state=final_state,
                 workspace=workspace)
    ws, wsb = _workspace(workspace, gated_scan_fwd_workspace_size(B, L, C), x.device)
    with _on(x.device):
        _check("ssm_gated_scan_fwd", _lib.ssm_gated_scan_fwd(
            _ptr(x), x_row, _ptr(gate), gate_row, _ptr(initial_state), _ptr(final_state),
            _ptr(seq_idx), _ptr(y), _rows(y, "y", C)[1], B, L, C, GATE[form], _dtype_code(x),
            _ptr(ws), wsb, _stream()))
    return y, final_state


def gated_scan_bwd(x, gate, dy, form="sigmoid", initial_state=None, dfinal_state=None,
                   seq_idx=None, dx=None, dgate=None, dinitial_state=None, workspace=None):
    """Backward of gated_scan_fwd from dy [b, L, C] and dfinal_state [b, C] fp32 (None = zero).
    Returns (dx, dgate [b, L, C], dinitial_state [b, C] fp32)."""
    B, L, C, x_row, gate_row = _gated_args(x, gate, form)
    _need(dy, "dy", x.dtype, x.shape, contiguous=False)
    _need(initial_state, "initial_state", torch.float32, (B, C))
    _need(dfinal_state, "dfinal_state", torch.float32, (B, C))
    _need(seq_idx, "seq_idx", torch.int32, (B, L))
    if dx is None:
        dx = torch.empty_like(x, memory_format=torch.contiguous_format)
    if dgate is None:
        dgate = torch.empty_like(x, memory_format=torch.contiguous_format)
    if dinitial_state is None:
        dinitial_state = torch.empty((B, C), dtype=torch.float32, device=x.device)
    _need(dx, "dx", x.dtype, x.shape, contiguous=False)
    _need(dgate, "dgate", x.dtype, x.shape, contiguous=False)
    _need(dinitial_state, "dinitial_state", torch.float32, (B, C))
    _need_device(x, dy=dy, initial_state=initial_state, dfinal_state=dfinal_state, seq_idx=seq_idx,
                 dx=dx, dgate=dgate, dinitial_state=dinitial_state, workspace=workspace)
    ws, wsb = _workspace(workspace, gated_scan_bwd_workspace_size(B, L, C), x.device)
    with _on(x.device):
        _check("ssm_gated_scan_bwd", _lib.ssm_gated_scan_bwd(
            _ptr(x), x_row, _ptr(gate), gate_row, _ptr(dy), _rows(dy, "dy", C)[1],
            _ptr(initial_state), _ptr(dfinal_state), _ptr(seq_idx), _ptr(dx),
            _rows(dx, "dx", C)[1], _ptr(dgate), _rows(dgate, "dgate", C)[1],
            _ptr(dinitial_state), B, L, C, GATE[form], _dtype_code(x), _ptr(ws), wsb, _stream()))
    return dx, dgate, dinitial_state


def gated_scan_step(x, gate, state, form="sigmoid", state_indices=None, y=None):
    """Decode update of a pool of gated_scan states: x, gate [b, n_new, C], state [n_slots, C]
    fp32 (updated in place), state_indices [b] int32 (None: row b uses slot b).  Returns y
    [b, n_new, C]."""
    B, T, C, x_row, gate_row = _gated_args(x, gate, form)
    if state.dim() != 2 or state.shape[1] != C:
        raise ValueError(f"state must be [n_slots, {C}], got shape {tuple(state.shape)}")
    _need(state, "state", torch.float32)
    _need(state_indices, "state_indices", torch.int32, (B,))
    if DEBUG_CHECKS:
        check_distinct_slots(state_indices, state.shape[0], "state_indices")
    if y is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
    _need(y, "y", x.dtype, x.shape, contiguous=False)
    _need_device(x, state=state, state_indices=state_indices, y=y)
    with _on(x.device):
        _check("ssm_gated_scan_step", _lib.ssm_gated_scan_step(
            _ptr(x), x_row, _ptr(gate), gate_row, _ptr(state), _ptr(state_indices), _ptr(y),
            _rows(y, "y", C)[1], B, T, C, state.shape[0], GATE[form], _dtype_code(x), _stream()))
    return y


def _token_row(t, name):
    """Row stride of token tensor t [b, L, heads, dim]: a token's heads side by side, tokens at one
    stride."""
    b, L, heads, dim = t.shape
    if t.is_contiguous():
        return heads * dim
    if (dim > 1 and t.stride(3) != 1) or (heads > 1 and t.stride(2) != dim):
        raise ValueError(f"{name} must have a token's heads side by side")
    row = t.stride(1) if L > 1 else t.stride(0) if b > 1 else heads * dim
    if L > 1 and b > 1 and t.stride(0) != L * row:
        raise ValueError(f"{name} must have its tokens at one stride")
    return row


def _delta_args(q, k, v, beta, gate, scale):
    """Checks shared by the delta scans; returns (the leading arguments of the C calls, the sizes
    batch, seqlen, nheads, headdim, ngroups, dstate)."""
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if t.dim() != 4:
            raise ValueError(f"{name} must be [batch, tokens, heads, dim], got shape {tuple(t.shape)}")
    b, L, H, P = v.shape
    G, N = k.shape[2:]
    if H < 1 or P < 1 or G < 1 or N < 1 or H % G != 0:
        raise ValueError(f"v's {H} heads must be a positive multiple of k's {G}, and no dimension of a head 0")
    _need(v, "v", contiguous=False)
    _need(k, "k", v.dtype, (b, L, G, N), contiguous=False)
    _need(q, "q", v.dtype, (b, L, G, N), contiguous=False)
    _need(beta, "beta", torch.float32, (b, L, H))
    _need(gate, "gate", torch.float32, (b, L, H))
    _need_device(v, q=q, k=k, beta=beta, gate=gate)
    return ((_ptr(q), _token_row(q, "q"), _ptr(k), _token_row(k, "k"), _ptr(v), _token_row(v, "v"),
             _ptr(beta), _ptr(gate), scale), (b, L, H, P, G, N))


def delta_scan_fwd_workspace_size(batch, seqlen, nheads, headdim, ngroups, dstate,
                                  dtype=torch.bfloat16) -> int:
    code = SSM_BF16 if dtype == torch.bfloat16 else SSM_F32
    return int(_lib.ssm_delta_scan_fwd_workspace_size(batch, seqlen, nheads, headdim, ngroups, dstate,
                                                      code))


def delta_scan_bwd_workspace_size(batch, seqlen, nheads, headdim, ngroups, dstate,
                                  dtype=torch.bfloat16) -> int:
    code = SSM_BF16 if dtype == torch.bfloat16 else SSM_F32
    return int(_lib.ssm_delta_scan_bwd_workspace_size(batch, seqlen, nheads, headdim, ngroups, dstate,
                                                      code))


def delta_scan_fwd(q, k, v, beta, gate=None, scale=1.0, initial_state=None, seq_idx=None,
                   return_final_state=True, final_state=None, y=None, workspace=None):
    """The gated delta rule (length-generalization notes Sec. 2.1 Eq. (1) with the transition
    a_t (I - beta_t k_t k_t^T)): e_t = v_t - a_t h_{t-1} k_t, h_t = a_t h_{t-1} + beta_t e_t k_t^T,
    y_t = scale h_t q_t, a_t = exp(gate_t).  q, k [b, L, G, N], v [b, L, H, P] (a token's heads side
    by side, tokens at any one stride; H a multiple of G, N a multiple of 4 up to 256), beta, gate
    [b, L, H] fp32 (gate None: 1 for every a); initial_state [b, H, P, N] fp32 (may be the same
    tensor as final_state); seq_idx [b, L] int32.  Returns (y [b, L, H, P], final_state or None)."""
    lead, sizes = _delta_args(q, k, v, beta, gate, scale)
    b, L, H, P, G, N = sizes
    _need(initial_state, "initial_state", torch.float32, (b, H, P, N))
    _need(seq_idx, "seq_idx", torch.int32, (b, L))
    if y is None:
        y = torch.empty((b, L, H, P), dtype=v.dtype, device=v.device)
    _need(y, "y", v.dtype, (b, L, H, P), contiguous=False)
    if final_state is None and return_final_state:
        final_state = torch.empty((b, H, P, N), dtype=torch.float32, device=v.device)
    _need(final_state, "final_state", torch.float32, (b, H, P, N))
    _need_device(v, initial_state=initial_state, seq_idx=seq_idx, y=y, final_state=final_state,
                 workspace=workspace)
    ws, wsb = _workspace(workspace, delta_scan_fwd_workspace_size(*sizes, v.dtype), v.device)
    with _on(v.device):
        _check("ssm_delta_scan_fwd", _lib.ssm_delta_scan_fwd(
            *lead, _ptr(initial_state), _ptr(final_state), _ptr(seq_idx), _ptr(y),
            _token_row(y, "y"), *sizes, _dtype_code(v), _ptr(ws), wsb, _stream()))
    return y, final_state


def delta_scan_bwd(q, k, v, beta, dy, gate=None, scale=1.0, initial_state=None, dfinal_state=None,
                   seq_idx=None, dq=None, dk=None, dv=None, dbeta=None, dgate=None,
                   dinitial_state=None, workspace=None):
    """Backward of delta_scan_fwd from dy [b, L, H, P] and dfinal_state [b, H, P, N] fp32 (None =
    zero); the other inputs as delta_scan_fwd's.  Returns (dq, dk [b, L, G, N], dv [b, L, H, P],
    dbeta [b, L, H] fp32, dgate [b, L, H] fp32 or None without gate, dinitial_state
    [b, H, P, N] fp32)."""
    lead, sizes = _delta_args(q, k, v, beta, gate, scale)
    b, L, H, P, G, N = sizes
    dev = v.device
    _need(dy, "dy", v.dtype, (b, L, H, P), contiguous=False)
    _need(initial_state, "initial_state", torch.float32, (b, H, P, N))
    _need(dfinal_state, "dfinal_state", torch.float32, (b, H, P, N))
    _need(seq_idx, "seq_idx", torch.int32, (b, L))
    if gate is None and dgate is not None:
        raise ValueError("dgate given without gate")
    if dq is None:
        dq = torch.empty((b, L, G, N), dtype=v.dtype, device=dev)
    if dk is None:
        dk = torch.empty((b, L, G, N), dtype=v.dtype, device=dev)
    if dv is None:
        dv = torch.empty((b, L, H, P), dtype=v.dtype, device=dev)
    if dbeta is None:
        dbeta = torch.empty_like(beta)
    if dgate is None and gate is not None:
        dgate = torch.empty_like(gate)
    if dinitial_state is None:
        dinitial_state = torch.empty((b, H, P, N), dtype=torch.float32, device=dev)
    _need(dq, "dq", v.dtype, (b, L, G, N), contiguous=False)
    _need(dk, "dk", v.dtype, (b, L, G, N), contiguous=False)
    _need(dv, "dv", v.dtype, (b, L, H, P), contiguous=False)
    _need(dbeta, "dbeta", torch.float32, (b, L, H))
    _need(dgate, "dgate", torch.float32, (b, L, H))
    _need(dinitial_state, "dinitial_state", torch.float32, (b, H, P, N))
    _need_device(v, dy=dy, initial_state=initial_state, dfinal_state=dfinal_state, seq_idx=seq_idx,
                 dq=dq, dk=dk, dv=dv, dbeta=dbeta, dgate=dgate, dinitial_state=dinitial_state,
                 workspace=workspace)
    ws, wsb = _workspace(workspace, delta_scan_bwd_workspace_size(*sizes, v.dtype), dev)
    with _on(dev):
        _check("ssm_delta_scan_bwd", _lib.ssm_delta_scan_bwd(
            *lead, _ptr(dy), _token_row(dy, "dy"), _ptr(initial_state), _ptr(dfinal_state),
            _ptr(seq_idx), _ptr(dq), _token_row(dq, "dq"), _ptr(dk), _token_row(dk, "dk"), _ptr(dv),
            _token_row(dv, "dv"), _ptr(dbeta), _ptr(dgate), _ptr(dinitial_state), *sizes,
            _dtype_code(v), _ptr(ws), wsb, _stream()))
    return dq, dk, dv, dbeta, dgate, dinitial_state


def delta_scan_step(q, k, v, beta, state, gate=None, scale=1.0, state_indices=None, y=None):
    """Decode update of a pool of delta_scan states: q, k [b, n_new, G, N], v [b, n_new, H, P], beta,
    gate [b, n_new, H] fp32, state [n_slots, H, P, N] fp32 (updated in place), state_indices [b]
    int32 (None: row b uses slot b).  Returns y [b, n_new, H, P]."""
    lead, sizes = _delta_args(q, k, v, beta, gate, scale)
    b, T, H, P, G, N = sizes
    if state.dim() != 4 or tuple(state.shape[1:]) != (H, P, N):
        raise ValueError(f"state must be [n_slots, {H}, {P}, {N}], got shape {tuple(state.shape)}")
    _need(state, "state", torch.float32)
    _need(state_indices, "state_indices", torch.int32, (b,))
    if DEBUG_CHECKS:
        check_distinct_slots(state_indices, state.shape[0], "state_indices")
    if y is None:
        y = torch.empty((b, T, H, P), dtype=v.dtype, device=v.device)
    _need(y, "y", v.dtype, (b, T, H, P), contiguous=False)
    _need_device(v, state=state, state_indices=state_indices, y=y)
    with _on(v.device):
        _check("ssm_delta_scan_step", _lib.ssm_delta_scan_step(
            *lead, _ptr(state), _ptr(state_indices), _ptr(y), _token_row(y, "y"), *sizes,
            state.shape[0], _dtype_code(v), _stream()))
    return y


QK_NORM = {"l2": 0, "rms": 1}


def _qk_args(q, k, q_weight, k_weight, inv_freq, positions, kind):
    """Checks shared by qk_norm_fwd and qk_norm_bwd; returns (the leading arguments of the C calls,
    the sizes batch, seqlen, nheads_q, nheads_k, headdim, rotary_dim)."""
    if kind not in QK_NORM:
        raise ValueError(f"kind must be one of {sorted(QK_NORM)}, got {kind!r}")
    for t, name in ((q, "q"), (k, "k")):
        if t.dim() != 4:
            raise ValueError(f"{name} must be [batch, tokens, heads, dim], got shape {tuple(t.shape)}")
    b, L, HQ, D = q.shape
    HK = k.shape[2]
    if HQ < 1 or HK < 1 or D < 1:
        raise ValueError("q and k must have at least one head and channel")
    _need(q, "q", contiguous=False)
    _need(k, "k", q.dtype, (b, L, HK, D), contiguous=False)
    _need(q_weight, "q_weight", torch.float32, (D,))
    _need(k_weight, "k_weight", torch.float32, (D,))
    if inv_freq is not None and inv_freq.dim() != 1:
        raise ValueError("inv_freq must be [rotary_dim / 2]")
    R = 0 if inv_freq is None else 2 * inv_freq.shape[0]
    if R > D:
        raise ValueError(f"inv_freq has {R // 2} pairs for {D} channels")
    if positions is not None and inv_freq is None:
        raise ValueError("positions given without inv_freq")
    _need(inv_freq, "inv_freq", torch.float32)
    _need(positions, "positions", torch.int32, (b, L))
    _need_device(q, k=k, q_weight=q_weight, k_weight=k_weight, inv_freq=inv_freq, positions=positions)
    return ((_ptr(q), _token_row(q, "q"), _ptr(k), _token_row(k, "k"), _ptr(q_weight), _ptr(k_weight),
             _ptr(inv_freq), _ptr(positions)), (b, L, HQ, HK, D, R))


def qk_norm_fwd(q, k, q_weight=None, k_weight=None, eps=1e-6, kind="l2", inv_freq=None,
                positions=None, interleaved=False, q_out=None, k_out=None):
    """Norm of every head of q [b, L, HQ, D] and k [b, L, HK, D] (a token's heads side by side, tokens
    at any one stride; D up to 256): x / sqrt(sum x^2 + eps) (kind "l2") or x / sqrt(mean x^2 + eps)
    ("rms"), times q_weight / k_weight [D] fp32; with inv_freq [R/2] fp32 the first R channels are
    turned in pairs (i, i + R/2), or (2i, 2i + 1) if interleaved, by positions * inv_freq[i]
    (positions [b, L] int32, None: token t of every row is at t).  q_out may be q, k_out may be k.
    Returns (q_out, k_out)."""
    lead, sizes = _qk_args(q, k, q_weight, k_weight, inv_freq, positions, kind)
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if k_out is None:
        k_out = torch.empty(k.shape, dtype=q.dtype, device=q.device)
    _need(q_out, "q_out", q.dtype, q.shape, contiguous=False)
    _need(k_out, "k_out", q.dtype, k.shape, contiguous=False)
    _need_device(q, q_out=q_out, k_out=k_out)
    with _on(q.device):
        _check("ssm_qk_norm_fwd", _lib.ssm_qk_norm_fwd(
            *lead, _ptr(q_out), _token_row(q_out, "q_out"), _ptr(k_out), _token_row(k_out, "k_out"),
            *sizes, int(interleaved), eps, QK_NORM[kind], _dtype_code(q), _stream()))
    return q_out, k_out


def qk_norm_bwd_workspace_size(batch, seqlen, headdim) -> int:
    return int(_lib.ssm_qk_norm_bwd_workspace_size(batch, seqlen, headdim))


def qk_norm_bwd(q, k, dq_out, dk_out, q_weight=None, k_weight=None, eps=1e-6, kind="l2",
                inv_freq=None, positions=None, interleaved=False, dq=None, dk=None, dq_weight=None,
                dk_weight=None, workspace=None):
    """Backward of qk_norm_fwd from dq_out [b, L, HQ, D] and dk_out [b, L, HK, D]: the statistics are
    recomputed from q and k.  dq may be dq_out, dk may be dk_out.  Returns (dq, dk, dq_weight [D] fp32
    or None without q_weight, dk_weight likewise)."""
    lead, sizes = _qk_args(q, k, q_weight, k_weight, inv_freq, positions, kind)
    D = q.shape[3]
    _need(dq_out, "dq_out", q.dtype, q.shape, contiguous=False)
    _need(dk_out, "dk_out", q.dtype, k.shape, contiguous=False)
    if dq is None:
        dq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if dk is None:
        dk = torch.empty(k.shape, dtype=q.dtype, device=q.device)
    for w, dw, name in ((q_weight, dq_weight, "q"), (k_weight, dk_weight, "k")):
        if w is None and dw is not None:
            raise ValueError(f"d{name}_weight given without {name}_weight")
    if q_weight is not None and dq_weight is None:
        dq_weight = torch.empty(D, dtype=torch.float32, device=q.device)
    if k_weight is not None and dk_weight is None:
        dk_weight = torch.empty(D, dtype=torch.float32, device=q.device)
    _need(dq, "dq", q.dtype, q.shape, contiguous=False)
    _need(dk, "dk", q.dtype, k.shape, contiguous=False)
    _need(dq_weight, "dq_weight", torch.float32, (D,))
    _need(dk_weight, "dk_weight", torch.float32, (D,))
    _need_device(q, dq_out=dq_out, dk_out=dk_out, dq=dq, dk=dk, dq_weight=dq_weight, dk_weight=dk_weight,
                 workspace=workspace)
    need = 0
    if dq_weight is not None or dk_weight is not None:
        need = qk_norm_bwd_workspace_size(*q.shape[:2], D)
    ws, wsb = _workspace(workspace, need, q.device)
    with _on(q.device):
        _check("ssm_qk_norm_bwd", _lib.ssm_qk_norm_bwd(
            *lead, _ptr(dq_out), _token_row(dq_out, "dq_out"), _ptr(dk_out),
            _token_row(dk_out, "dk_out"), _ptr(dq), _token_row(dq, "dq"), _ptr(dk),
            _token_row(dk, "dk"), _ptr(dq_weight), _ptr(dk_weight), _ptr(ws), wsb, *sizes,
            int(interleaved), eps, QK_NORM[kind], _dtype_code(q), _stream()))
    return dq, dk, dq_weight, dk_weight


NORM = {"rms": 0, "layer": 1}


def _norm_args(x, weight, bias, z, kind, ngroups):
    """Checks shared by norm_fwd and norm_bwd; returns (channels, rows, x_row, z_row)."""
    if kind not in NORM:
        raise ValueError(f"kind must be one of {sorted(NORM)}, got {kind!r}")
    if x.dim() < 1:
        raise ValueError("x must be [..., channels]")
    C = x.shape[-1]
    if ngroups < 1 or C < 1 or C % ngroups != 0:
        raise ValueError(f"channels {C} must be a positive multiple of ngroups {ngroups}")
    _need(x, "x", contiguous=False)
    _need(weight, "weight", torch.float32, (C,))
    _need(bias, "bias", torch.float32, (C,))
    _need(z, "z", x.dtype, x.shape, contiguous=False)
    rows, x_row = _rows(x, "x", C)
    return C, rows, x_row, 0 if z is None else _rows(z, "z", C)[1]


def _norm_limits(channels, ngroups, eps, rows, out_row):
    """What ssm_norm_fwd itself refuses, refused before the call: a norm that follows a step on
    state pools must not fail after the step has moved them."""
    def refuse(status, detail):
        raise SSMError("ssm_norm_fwd", status, detail)
    if not ctypes.c_float(eps).value >= 0.0:
        refuse(1, "eps must be >= 0")
    if channels // operator.index(ngroups) > 16384:
        refuse(2, "channels / ngroups must be <= 16384")
    if ngroups > 0x7FFFFFFF or channels > 1 << 36:
        refuse(2, "too many channels")
    if rows > 1 and out_row < channels:
        refuse(1, f"out row stride below {channels}")


def _norm_plan(x, weight=None, bias=None, z=None, eps=1e-5, kind="rms", ngroups=1,
               norm_before_gate=False, out=None):
    """norm_fwd checked and its output allocated, not run: (out, the call)."""
    C, rows, x_row, z_row = _norm_args(x, weight, bias, z, kind, ngroups)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    _need(out, "out", x.dtype, x.shape, contiguous=False)
    _need_device(x, weight=weight, bias=bias, z=z, out=out)
    out_row = _rows(out, "out", C)[1]
    _norm_limits(C, ngroups, eps, rows, out_row)
    args = (_ptr(x), x_row, _ptr(z), z_row, _ptr(weight), _ptr(bias), _ptr(out), out_row, rows, C,
            ngroups, eps, NORM[kind], int(norm_before_gate), _dtype_code(x))

    def run():
        with _on(x.device):
            _check("ssm_norm_fwd", _lib.ssm_norm_fwd(*args, _stream()))
        return out
    return out, run


def norm_fwd(x, weight=None, bias=None, z=None, eps=1e-5, kind="rms", ngroups=1,
             norm_before_gate=False, out=None):
    """RMS (kind "rms") or layer (kind "layer") norm of x [..., channels] over ngroups groups of
    channels, times weight [channels] fp32, plus bias; z [..., channels] gates with silu(z),
    before the norm or (norm_before_gate) after it.  x, z and out: consecutive channels, rows at
    any one stride.  Returns out [..., channels] (x's dtype)."""
    return _norm_plan(x, weight, bias, z, eps, kind, ngroups, norm_before_gate, out)[1]()


def norm_bwd_workspace_size(rows, channels, ngroups=1) -> int:
    return int(_lib.ssm_norm_bwd_workspace_size(rows, channels, ngroups))


def norm_bwd(x, weight, dout, bias=None, z=None, eps=1e-5, kind="rms", ngroups=1,
             norm_before_gate=False, dx=None, dz=None, dweight=None, dbias=None, workspace=None):
    """Backward of norm_fwd from dout [..., channels]: the statistics are recomputed from x and
    z.  Returns (dx, dz or None without z, dweight [channels] fp32, dbias [channels] fp32 or
    None without bias)."""
    C, rows, x_row, z_row = _norm_args(x, weight, bias, z, kind, ngroups)
    _need(dout, "dout", x.dtype, x.shape, contiguous=False)
    if dx is None:
        dx = torch.empty_like(x, memory_format=torch.contiguous_format)
    if z is None and dz is not None:
        raise ValueError("dz given without z")
    if z is not None and dz is None:
        dz = torch.empty_like(x, memory_format=torch.contiguous_format)
    if dweight is None:
        dweight = torch.empty(C, dtype=torch.float32, device=x.device)
    if bias is not None and dbias is None:
        dbias = torch.empty(C, dtype=torch.float32, device=x.device)
    _need(dx, "dx", x.dtype, x.shape, contiguous=False)
    _need(dz, "dz", x.dtype, x.shape, contiguous=False)
    _need(dweight, "dweight", torch.float32, (C,))
    _need(dbias, "dbias", torch.float32, (C,))
    _need_device(x, weight=weight, bias=bias, z=z, dout=dout, dx=dx, dz=dz, dweight=dweight, dbias=dbias, workspace=workspace)
    ws, wsb = _workspace(workspace, norm_bwd_workspace_size(rows, C, ngroups), x.device)
    with _on(x.device):
        _check("ssm_norm_bwd", _lib.ssm_norm_bwd(
            _ptr(x), x_row, _ptr(z), z_row, _ptr(dout), _rows(dout, "dout", C)[1], _ptr(weight),
            _ptr(bias), _ptr(dx), _rows(dx, "dx", C)[1], _ptr(dz),
            0 if dz is None else _rows(dz, "dz", C)[1], _ptr(dweight), _ptr(dbias), _ptr(ws), wsb,
            rows, C, ngroups, eps, NORM[kind], int(norm_before_gate), _dtype_code(x), _stream()))
    return dx, dz, dweight, dbias


def stream_copy(src, dst):
    """dst <- src (same number of bytes, no overlap) with the library's streaming copy: the
    bandwidth reference of the benchmark, not part of the method."""
    nb = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nb:
        raise ValueError("stream_copy: src and dst differ in size")
    _need(src, "src")
    _need(dst, "dst")
    _check("ssm_stream_copy", _lib.ssm_stream_copy(_ptr(src), _ptr(dst), nb, _stream()))
    return dst


def timing_enable(enable: bool = True):
    _check("ssm_timing_enable", _lib.ssm_timing_enable(1 if enable else 0))


def timing_read():
    """(summed main-kernel milliseconds, launches) since the last read."""
    ms = ctypes.c_double()
    n = ctypes.c_int64()
    _check("ssm_timing_read", _lib.ssm_timing_read(ctypes.byref(ms), ctypes.byref(n)))
    return ms.value, n.value
