"""MoE expert-MLP + Split-LoRA layer for NVIDIA B200 (sm_100a).

A thin ctypes binding over the C ABI in include/moelora.h (libmoelora.so, built
in-tree by `python -m mixture_experts_lora_b200.build`).  The functions below
carry the ABI's names and only marshal arguments: PyTorch provides device
memory and the current stream; every step of the layer runs in the library's
CUDA kernels.  There is no CPU or PyTorch fallback: if the library is missing
or was not built, every call raises.
"""
from __future__ import annotations

import bisect
import ctypes
import itertools
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoelora.so")

# status codes (include/moelora.h)
MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_CUDA = 4
MOE_ERR_DEVICE_INDEX = 5
MOE_ERR_TIMEOUT = 6
MOE_ERR_DEVICE_CHECK = 7

EXPORTED = (
    "moe_workspace_bytes", "moe_route_topk", "moe_permute", "moe_grouped_gemm_lora_fwd",
    "moe_grouped_gemm_lora_bwd", "moe_unpermute_combine", "moe_get_device_error",
    "moe_status_string", "moe_profile_enable", "moe_profile_select", "moe_profile_read",
    "moe_permute_noalloc", "moe_router_backward", "moe_grouped_gemm_full_bwd",
    "moe_check_permutation", "moe_selftest_bounded_wait", "moe_route_permute",
    "moe_balance_workspace_bytes", "moe_balance_loss", "moe_balance_loss_backward",
    "moe_adamw_step", "moe_lora_requests",
)


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {msg} (status {status})")
        self.status = status


class moe_dims_t(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("m", ctypes.c_int32), ("n", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("r", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class moe_adamw_tensor_t(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p),
                ("exp_avg_scale", ctypes.c_void_p), ("exp_avg_sq_scale", ctypes.c_void_p),
                ("size", ctypes.c_int64 * 3), ("param_stride", ctypes.c_int64 * 3),
                ("grad_stride", ctypes.c_int64 * 3)]


class moe_adamw_config_t(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("param_bf16", ctypes.c_int32), ("grad_bf16", ctypes.c_int32),
                ("has_master", ctypes.c_int32), ("state_bits", ctypes.c_int32)]


_lib_handle = None


def lib() -> ctypes.CDLL:
    """Load libmoelora.so (raises if it was not built)."""
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m mixture_experts_lora_b200.build`")
        h = ctypes.CDLL(LIB_PATH)
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        D = ctypes.POINTER(moe_dims_t)
        h.moe_workspace_bytes.argtypes = [D]
        h.moe_workspace_bytes.restype = SZ
        h.moe_route_topk.argtypes = [P, I64, I32, I32, P, P, P]
        h.moe_permute.argtypes = [P, I64, I32, I32, P, P, P, P, P, SZ, P]
        h.moe_permute_noalloc.argtypes = [P, I64, I32, I32, P, P, P, P, P]
        h.moe_route_permute.argtypes = [P, I64, I32, I32, P, P, P, P, P, P, P, SZ, P]
        h.moe_check_permutation.argtypes = [P, I64, I32, I32, P, P, P, P, P]
        h.moe_grouped_gemm_lora_fwd.argtypes = [D] + [P] * 16 + [SZ, P]
        h.moe_grouped_gemm_lora_bwd.argtypes = [D] + [P] * 21 + [SZ, P]
        h.moe_grouped_gemm_full_bwd.argtypes = [D] + [P] * 23 + [SZ, P]
        h.moe_unpermute_combine.argtypes = [P, P, P, I64, I32, I32, P, P]
        h.moe_router_backward.argtypes = [P, P, P, P, P, I64, I32, I32, I32, P, P]
        h.moe_selftest_bounded_wait.argtypes = [ctypes.c_uint64, P, P]
        h.moe_balance_workspace_bytes.argtypes = [I64, I32, I32]
        h.moe_balance_workspace_bytes.restype = SZ
        h.moe_balance_loss.argtypes = [P, P, I64, I32, I32, P, I32, P, P, P, P, P, SZ, P]
        h.moe_balance_loss_backward.argtypes = [P, P, P, P, I64, I32, I32, P, I32, P, P, I32, P]
        h.moe_adamw_step.argtypes = [ctypes.POINTER(moe_adamw_tensor_t), I32,
                                     ctypes.POINTER(moe_adamw_config_t), P, P, P, I32, P]
        h.moe_lora_requests.argtypes = [P, I64, P, P, I64, I32, P, P, P, I32, I32, I32, I32, P, I64, P]
        h.moe_get_device_error.argtypes = [P]
        h.moe_status_string.argtypes = [ctypes.c_int]
        h.moe_status_string.restype = ctypes.c_char_p
        h.moe_profile_enable.argtypes = [ctypes.c_int]
        h.moe_profile_enable.restype = None
        h.moe_profile_select.argtypes = [ctypes.c_char_p]
        h.moe_profile_read.argtypes = [ctypes.c_int, ctypes.c_char_p, ctypes.c_int,
                                       ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_double)]
        for name in EXPORTED:
            if name not in ("moe_workspace_bytes", "moe_status_string", "moe_profile_enable",
                            "moe_balance_workspace_bytes"):
                getattr(h, name).restype = ctypes.c_int
        _lib_handle = h
    return _lib_handle


def status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def debug_checks() -> bool:
    """True when the environment variable MOE_CHECK is set (and not "0"): every call
    then synchronises and reads the device error word, and every permutation is
    checked on the device (moe_check_permutation).  For eager debugging; calls made
    while a CUDA graph is being captured are not checked."""
    return os.environ.get("MOE_CHECK", "") not in ("", "0")


def _check(fn: str, status: int):
    if status != MOE_OK:
        raise MoEError(fn, status, status_string(status))
    if debug_checks() and not torch.cuda.is_current_stream_capturing():
        torch.cuda.synchronize()
        st = int(lib().moe_get_device_error(_stream()))
        if st != MOE_OK:
            raise MoEError(fn, st, status_string(st))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def make_dims(T, m, n, E, k, r, scale) -> moe_dims_t:
    return moe_dims_t(int(T), int(m), int(n), int(E), int(k), int(r), float(scale))


# ---------------------------------------------------------------- ABI calls
def moe_workspace_bytes(dims: moe_dims_t) -> int:
    return int(lib().moe_workspace_bytes(ctypes.byref(dims)))


def moe_route_topk(logits, k, topk_ids, topk_w, stream=None):
    T, E = logits.shape
    _check("moe_route_topk", lib().moe_route_topk(_ptr(logits), T, E, int(k), _ptr(topk_ids),
                                                  _ptr(topk_w), _stream(stream)))


def moe_permute(topk_ids, E, counts, offsets, sorted_pairs, pair_pos, ws, stream=None):
    T, k = topk_ids.shape
    _check("moe_permute", lib().moe_permute(_ptr(topk_ids), T, k, int(E), _ptr(counts),
                                            _ptr(offsets), _ptr(sorted_pairs), _ptr(pair_pos),
                                            _ptr(ws), ws.numel() * ws.element_size(),
                                            _stream(stream)))
    if debug_checks():
        moe_check_permutation(topk_ids, E, counts, offsets, sorted_pairs, pair_pos, stream)


def moe_route_permute(logits, k, topk_ids, topk_w, counts, offsets, sorted_pairs, pair_pos, ws,
                      stream=None):
    """moe_route_topk and moe_permute in one call (one cooperative launch)."""
    T, E = logits.shape
    _check("moe_route_permute", lib().moe_route_permute(
        _ptr(logits), T, E, int(k), _ptr(topk_ids), _ptr(topk_w), _ptr(counts), _ptr(offsets),
        _ptr(sorted_pairs), _ptr(pair_pos), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream)))
    if debug_checks():
        moe_check_permutation(topk_ids, E, counts, offsets, sorted_pairs, pair_pos, stream)


def moe_check_permutation(topk_ids, E, counts, offsets, sorted_pairs, pair_pos, stream=None):
    """Device check of every invariant moe_permute promises; a violation sets
    MOE_ERR_DEVICE_CHECK in the device error word (see moe_get_device_error)."""
    T, k = topk_ids.shape
    _check("moe_check_permutation", lib().moe_check_permutation(
        _ptr(topk_ids), T, k, int(E), _ptr(counts), _ptr(offsets), _ptr(sorted_pairs),
        _ptr(pair_pos), _stream(stream)))


def moe_permute_noalloc(topk_ids, E, counts, offsets, sorted_pairs, pair_pos, stream=None):
    """moe_permute without a workspace (scratch built into the library)."""
    T, k = topk_ids.shape
    _check("moe_permute_noalloc", lib().moe_permute_noalloc(
        _ptr(topk_ids), T, k, int(E), _ptr(counts), _ptr(offsets), _ptr(sorted_pairs),
        _ptr(pair_pos), _stream(stream)))
    if debug_checks():
        moe_check_permutation(topk_ids, E, counts, offsets, sorted_pairs, pair_pos, stream)


def moe_grouped_gemm_lora_fwd(dims, X, sorted_pairs, offsets, W_gu, W_d, A_gu, B_gu, A_d, B_d,
                              Y_sorted, save_Xs, save_GU, save_H, save_XA, save_HA, ws, stream=None):
    args = [X, sorted_pairs, offsets, W_gu, W_d, A_gu, B_gu, A_d, B_d, Y_sorted, save_Xs, save_GU,
            save_H, save_XA, save_HA, ws]
    _check("moe_grouped_gemm_lora_fwd", lib().moe_grouped_gemm_lora_fwd(
        ctypes.byref(dims), *[_ptr(a) for a in args], ws.numel() * ws.element_size(),
        _stream(stream)))


def moe_grouped_gemm_lora_bwd(dims, dY, topk_w, sorted_pairs, offsets, W_gu, W_d, A_gu, B_gu,
                              A_d, B_d, save_Xs, save_GU, save_H, save_XA, save_HA, dX_sorted, dA_gu,
                              dB_gu, dA_d, dB_d, ws, stream=None):
    args = [dY, topk_w, sorted_pairs, offsets, W_gu, W_d, A_gu, B_gu, A_d, B_d, save_Xs, save_GU,
            save_H, save_XA, save_HA, dX_sorted, dA_gu, dB_gu, dA_d, dB_d, ws]
    _check("moe_grouped_gemm_lora_bwd", lib().moe_grouped_gemm_lora_bwd(
        ctypes.byref(dims), *[_ptr(a) for a in args], ws.numel() * ws.element_size(),
        _stream(stream)))


def moe_grouped_gemm_full_bwd(dims, dY, topk_w, sorted_pairs, offsets, W_gu, W_d, A_gu, B_gu,
                              A_d, B_d, save_Xs, save_GU, save_H, save_XA, save_HA, dX_sorted, dW_gu,
                              dW_d, dA_gu=None, dB_gu=None, dA_d=None, dB_d=None, ws=None,
                              stream=None):
    """Backward with the expert-weight gradients dW_gu [E, m, 2n] and dW_d [E, n, m]
    (full fine-tuning); the adapter gradients are computed when all four are given."""
    if ws is None:
        raise ValueError("moe_grouped_gemm_full_bwd needs the workspace")
    args = [dY, topk_w, sorted_pairs, offsets, W_gu, W_d, A_gu, B_gu, A_d, B_d, save_Xs, save_GU,
            save_H, save_XA, save_HA, dX_sorted, dW_gu, dW_d, dA_gu, dB_gu, dA_d, dB_d, ws]
    _check("moe_grouped_gemm_full_bwd", lib().moe_grouped_gemm_full_bwd(
        ctypes.byref(dims), *[_ptr(a) for a in args], ws.numel() * ws.element_size(),
        _stream(stream)))


def moe_unpermute_combine(Y_sorted, topk_w, pair_pos, T, k, m, Y, stream=None):
    _check("moe_unpermute_combine", lib().moe_unpermute_combine(
        _ptr(Y_sorted), _ptr(topk_w), _ptr(pair_pos), int(T), int(k), int(m), _ptr(Y),
        _stream(stream)))


def moe_router_backward(dY, Y_sorted, topk_ids, topk_w, pair_pos, E: int, dlogits, stream=None):
    """dlogits [T, E] fp32: gradient into the router logits (see include/moelora.h)."""
    T, m = dY.shape
    k = topk_ids.shape[1]
    _check("moe_router_backward", lib().moe_router_backward(
        _ptr(dY), _ptr(Y_sorted), _ptr(topk_ids), _ptr(topk_w), _ptr(pair_pos), int(T), int(k),
        int(E), int(m), _ptr(dlogits), _stream(stream)))


def moe_selftest_bounded_wait(limit_ns: int, done, stream=None):
    """Run one bounded wait that nothing ends (see include/moelora.h); afterwards
    moe_get_device_error() reports MOE_ERR_TIMEOUT and done[0] == 1."""
    st = lib().moe_selftest_bounded_wait(int(limit_ns), _ptr(done), _stream(stream))
    if st != MOE_OK:
        raise MoEError("moe_selftest_bounded_wait", st, status_string(st))


def moe_get_device_error(stream=None) -> int:
    return int(lib().moe_get_device_error(_stream(stream)))


def moe_profile_enable(on: bool = True):
    lib().moe_profile_enable(1 if on else 0)


def moe_profile_select(kinds=None) -> int:
    """Trace only the named kernel kinds (a list or comma-separated string); None = all."""
    if kinds is not None and not isinstance(kinds, str):
        kinds = ",".join(kinds)
    n = lib().moe_profile_select(None if not kinds else kinds.encode())
    if n < 0:
        raise ValueError(f"unknown kernel kind in {kinds!r}")
    return n


def moe_profile_read() -> dict:
    """{kernel name: (launches, total ms)} since the last read (waits for the GPU)."""
    n, L = 32, 48
    names = ctypes.create_string_buffer(n * L)
    cnt = (ctypes.c_int * n)()
    ms = (ctypes.c_double * n)()
    w = lib().moe_profile_read(n, names, L, cnt, ms)
    return {names.raw[i * L:(i + 1) * L].split(b"\0", 1)[0].decode(): (cnt[i], ms[i])
            for i in range(w)}


# ---------------------------------------------------------------- balance loss
# (These calls run beside kernels of a few microseconds, so their checks are kept to a few
# attribute reads per tensor, and pointers go through ctypes as plain integers.)
_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32


def _need(name, t, dtype, shape, index):
    """A contiguous tensor of this type and shape on CUDA device `index`, or ValueError."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}, got "
                         f"{t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _index_of(name, t):
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be on a CUDA device")
    return index


def _launch(name, index, stream, *args):
    """Calls the library's function `name` with device `index` current and, as its last argument,
    `stream` or that device's current one."""
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == index:
        _check(name, getattr(lib(), name)(*args, raw))
    else:
        with torch.cuda.device(index):
            _check(name, getattr(lib(), name)(*args, raw))


def _addr(t):
    return None if t is None else t.data_ptr()


def _check_rows(logits, seq_offsets, token_mask, S):
    T, E = logits.shape
    index = _index_of("logits", logits)
    _need("logits", logits, _F32, (T, E), index)
    if seq_offsets is not None:
        _need("seq_offsets", seq_offsets, _I32, (S + 1,), index)
    elif S != 1:
        raise ValueError("without seq_offsets there is one sequence")
    if token_mask is not None:
        if token_mask.dtype not in (torch.bool, torch.uint8):
            raise ValueError("token_mask must be bool or uint8")
        _need("token_mask", token_mask, token_mask.dtype, (T,), index)
    return T, E, index


def moe_balance_workspace_bytes(T: int, E: int, S: int = 1) -> int:
    return int(lib().moe_balance_workspace_bytes(int(T), int(E), int(S)))


def moe_balance_loss(logits, topk_ids, loss, counts, n_tokens, ws, seq_offsets=None, token_mask=None,
                     stream=None):
    """Balance loss [S] of the router for every sequence of a packed batch, with the pairs per
    expert counts [S, E] and the valid rows n_tokens [S] (see include/moelora.h)."""
    S = loss.shape[0]
    T, E, index = _check_rows(logits, seq_offsets, token_mask, S)
    k = topk_ids.shape[1]
    _need("topk_ids", topk_ids, _I32, (T, k), index)
    _need("loss", loss, _F32, (S,), index)
    _need("counts", counts, _I32, (S, E), index)
    _need("n_tokens", n_tokens, _I32, (S,), index)
    if ws.get_device() != index or not ws.is_contiguous():
        raise ValueError(f"the workspace must be a contiguous tensor on cuda:{index}")
    _launch("moe_balance_loss", index, stream, logits.data_ptr(), topk_ids.data_ptr(), T, E, k,
            _addr(seq_offsets), S, _addr(token_mask), loss.data_ptr(), counts.data_ptr(), n_tokens.data_ptr(),
            ws.data_ptr(), ws.nbytes)


def moe_balance_loss_backward(logits, counts, n_tokens, dloss, k, dlogits, seq_offsets=None,
                              token_mask=None, accumulate=False, stream=None):
    """Gradient of moe_balance_loss into the logits for the upstream gradient dloss [S], written
    to dlogits [T, E] or added to it."""
    S = dloss.shape[0]
    T, E, index = _check_rows(logits, seq_offsets, token_mask, S)
    _need("counts", counts, _I32, (S, E), index)
    _need("n_tokens", n_tokens, _I32, (S,), index)
    _need("dloss", dloss, _F32, (S,), index)
    _need("dlogits", dlogits, _F32, (T, E), index)
    _launch("moe_balance_loss_backward", index, stream, logits.data_ptr(), counts.data_ptr(), n_tokens.data_ptr(),
            dloss.data_ptr(), T, E, int(k), _addr(seq_offsets), S, _addr(token_mask), dlogits.data_ptr(),
            1 if accumulate else 0)


# ---------------------------------------------------------------- adapters of many requests
def moe_lora_requests(X, adapters, A, B, scale, Y, seq_offsets=None, stream=None):
    """Y[t] += scale[a] (X[t] A[a]) B[a] in place, a = adapters[request of row t] (negative: row
    left alone).  X [T, K] and Y [T, N] may be views with a row stride; seq_offsets [S + 1] gives
    the requests' rows, None one row per request (see include/moelora.h)."""
    T, K = X.shape
    n, _, r = A.shape
    N = Y.shape[1]
    S = adapters.shape[0]
    index = _index_of("X", X)
    sx, sy = X.stride(), Y.stride()
    if X.dtype is not _BF16 or sx[1] != 1:
        raise ValueError("X must be bfloat16 with unit stride inside its rows")
    if Y.dtype is not _BF16 or Y.shape[0] != T or sy[1] != 1 or Y.get_device() != index:
        raise ValueError(f"Y must be bfloat16 of {T} rows on cuda:{index} with unit stride inside its rows")
    _need("A", A, _BF16, (n, K, r), index)
    _need("B", B, _BF16, (n, r, N), index)
    _need("scale", scale, _F32, (n,), index)
    _need("adapters", adapters, _I32, (S,), index)
    if seq_offsets is not None:
        _need("seq_offsets", seq_offsets, _I32, (S + 1,), index)
    elif S != T:
        raise ValueError("without seq_offsets every row is a request: adapters must have one entry per row")
    # (the stride of a single row means nothing)
    ldx, ldy = (sx[0], sy[0]) if T > 1 else (K, N)
    _launch("moe_lora_requests", index, stream, X.data_ptr(), ldx, _addr(seq_offsets), adapters.data_ptr(), T, S,
            A.data_ptr(), B.data_ptr(), scale.data_ptr(), n, K, N, r, Y.data_ptr(), ldy)


# ---------------------------------------------------------------- AdamW
STATE_BLOCK = 256     # elements that share a scale in 8-bit states
LOOKED_AT = 16        # tensors whose addresses one step compares (50 ns each; a step's own host time is 5 us)
_data_ptr = torch.Tensor.data_ptr


def _joint_view(p, g):
    """Sizes and the two tensors' strides of a common view of at most three dimensions."""
    if p.is_contiguous() and g.is_contiguous():
        return [(1, 0, 0), (1, 0, 0), (p.numel(), 1, 1)]
    dims = [(n, sp, sg) for n, sp, sg in zip(p.shape, p.stride(), g.stride()) if n != 1]
    out = []
    for n, sp, sg in dims:
        if out and out[-1][1] == sp * n and out[-1][2] == sg * n:
            out[-1] = (out[-1][0] * n, sp, sg)
        else:
            out.append((n, sp, sg))
    if not out:
        out = [(1, 1, 1)]
    if len(out) > 3:
        raise ValueError(f"a tensor of shape {tuple(p.shape)} with strides {p.stride()} (gradient {g.stride()}) "
                         "does not fit a view of three dimensions")
    return [(1, 0, 0)] * (3 - len(out)) + out


def _need_apart(params):
    """ValueError where two parameters share an element's memory."""
    spans = []
    for i, p in enumerate(params):
        if p.numel():
            last = sum((n - 1) * st for n, st in zip(p.shape, p.stride()))
            spans.append((p.data_ptr(), p.data_ptr() + (last + 1) * p.element_size(), i))
    spans.sort()
    at = 0
    while at < len(spans):                # runs of spans that meet
        lo, hi, end = spans[at][0], spans[at][1], at + 1
        while end < len(spans) and spans[end][0] < hi:
            hi = max(hi, spans[end][1])
            end += 1
        run, at = [i for _, _, i in spans[at:end]], end
        if len(run) == 1:
            continue
        # interleaved views: their elements are marked one tensor after the other, in units of two bytes
        taken = None
        if not all(params[i].is_contiguous() for i in run):
            taken = torch.zeros((hi - lo) // 2, dtype=torch.bool, device=params[run[0]].device)
        for i in run:
            p = params[i]
            if taken is not None:
                u = p.element_size() // 2
                mine = taken.as_strided((*p.shape, u), (*(s * u for s in p.stride()), 1), (p.data_ptr() - lo) // 2)
                if not mine.any():
                    mine.fill_(True)
                    continue
            raise ValueError(f"parameter {i} shares memory with another one (of parameters {run})")


class AdamW:
    """AdamW over many tensors in one launch (moe_adamw_step), e.g. the adapters of all layers.

    params: bf16 or fp32 tensors, updated in place; grads: a gradient buffer for each (bf16 or
    fp32, the same shape), kept and read at every step().  Both may be strided views of up to
    three dimensions (SplitGateUpAdapters' views).  state_bits: 32 (fp32 moments) or 8 (e4m3
    codes of m and of sqrt(v) with an fp32 scale per 256 elements).  master_weights: an fp32
    copy of every bf16 parameter that the step updates and the parameter is rounded from; without
    it a change smaller than half a bf16 step of the weight is lost.  The copies are made at
    construction: after writing to the parameters (loading weights), call refresh_master(), or the next
    step puts the old weights back.

    lr may be set between steps, or be a device fp32 tensor that captured steps read.  The
    states live in flat tensors, each parameter's part beginning at a multiple of 256 elements
    (`starts`): exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale (8 bits), master.  steps is
    the number of steps taken, a device int64 that step() moves on, so that a captured step
    counts too.  Steps of one optimizer must be ordered on the device.

    The parameters and gradients must keep their memory, and their sizes and strides, while the
    optimizer is in use: steps, captured ones too, go to the addresses of its construction, whose
    storage it keeps alive.  step() raises ValueError, without a launch, when it sees a tensor that has
    been given other memory (`p.data = ...`, a module's cast or move); it looks at 16 of them, the next
    ones each time where there are more."""

    def __init__(self, params, grads, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
                 state_bits: int = 32, master_weights: bool = False):
        self.params, self.grads = list(params), list(grads)
        if len(self.params) != len(self.grads) or not self.params:
            raise ValueError("AdamW needs one gradient buffer for each of one or more parameters")
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        self.device = dev = self.params[0].device
        self.index = _index_of("parameters", self.params[0])
        self.lr, self.state_bits = lr, state_bits
        ok = (torch.bfloat16, torch.float32)
        groups, at = {}, 0
        self.starts, views = [], []
        for i, (p, g) in enumerate(zip(self.params, self.grads)):
            if p.dtype not in ok or g.dtype not in ok or p.shape != g.shape or p.device != dev or g.device != dev:
                raise ValueError(f"parameter {i}: bf16 or fp32 with a gradient of its shape on {dev} is needed")
            view = _joint_view(p, g)
            if not p.is_contiguous():
                reach = 1         # elements of the dimensions of smaller strides lie below this one's
                for n, sp, _ in sorted((v for v in view if v[0] > 1), key=lambda v: v[1]):
                    if sp < reach:
                        raise ValueError(f"parameter {i} has several elements in one place")
                    reach = sp * (n - 1) + reach
            if any(v[0] > 1 for v in view[:2]) and p.numel() >= 1 << 31:
                raise ValueError(f"parameter {i}: a strided view holds fewer than 2^31 elements")
            views.append(view)
            self.starts.append(at)
            at += -(-p.numel() // STATE_BLOCK) * STATE_BLOCK
            with_master = master_weights and p.dtype == torch.bfloat16
            groups.setdefault((p.dtype == torch.bfloat16, g.dtype == torch.bfloat16, with_master), []).append(i)
        _need_apart(self.params)
        if state_bits == 8:
            self.exp_avg = torch.zeros(at, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
            self.exp_avg_sq = torch.zeros(at, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
            self.exp_avg_scale = torch.zeros(at // STATE_BLOCK, dtype=torch.float32, device=dev)
            self.exp_avg_sq_scale = torch.zeros(at // STATE_BLOCK, dtype=torch.float32, device=dev)
        else:
            self.exp_avg = torch.zeros(at, dtype=torch.float32, device=dev)
            self.exp_avg_sq = torch.zeros(at, dtype=torch.float32, device=dev)
            self.exp_avg_scale = self.exp_avg_sq_scale = None
        self.master = None
        self._with_master = [i for g, idx in groups.items() if g[2] for i in idx]
        if self._with_master:
            self.master = torch.zeros(at, dtype=torch.float32, device=dev)
            self.refresh_master()
        tensors = self.params + self.grads
        self._held = [t.detach() for t in tensors]
        self._looks = [(ts, list(map(_data_ptr, ts)))
                       for ts in (tensors[i:i + LOOKED_AT] for i in range(0, len(tensors), LOOKED_AT))]
        self._next_look = itertools.cycle(self._looks).__next__
        self._by_address = sorted((p.data_ptr(), i) for i, p in enumerate(self.params) if p.numel())
        self._count = torch.zeros(2, dtype=torch.int64, device=dev)
        self._count_ptr = self._count.data_ptr()
        self.steps = self._count[0]
        elem = 1 if state_bits == 8 else 4
        self._calls = []
        for (p16, g16, master), idx in groups.items():
            table = (moe_adamw_tensor_t * len(idx))()
            for row, i in zip(table, idx):
                row.param, row.grad = self.params[i].data_ptr(), self.grads[i].data_ptr()
                row.exp_avg = self.exp_avg.data_ptr() + self.starts[i] * elem
                row.exp_avg_sq = self.exp_avg_sq.data_ptr() + self.starts[i] * elem
                if state_bits == 8:
                    row.exp_avg_scale = self.exp_avg_scale.data_ptr() + self.starts[i] // STATE_BLOCK * 4
                    row.exp_avg_sq_scale = self.exp_avg_sq_scale.data_ptr() + self.starts[i] // STATE_BLOCK * 4
                if master:
                    row.master = self.master.data_ptr() + self.starts[i] * 4
                for d, (n, sp, sg) in enumerate(views[i]):
                    row.size[d], row.param_stride[d], row.grad_stride[d] = n, sp, sg
            cfg = moe_adamw_config_t(0.0, betas[0], betas[1], eps, weight_decay, int(p16), int(g16), int(master),
                                     state_bits)
            self._calls.append((table, len(idx), cfg, ctypes.byref(cfg), int(len(self._calls) == len(groups) - 1)))

    def refresh_master(self):
        """Takes the master weights anew from the parameters, for weights written to them since."""
        for i in self._with_master:
            self._part(self.master, i).copy_(self.params[i])

    def _part(self, flat, i):
        p = self.params[i]
        return flat[self.starts[i]:self.starts[i] + p.numel()].view(p.shape)

    def step(self, grad_scale=None, stream=None):
        """One step with the gradients in the buffers, times grad_scale (a device fp32 tensor of
        one element) where given."""
        tensors, addresses = self._next_look()
        if list(map(_data_ptr, tensors)) != addresses:
            self._moved()
        lr, scale = self.lr, None
        lr_dev = None
        if isinstance(lr, torch.Tensor):
            self._scalar("lr", lr)
            lr, lr_dev = 0.0, lr.data_ptr()
        if grad_scale is not None:
            self._scalar("grad_scale", grad_scale)
            scale = grad_scale.data_ptr()
        for table, n, cfg, ref, last in self._calls:
            cfg.lr = lr
            _launch("moe_adamw_step", self.index, stream, table, n, ref, lr_dev, scale, self._count_ptr, last)

    def _check_gradients(self, pairs):
        """For pairs (weights, gradient of the same shape): ValueError unless this optimizer holds some of the
        weights, or views of them, each with the same place of the gradient as its buffer."""
        any_held = False
        for w, g in pairs:
            lo = w.data_ptr()
            for at, i in self._by_address[bisect.bisect_left(self._by_address, (lo, -1)):]:
                if at >= lo + w.nbytes:
                    break
                any_held = True
                if self.grads[i].data_ptr() != g.data_ptr() + (at - lo) // w.element_size() * g.element_size():
                    raise ValueError(f"the optimizer's gradient of parameter {i} is not the buffer that the layer's "
                                     "backward writes")
        if not any_held:
            raise ValueError("the optimizer holds none of the layer's adapters")

    def _moved(self):
        raise ValueError("a parameter or gradient has been given other memory since this optimizer was made: "
                         "make a new one over the tensors as they are now")

    def _scalar(self, name, t):
        if t.dtype is not _F32 or t.numel() != 1 or t.get_device() != self.index:
            raise ValueError(f"{name} must be a float32 tensor of one element on cuda:{self.index}")

    def moments(self, i: int):
        """(m, v) of parameter i as fp32 tensors of its shape (what the codes stand for in 8 bits)."""
        if self.state_bits == 32:
            return self._part(self.exp_avg, i), self._part(self.exp_avg_sq, i)
        a = self.starts[i]
        n = -(-self.params[i].numel() // STATE_BLOCK) * STATE_BLOCK
        out = []
        for codes, scales in ((self.exp_avg, self.exp_avg_scale), (self.exp_avg_sq, self.exp_avg_sq_scale)):
            x = codes[a:a + n].float().view(-1, STATE_BLOCK)
            x = x * scales[a // STATE_BLOCK:(a + n) // STATE_BLOCK, None]
            out.append(x.view(-1)[:self.params[i].numel()].view(self.params[i].shape))
        return out[0], out[1].square()

    _STATE = ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale", "master", "steps")

    def state_dict(self) -> dict:
        """The optimizer's own tensors (not copies), for checkpoints; None where it has none."""
        return {k: getattr(self, k) for k in self._STATE}

    def load_state_dict(self, state: dict):
        """Copies a state_dict() of an optimizer over the same parameters and settings, the master weights
        with it; the parameters themselves are loaded apart from it."""
        if any(list(map(_data_ptr, tensors)) != addresses for tensors, addresses in self._looks):
            self._moved()
        for k in self._STATE:
            mine, other = getattr(self, k), state[k]
            if (mine is None) != (other is None) or (mine is not None and (mine.shape != other.shape
                                                                          or mine.dtype != other.dtype)):
                raise ValueError(f"{k} does not fit this optimizer")
        for k in self._STATE:
            if getattr(self, k) is not None:
                getattr(self, k).copy_(state[k])


# ---------------------------------------------------------------- whole layer
@dataclass
class LayerBuffers:
    """Device buffers of one layer step (allocated once with PyTorch, reused)."""
    ids: torch.Tensor
    w: torch.Tensor
    counts: torch.Tensor
    offsets: torch.Tensor
    sorted_pairs: torch.Tensor
    pair_pos: torch.Tensor
    Y_sorted: torch.Tensor
    save_Xs: torch.Tensor
    save_GU: torch.Tensor
    save_H: torch.Tensor
    save_XA: torch.Tensor
    save_HA: torch.Tensor
    Y: torch.Tensor
    dX_sorted: torch.Tensor
    dX: torch.Tensor
    dA_gu: torch.Tensor
    dB_gu: torch.Tensor
    dA_d: torch.Tensor
    dB_d: torch.Tensor
    ws: torch.Tensor


def alloc_buffers(T, m, n, E, k, r, scale, device="cuda") -> LayerBuffers:
    P = T * k
    bf = dict(dtype=torch.bfloat16, device=device)
    i32 = dict(dtype=torch.int32, device=device)
    wsb = moe_workspace_bytes(make_dims(T, m, n, E, k, r, scale))
    if wsb == 0:
        raise MoEError("moe_workspace_bytes", MOE_ERR_UNSUPPORTED, "unsupported shape")
    return LayerBuffers(
        ids=torch.empty(T, k, **i32), w=torch.empty(T, k, dtype=torch.float32, device=device),
        counts=torch.empty(E, **i32), offsets=torch.empty(E + 1, **i32),
        sorted_pairs=torch.empty(P, **i32), pair_pos=torch.empty(P, **i32),
        Y_sorted=torch.empty(P, m, **bf), save_Xs=torch.empty(P, m, **bf),
        save_GU=torch.empty(P, 2 * n, **bf),
        save_H=torch.empty(P, n, **bf), save_XA=torch.empty(P, r, **bf),
        save_HA=torch.empty(P, r, **bf), Y=torch.empty(T, m, **bf),
        dX_sorted=torch.empty(P, m, **bf), dX=torch.empty(T, m, **bf),
        dA_gu=torch.empty(E, m, r, **bf), dB_gu=torch.empty(E, r, 2 * n, **bf),
        dA_d=torch.empty(E, n, r, **bf), dB_d=torch.empty(E, r, m, **bf),
        ws=torch.empty(wsb, dtype=torch.uint8, device=device))


def layer_forward(inp: dict, k: int, scale: float, buf: LayerBuffers, stream=None):
    """route -> permute -> grouped GEMMs -> combine; fills buf.Y (and the saves)."""
    T, m = inp["X"].shape
    E, _, n2 = inp["W_gu"].shape
    r = inp["A_gu"].shape[2]
    dims = make_dims(T, m, n2 // 2, E, k, r, scale)
    moe_route_permute(inp["logits"], k, buf.ids, buf.w, buf.counts, buf.offsets, buf.sorted_pairs,
                      buf.pair_pos, buf.ws, stream)
    moe_grouped_gemm_lora_fwd(dims, inp["X"], buf.sorted_pairs, buf.offsets, inp["W_gu"],
                              inp["W_d"], inp["A_gu"], inp["B_gu"], inp["A_d"], inp["B_d"],
                              buf.Y_sorted, buf.save_Xs, buf.save_GU, buf.save_H, buf.save_XA,
                              buf.save_HA, buf.ws, stream)
    moe_unpermute_combine(buf.Y_sorted, buf.w, buf.pair_pos, T, k, m, buf.Y, stream)
    return buf.Y


def layer_backward(inp: dict, dY, k: int, scale: float, buf: LayerBuffers, stream=None):
    """grouped GEMM backward -> unweighted combine; fills buf.dX and the adapter grads."""
    T, m = inp["X"].shape
    E, _, n2 = inp["W_gu"].shape
    r = inp["A_gu"].shape[2]
    dims = make_dims(T, m, n2 // 2, E, k, r, scale)
    moe_grouped_gemm_lora_bwd(dims, dY, buf.w, buf.sorted_pairs, buf.offsets,
                              inp["W_gu"], inp["W_d"], inp["A_gu"], inp["B_gu"], inp["A_d"],
                              inp["B_d"], buf.save_Xs, buf.save_GU, buf.save_H, buf.save_XA,
                              buf.save_HA,
                              buf.dX_sorted, buf.dA_gu, buf.dB_gu, buf.dA_d, buf.dB_d, buf.ws,
                              stream)
    moe_unpermute_combine(buf.dX_sorted, None, buf.pair_pos, T, k, m, buf.dX, stream)
    return buf.dX


def layer_backward_full(inp: dict, dY, k: int, scale: float, buf: LayerBuffers, dW_gu, dW_d,
                        adapters: bool = True, stream=None):
    """layer_backward plus the expert-weight gradients (full fine-tuning) into dW_gu
    [E, m, 2n] and dW_d [E, n, m]; adapters=False skips the adapter gradients."""
    T, m = inp["X"].shape
    E, _, n2 = inp["W_gu"].shape
    r = inp["A_gu"].shape[2]
    dims = make_dims(T, m, n2 // 2, E, k, r, scale)
    lora = (buf.dA_gu, buf.dB_gu, buf.dA_d, buf.dB_d) if adapters else (None,) * 4
    moe_grouped_gemm_full_bwd(dims, dY, buf.w, buf.sorted_pairs, buf.offsets,
                              inp["W_gu"], inp["W_d"], inp["A_gu"], inp["B_gu"], inp["A_d"],
                              inp["B_d"], buf.save_Xs, buf.save_GU, buf.save_H, buf.save_XA,
                              buf.save_HA,
                              buf.dX_sorted, dW_gu, dW_d, *lora, ws=buf.ws, stream=stream)
    moe_unpermute_combine(buf.dX_sorted, None, buf.pair_pos, T, k, m, buf.dX, stream)
    return buf.dX


def layer_step(inp: dict, k: int, scale: float, buf: LayerBuffers, stream=None):
    """One pass of the whole hot path: forward then backward against inp['dY']."""
    layer_forward(inp, k, scale, buf, stream)
    layer_backward(inp, inp["dY"], k, scale, buf, stream)
    return buf


@dataclass
class BalanceBuffers:
    """Device buffers of the balance loss in a training step: the loss and its upstream gradient
    per sequence, the counts, and the gradient into the router logits."""
    loss: torch.Tensor
    dloss: torch.Tensor
    counts: torch.Tensor
    n_tokens: torch.Tensor
    dlogits: torch.Tensor
    ws: torch.Tensor


def alloc_balance(T, E, S=1, weight=0.01, device="cuda") -> BalanceBuffers:
    """Buffers for S sequences; every sequence's loss gets the weight `weight` / S."""
    f32 = dict(dtype=torch.float32, device=device)
    i32 = dict(dtype=torch.int32, device=device)
    wsb = moe_balance_workspace_bytes(T, E, S)
    if wsb == 0:
        raise MoEError("moe_balance_workspace_bytes", MOE_ERR_UNSUPPORTED, "unsupported shape")
    return BalanceBuffers(loss=torch.empty(S, **f32), dloss=torch.full((S,), weight / S, **f32),
                          counts=torch.empty(S, E, **i32), n_tokens=torch.empty(S, **i32),
                          dlogits=torch.empty(T, E, **f32),
                          ws=torch.empty(wsb, dtype=torch.uint8, device=device))


def layer_train_step(inp: dict, k: int, scale: float, buf: LayerBuffers, opt: AdamW,
                     balance: BalanceBuffers | None = None, seq_offsets=None, token_mask=None, group=None,
                     grad_scale=None, stream=None):
    """One training step of the layer: forward, backward against inp['dY'], the adapter gradients
    summed over the data-parallel ranks, and the optimizer's step (opt holds the layer's adapters,
    or some of them or views, with buf's gradient buffers or the same views of those; it may hold
    other tensors too).  With `balance` the router's gradient comes too: balance.dlogits
    is that of the output through the routing weights plus that of the balance loss."""
    opt._check_gradients([(inp["A_gu"], buf.dA_gu), (inp["B_gu"], buf.dB_gu), (inp["A_d"], buf.dA_d),
                          (inp["B_d"], buf.dB_d)])
    layer_forward(inp, k, scale, buf, stream)
    if balance is not None:
        moe_balance_loss(inp["logits"], buf.ids, balance.loss, balance.counts, balance.n_tokens, balance.ws,
                         seq_offsets, token_mask, stream)
        moe_router_backward(inp["dY"], buf.Y_sorted, buf.ids, buf.w, buf.pair_pos, inp["logits"].shape[1],
                            balance.dlogits, stream)
        moe_balance_loss_backward(inp["logits"], balance.counts, balance.n_tokens, balance.dloss, k,
                                  balance.dlogits, seq_offsets, token_mask, True, stream)
    layer_backward(inp, inp["dY"], k, scale, buf, stream)
    from .dp import allreduce_adapter_grads
    with torch.cuda.stream(stream):       # (None: the current stream stays)
        allreduce_adapter_grads([buf.dA_gu, buf.dB_gu, buf.dA_d, buf.dB_d], group)
    opt.step(grad_scale, stream)
    return buf


def shared_expert_step(inp: dict, scale: float, buf: LayerBuffers, stream=None):
    """Shared expert: a dense SwiGLU MLP with LoRA applied to every token, whose output
    the caller adds to the routed experts' Y (and its dX to theirs).  It is this layer
    with one expert, k = 1 and routing weight 1: `inp` holds X, dY and the six weight
    tensors with a leading expert dimension of 1, plus logits [T, 1] (any values; the
    softmax over one picked logit is 1).  Outputs land in buf.Y, buf.dX and the
    adapter gradients like layer_step; `buf` comes from alloc_buffers(T, m, n, 1, 1, r, scale)."""
    if inp["W_gu"].shape[0] != 1 or inp["logits"].shape[1] != 1:
        raise ValueError("a shared expert has exactly one expert and logits of width 1")
    return layer_step(inp, 1, scale, buf, stream)


# ---------------------------------------------------------------- adapter variants
class SplitGateUpAdapters:
    """Separate gate and up adapters (rank r each) held in the library's fused layout.

    gate_up carries one adapter of rank 2r with A_gu = [A_g | A_u] and
    B_gu = [[B_g, 0], [0, B_u]]; the down adapter is zero-padded to the same rank
    (the library uses one rank for both projections).  The result is exactly the
    layer with separate adapters.  The attributes A_g, B_g, A_u, B_u, A_d, B_d are
    views into the packed tensors: write them, or let an optimizer update them, in
    place.  Nothing ever writes the off-diagonal blocks or the padding, so those
    stay zero.  Pass A_gu, B_gu, A_d_packed and B_d_packed to the layer with rank 2r
    and the scale of one adapter (alpha / r, or alpha / sqrt(r) for rsLoRA)."""

    def __init__(self, E: int, m: int, n: int, r: int, device="cuda"):
        if 2 * r > 128:
            raise ValueError("separate gate/up adapters need 2r <= 128")
        bf = dict(dtype=torch.bfloat16, device=device)
        self.r, self.n = r, n
        self.A_gu = torch.zeros(E, m, 2 * r, **bf)
        self.B_gu = torch.zeros(E, 2 * r, 2 * n, **bf)
        self.A_d_packed = torch.zeros(E, n, 2 * r, **bf)
        self.B_d_packed = torch.zeros(E, 2 * r, m, **bf)
        self.A_g, self.A_u = self.A_gu[:, :, :r], self.A_gu[:, :, r:]
        self.B_g, self.B_u = self.B_gu[:, :r, :n], self.B_gu[:, r:, n:]
        self.A_d, self.B_d = self.A_d_packed[:, :, :r], self.B_d_packed[:, :r, :]

    def layer_inputs(self, inp: dict) -> dict:
        """inp (X, logits, dY, W_gu, W_d) completed with the packed adapters."""
        out = dict(inp)
        out.update(A_gu=self.A_gu, B_gu=self.B_gu, A_d=self.A_d_packed, B_d=self.B_d_packed)
        return out

    def grads(self, buf: LayerBuffers) -> dict:
        """Views of the separate adapters' gradients in a rank-2r LayerBuffers."""
        r, n = self.r, self.n
        return {"dA_g": buf.dA_gu[:, :, :r], "dA_u": buf.dA_gu[:, :, r:],
                "dB_g": buf.dB_gu[:, :r, :n], "dB_u": buf.dB_gu[:, r:, n:],
                "dA_d": buf.dA_d[:, :, :r], "dB_d": buf.dB_d[:, :r, :]}
