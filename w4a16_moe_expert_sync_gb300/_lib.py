"""ctypes binding of libw4moe.so: the C entry points of include/w4moe.h under
the same names, taking torch tensors.  Argument marshalling only: shapes are
read from the tensors, outputs are allocated with torch (device memory), the
pointers and the current CUDA stream are passed through, and a nonzero status
raises W4Error.  (A step's calls of a few microseconds on the GPU go the same way in
C++: csrc/calls.cpp.)  Every step of the layer runs in the library's CUDA kernels;
there is no fallback of any kind.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import re
import threading

from .build import LIB as _LIB_PATH, calls_path

_lock = threading.Lock()
_lib = None
_torch = None


def _load_torch():
    """torch, for the calls where an import statement's half microsecond counts."""
    global _torch
    import torch
    _torch = torch
    return torch


HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "include", "w4moe.h")

# device status bits (include/w4moe.h)
W4_DEV_BAD_EXPERT_ID = 0x1
W4_DEV_PIPELINE_TIMEOUT = 0x2
W4_DEV_TOO_MANY_JOBS = 0x4
W4_DEV_FP16_RANGE = 0x8
W4_DEV_OUT_OF_BOUNDS = 0x10
W4_DEV_BAD_SLOT = 0x20
W4_DEV_BAD_PAGE = 0x40
W4_DEV_NO_PAGES = 0x80
# xg and h rows end in one block of 64 columns of activation group sums, the
# grouped GEMMs' input for the low parts of their dequantisation constants
SUM_COLS = 64


class W4Error(RuntimeError):
    def __init__(self, status: int, name: str, detail: str):
        super().__init__(f"{name} ({status}): {detail}")
        self.status = status
        self.name = name
        self.detail = detail


def header_functions() -> list[str]:
    """Names of the functions declared in include/w4moe.h."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[a-z_0-9]+\s*\*?\s*(w4_[a-z_0-9]+)\s*\(",
                                 text, flags=re.M)))


def load_library(path: str | None = None):
    """Load libw4moe.so (built by __graft_entry__.build()); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or _LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is missing: build the CUDA library first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(p)
        V, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        U64 = ctypes.c_uint64
        sig = {
            "w4_status_string": ([I], ctypes.c_char_p),
            "w4_last_error_detail": ([], ctypes.c_char_p),
            "w4_abi_version": ([], I),
            "w4_quantize": ([V, I, I, I, I, V, V, V, V], I),
            "w4_moe_route": ([V, I, I, I, V, V, V], I),
            "w4_moe_align_capacity": ([I, I, I, I], I64),
            "w4_moe_align": ([V, I, I, I, I, V, V, V, V, V, V], I),
            "w4_gather_activations": ([V, I, I, I, I, I, V, V, V, V, V], I),
            "w4_moe_align_gather": ([V, V, I, I, I, I, I, V, V, V, V, V, V, V], I),
            "w4_moe_route_align_gather": ([V, V, I, I, I, I, I, V, V, V, V, V, V, V, V, V],
                                          I),
            "w4_grouped_gemm_gate_up": ([V, I, I, I, I, I, I, V, V, V, I, V, V, V, V, V], I),
            "w4_grouped_gemm_down": ([V, I, I, I, I, I, I, V, V, V, I, V, V, V, V, V], I),
            "w4_moe_combine_fixed_order": ([V, V, V, I, I, I, I, V, V], I),
            "w4_grouped_gemm_down_combine": ([V, I, I, I, I, I, I, V, V, V, I, V, V, V, V, V, V,
                                              V, V, V], I),
            "w4_moe_combine_prepare": ([V, I, I, I, I, V, V, V], I),
            "w4_test_pipeline_hooks": ([U64, I], I),
            "w4_moe_layer_workspace_size": ([I, I, I, I, I, I], SZ),
            "w4_moe_layer": ([V, V, V, I, I, I, I, I, I, V, V, V, I, V, V, V, I, V, SZ, V, V,
                              V], I),
            "w4_moe_layer_host_workspace_size": ([I, I, I, I, I, I], SZ),
            "w4_moe_layer_host": ([V, V, V, I, I, I, I, I, I, V, V, V, I, V, V, V, I, V, SZ, V,
                                   V, V], I),
            "w4_moe_layer_static_scratch": ([V, V, V, I, I, I, I, I, I, V, V, V, I, V, V, V, I,
                                             V, V, V], I),
            "w4_moe_layer_from_logits": ([V, V, I, I, I, I, I, I, V, V, V, I, V, V, V, I, V,
                                          SZ, V, V, V, V, V], I),
            "w4_moe_layer_few_workspace_size": ([I, I, I, I, I], SZ),
            "w4_moe_layer_few": ([V, V, V, I, I, I, I, I, V, V, V, I, V, V, V, I, V, SZ, V, V, V],
                                 I),
            "w4_moe_layer_few_from_logits": ([V, V, I, I, I, I, I, V, V, V, I, V, V, V, I, V, SZ,
                                              V, V, V, V, V], I),
            "w4_w4a16_linear_workspace_size": ([I, I, I, I], SZ),
            "w4_w4a16_linear": ([V, I, I, I, V, V, V, I, V, SZ, V, V, V], I),
            "w4_w4a16_linear_few": ([V, I, I, I, V, V, V, I, V, V, V], I),
            "w4_kv_workspace_size": ([I, I], SZ),
            "w4_kv_reserve": ([V, I, I, V, V, I, V, V, I, I, V, V], I),
            "w4_kv_free": ([V, I, I, V, V, I, V, I, V, V], I),
            "w4_kv_fork": ([V, I, I64, V, I, I, V, V, I, V, V, I, I, V, SZ, V, V], I),
            "w4_kv_copy_pages": ([V, I, I64, I, V, V, I, V, V], I),
            "w4_kv_compact": ([V, I, I64, V, I, I, V, I, V, V, V, SZ, V, V], I),
            "w4_kv_append": ([V, V, I64, I64, I64, I, I, I, I, V, I, I, V, V, I64, I64, V, I64, I64,
                              V, I, V, V], I),
            "w4_kv_keep": ([V, I, I64, V, I, I, V, V, I, V, V, V, I, I, V, V, V], I),
            "w4_rope_steps": ([I, ctypes.c_double, I] + [ctypes.c_double] * 4 + [V], I),
            "w4_qk_norm_rope": ([V, I64, I64, V, I64, I64, V, V, V, V, I, I, I, I, I, I, I,
                                 ctypes.c_float, ctypes.c_float, V, I64, I64, V, I64, I64, V], I),
            "w4_kv_append_rope": ([V, V, I64, I64, I64, I, I, V, I, I, V, V, I64, I64, V, I64, I64,
                                   V, I64, I64, V, V, V, V, V, I, I, I, I, I, I, I, ctypes.c_float,
                                   ctypes.c_float, V, I64, I64, V, V], I),
            "w4_attn_shared_prefix_workspace_size": ([I, I, I, I, I, I, I], SZ),
            "w4_attn_shared_prefix": ([V, I64, I64, V, V, I64, I64, I64, I, I, V, I, V, V, I, I, I,
                                       V, V, I, I, I, I, I, I, ctypes.c_float, V, SZ, V, V, V], I),
            "w4_attn_tree": ([V, I64, I64, V, V, I64, I64, I64, I, I, V, I, V, V, I, I, I, V, I, V, V,
                              I, I, I, I, I, ctypes.c_float, V, SZ, V, V, V], I),
            "w4_rmsnorm": ([V, V, I, I, ctypes.c_float, V, V], I),
            "w4_sample_logits_workspace_size": ([I, I64], SZ),
            "w4_sample_logits": ([V, I, I64, U64, U64, V, V, V, V, SZ, V], I),
            "w4_fused_entropy": ([V, I, I64, V, V, SZ, V], I),
            "w4_gumbel_argmax_sample": ([V, I, I64, U64, U64, V, V, V, SZ, V], I),
        }
        for name, (args, res) in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
        return lib


_calls_module = None
_calls_file = None                         # the module's path, once asked for


def _calls_built() -> bool:
    """Whether the module has been built for this version of torch."""
    global _calls_file
    if _calls_file is None:
        _calls_file = calls_path()
    return os.path.exists(_calls_file)


def _calls():
    """The module that calls a step's entry points (csrc/calls.cpp), bound to the library."""
    global _calls_module
    lib = load_library()
    with _lock:
        if _calls_module is not None:
            return _calls_module
        import torch                       # its libraries are the module's too
        if not _calls_built():
            raise RuntimeError(f"{_calls_file} is missing: build the CUDA library for this version of "
                               "torch first (python -c 'import __graft_entry__ as g; g.build()')")
        path = _calls_file
        loader = importlib.machinery.ExtensionFileLoader("w4_calls", path)
        module = importlib.util.module_from_spec(
            importlib.machinery.ModuleSpec("w4_calls", loader, origin=path))
        loader.exec_module(module)
        functions = (ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in (
            "w4_w4a16_linear_few", "w4_qk_norm_rope", "w4_kv_append_rope", "w4_kv_keep",
            "w4_attn_shared_prefix", "w4_attn_tree", "w4_attn_shared_prefix_workspace_size"))
        module.bind(*functions, _check,
                    lambda t, shape, stream: _result(shape, t.dtype, t.device, stream),
                    lambda t, nbytes, stream: _scratch(nbytes, torch.uint8, t.device, stream))
        _calls_module = module
        return module


def _check(rc: int, what: str):
    if rc != 0:
        lib = load_library()
        raise W4Error(rc, lib.w4_status_string(rc).decode(),
                      f"{what}: {lib.w4_last_error_detail().decode()}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    torch = _torch or _load_torch()
    # the handle alone: building a Stream object costs several microseconds a call
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _scratch(shape, dtype, device, stream):
    """Memory that a call on `stream` needs until its kernels have run: of that
    stream's pool, so that nothing takes it before they have, once it is let go."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _result(shape, dtype, device, stream):
    """A tensor that a call on `stream` fills and returns: of that stream's pool, for
    earlier work of another stream may still use what that one's pool hands out, and
    held, once let go, until the current stream's work of then has run."""
    torch = _torch or _load_torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    t = _scratch(shape, dtype, device, stream)
    if t.numel():
        current = torch.cuda.current_stream(t.device)
        if current.cuda_stream != stream.cuda_stream:
            t.record_stream(current)
    return t


def _require_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("tensors passed to the CUDA library must live on the GPU")
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors passed to the CUDA library must be contiguous")


def _require(specs):
    """Every (tensor, type, shape, name) is a contiguous CUDA tensor like that."""
    for t, dtype, shape, name in specs:
        if not t.is_cuda:
            raise ValueError("tensors passed to the CUDA library must live on the GPU")
        if not t.is_contiguous():
            raise ValueError("tensors passed to the CUDA library must be contiguous")
        if t.dtype is not dtype or t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)} {dtype}, not {list(t.shape)} {t.dtype}")


# --------------------------------------------------------------------------
# entry points (same names as the C ABI)
# --------------------------------------------------------------------------
def w4_quantize(W, group: int, out=None, stream=None):
    """quantize_w4: W [E, N, K] fp32 -> (q [E,N,K/2] u8, s, z [E,N,K/group] fp16)."""
    import torch
    _require_cuda(W)
    if W.dim() == 2:
        W = W.unsqueeze(0)
    E, N, K = W.shape
    if out is None:
        out = (_result((E, N, K // 2), torch.uint8, W.device, stream),
               _result((E, N, K // group), torch.float16, W.device, stream),
               _result((E, N, K // group), torch.float16, W.device, stream))
    q, s, z = out
    _check(load_library().w4_quantize(_ptr(W), E, N, K, group, _ptr(q), _ptr(s), _ptr(z),
                                      _stream(stream)), "w4_quantize")
    return q, s, z


def w4_moe_route(logits, k: int, stream=None):
    """Router: logits [M, E] fp32 -> (topk_ids [M,k] int32, topk_weights [M,k] fp32)."""
    import torch
    _require_cuda(logits)
    M, E = logits.shape
    ids = _result((M, k), torch.int32, logits.device, stream)
    w = _result((M, k), torch.float32, logits.device, stream)
    _check(load_library().w4_moe_route(_ptr(logits), M, E, k, _ptr(ids), _ptr(w),
                                       _stream(stream)), "w4_moe_route")
    return ids, w


def w4_moe_align_capacity(M: int, k: int, E: int, block_m: int) -> int:
    cap = load_library().w4_moe_align_capacity(M, k, E, block_m)
    if cap < 0:
        raise W4Error(1, "W4_ERR_INVALID_ARG", "w4_moe_align_capacity: bad arguments")
    return int(cap)


def w4_moe_align(topk_ids, E: int, block_m: int = 16, dev_status=None, out=None,
                 stream=None):
    """Alignment: topk_ids [M, k] int32 -> dict of device tensors (sorted_ids,
    block_expert, expert_offsets, num_padded) plus the shape keys the GEMMs
    need.  Pass a previous result as ``out`` to reuse its buffers."""
    import torch
    _require_cuda(topk_ids, dev_status)
    M, k = topk_ids.shape
    cap = w4_moe_align_capacity(M, k, E, block_m)
    dev = topk_ids.device
    if out is not None:
        if (out["sorted_ids"].numel() != cap or out["expert_offsets"].numel() != E + 1
                or out["block_expert"].numel() != cap // block_m):
            raise ValueError("w4_moe_align: reused buffers have the wrong sizes")
        r = out
        r.update(M=M, k=k, E=E, block_m=block_m)
    else:
        r = dict(sorted_ids=_result(cap, torch.int32, dev, stream),
                 block_expert=_result(cap // block_m, torch.int32, dev, stream),
                 expert_offsets=_result(E + 1, torch.int32, dev, stream),
                 num_padded=_result(1, torch.int32, dev, stream),
                 M=M, k=k, E=E, block_m=block_m)
    _check(load_library().w4_moe_align(_ptr(topk_ids), M, k, E, block_m, _ptr(r["sorted_ids"]),
                                       _ptr(r["block_expert"]), _ptr(r["expert_offsets"]),
                                       _ptr(r["num_padded"]), _ptr(dev_status),
                                       _stream(stream)), "w4_moe_align")
    return r


def w4_gather_activations(x, align: dict, out=None, dev_status=None, stream=None):
    """x [M, d] bf16 -> xg [cap, d + 64] fp16 in slot order: d values in block
    order, then the sums of the groups of 128 (zero rows for padding slots;
    rows past num_padded are left untouched).  Values beyond fp16's range
    saturate and set W4_DEV_FP16_RANGE in dev_status."""
    import torch
    _require_cuda(x, out, dev_status)
    M, d = x.shape
    cap = align["sorted_ids"].numel()
    if out is None:
        out = _result((cap, d + SUM_COLS), torch.float16, x.device, stream)
    _check(load_library().w4_gather_activations(
        _ptr(x), M, d, align["k"], align["E"], align["block_m"], _ptr(align["sorted_ids"]),
        _ptr(align["num_padded"]), _ptr(out), _ptr(dev_status), _stream(stream)),
        "w4_gather_activations")
    return out


def w4_moe_align_gather(topk_ids, x, E: int, block_m: int = 16, dev_status=None, out=None,
                        xg=None, stream=None):
    """Alignment and activation gather in one launch.  Returns (align dict, xg)."""
    import torch
    _require_cuda(topk_ids, x, dev_status, xg)
    M, k = topk_ids.shape
    d = x.shape[1]
    cap = w4_moe_align_capacity(M, k, E, block_m)
    dev = x.device
    if out is None:
        out = dict(sorted_ids=_result(cap, torch.int32, dev, stream),
                   block_expert=_result(cap // block_m, torch.int32, dev, stream),
                   expert_offsets=_result(E + 1, torch.int32, dev, stream),
                   num_padded=_result(1, torch.int32, dev, stream))
    out.update(M=M, k=k, E=E, block_m=block_m)
    if xg is None:
        xg = _result((cap, d + SUM_COLS), torch.float16, dev, stream)
    _check(load_library().w4_moe_align_gather(
        _ptr(topk_ids), _ptr(x), M, d, k, E, block_m, _ptr(out["sorted_ids"]),
        _ptr(out["block_expert"]), _ptr(out["expert_offsets"]), _ptr(out["num_padded"]),
        _ptr(xg), _ptr(dev_status), _stream(stream)), "w4_moe_align_gather")
    return out, xg


def w4_grouped_gemm_gate_up(xg, gu_q, gu_s, gu_z, align: dict, group: int = 128, h=None,
                            dev_status=None, stream=None):
    """xg [cap, d + 64] fp16 (from w4_gather_activations) -> h [cap, m + 64]
    fp16: m values in block order, gelu_tanh(gate) * up per alignment slot,
    then the sums of every quarter (16 values) of each group of 64."""
    import torch
    _require_cuda(xg, gu_q, gu_s, gu_z, h, dev_status)
    M, d = align["M"], xg.shape[1] - SUM_COLS
    E, two_m, _ = gu_q.shape
    m = two_m // 2
    cap = align["sorted_ids"].numel()
    if h is None:
        h = _result((cap, m + SUM_COLS), torch.float16, xg.device, stream)
    _check(load_library().w4_grouped_gemm_gate_up(
        _ptr(xg), M, d, m, E, align["k"], align["block_m"], _ptr(gu_q), _ptr(gu_s), _ptr(gu_z),
        group, _ptr(align["sorted_ids"]), _ptr(align["expert_offsets"]), _ptr(h),
        _ptr(dev_status), _stream(stream)), "w4_grouped_gemm_gate_up")
    return h


def korder_to_natural(a):
    """Undo the GEMMs' block order along the last axis (for inspection and
    tests): column p of every block of 8 holds element (p >> 1) + 4 * (p & 1)."""
    import numpy as np
    n = a.shape[-1]
    perm = np.array([(p >> 1) + 4 * (p & 1) for p in range(8)])
    src = (np.arange(n) // 8) * 8
    inv = np.empty(8, dtype=np.int64)
    inv[perm] = np.arange(8)
    return a[..., src + inv[np.arange(n) % 8]]


def w4_grouped_gemm_down(h, dn_q, dn_s, dn_z, align: dict, group: int = 64, y=None,
                         dev_status=None, stream=None):
    """h [cap, m + 64] fp16 (from w4_grouped_gemm_gate_up) -> y [M*k, d] fp32
    (row = flat assignment index)."""
    import torch
    _require_cuda(h, dn_q, dn_s, dn_z, y, dev_status)
    E, d, half_m = dn_q.shape
    m = half_m * 2
    M, k = align["M"], align["k"]
    if y is None:
        y = _result((M * k, d), torch.float32, h.device, stream)
    _check(load_library().w4_grouped_gemm_down(
        _ptr(h), M, d, m, E, k, align["block_m"], _ptr(dn_q), _ptr(dn_s), _ptr(dn_z), group,
        _ptr(align["sorted_ids"]), _ptr(align["expert_offsets"]), _ptr(y), _ptr(dev_status),
        _stream(stream)), "w4_grouped_gemm_down")
    return y


def w4_moe_combine_fixed_order(y, topk_ids, topk_weights, E: int, out=None, stream=None):
    """out [M, d] bf16 = fixed-order sum_j w[t,j] * y[t*k+j]."""
    import torch
    _require_cuda(y, topk_ids, topk_weights, out)
    M, k = topk_ids.shape
    d = y.shape[1]
    if out is None:
        out = _result((M, d), torch.bfloat16, y.device, stream)
    _check(load_library().w4_moe_combine_fixed_order(
        _ptr(y), _ptr(topk_ids), _ptr(topk_weights), M, k, d, E, _ptr(out), _stream(stream)),
        "w4_moe_combine_fixed_order")
    return out


def w4_moe_combine_prepare(topk_ids, E: int, d: int, counters=None, out=None, stream=None):
    """The counters [M, d/128] int32 of w4_grouped_gemm_down_combine (and
    the zero out rows of tokens with no valid expert id); returns
    (counters, out)."""
    import torch
    _require_cuda(topk_ids, counters, out)
    M, k = topk_ids.shape
    if counters is None:
        counters = _result((M, d // 128), torch.int32, topk_ids.device, stream)
    if out is None:
        out = _result((M, d), torch.bfloat16, topk_ids.device, stream)
    _check(load_library().w4_moe_combine_prepare(
        _ptr(topk_ids), M, k, E, d, _ptr(counters), _ptr(out), _stream(stream)),
        "w4_moe_combine_prepare")
    return counters, out


def w4_grouped_gemm_down_combine(h, dn_q, dn_s, dn_z, align: dict, topk_ids, topk_weights,
                                 counters, out, group: int = 64, y=None, dev_status=None,
                                 stream=None):
    """w4_grouped_gemm_down with the fixed-order combine folded in: out
    [M, d] bf16 (prepared with w4_moe_combine_prepare, which set counters);
    returns (y, out)."""
    import torch
    _require_cuda(h, dn_q, dn_s, dn_z, topk_ids, topk_weights, counters, out, y, dev_status)
    E, d, half_m = dn_q.shape
    m = half_m * 2
    M, k = align["M"], align["k"]
    if y is None:
        y = _result((M * k, d), torch.float32, h.device, stream)
    _check(load_library().w4_grouped_gemm_down_combine(
        _ptr(h), M, d, m, E, k, align["block_m"], _ptr(dn_q), _ptr(dn_s), _ptr(dn_z), group,
        _ptr(align["sorted_ids"]), _ptr(align["expert_offsets"]), _ptr(topk_ids),
        _ptr(topk_weights), _ptr(counters), _ptr(y), _ptr(out), _ptr(dev_status),
        _stream(stream)), "w4_grouped_gemm_down_combine")
    return y, out


def w4_moe_layer_workspace_size(M, d, m, E, k, block_m=16) -> int:
    return int(load_library().w4_moe_layer_workspace_size(M, d, m, E, k, block_m))


def w4_moe_layer(x, topk_ids, topk_weights, gu, dn, block_m: int = 16, gu_group: int = 128,
                 dn_group: int = 64, workspace=None, out=None, dev_status=None, stream=None):
    """The whole routed-expert layer (align+gather, gate_up + activation,
    down, fixed-order combine) as four launches on the current stream.  For up
    to 32 tokens w4_moe_layer_few is the faster one."""
    import torch
    gu_q, gu_s, gu_z = gu
    dn_q, dn_s, dn_z = dn
    _require_cuda(x, topk_ids, topk_weights, gu_q, gu_s, gu_z, dn_q, dn_s, dn_z, workspace,
                  out, dev_status)
    M, d = x.shape
    E, two_m, _ = gu_q.shape
    m = two_m // 2
    k = topk_ids.shape[1]
    need = w4_moe_layer_workspace_size(M, d, m, E, k, block_m)
    if workspace is None:
        workspace = _scratch(need, torch.uint8, x.device, stream)
    if out is None:
        out = _result((M, d), torch.bfloat16, x.device, stream)
    _check(load_library().w4_moe_layer(
        _ptr(x), _ptr(topk_ids), _ptr(topk_weights), M, d, m, E, k, block_m, _ptr(gu_q),
        _ptr(gu_s), _ptr(gu_z), gu_group, _ptr(dn_q), _ptr(dn_s), _ptr(dn_z), dn_group,
        _ptr(workspace), workspace.numel(), _ptr(out), _ptr(dev_status), _stream(stream)),
        "w4_moe_layer")
    return out


def w4_moe_layer_host_workspace_size(M, d, m, E, k, block_m=16) -> int:
    return int(load_library().w4_moe_layer_host_workspace_size(M, d, m, E, k, block_m))


def w4_moe_layer_host(x_host, topk_ids_host, topk_weights_host, gu, dn, out_host, workspace,
                      block_m: int = 16, gu_group: int = 128, dn_group: int = 64,
                      dev_status=None, stream=None):
    """w4_moe_layer from host memory: x [M, d] bf16, topk_ids [M, k] int32
    and topk_weights [M, k] fp32 (page-locked CPU tensors) are copied in and
    out [M, d] bf16 is copied back to out_host, all enqueued on the stream;
    synchronise before reading out_host.  workspace: a device uint8 tensor of
    w4_moe_layer_host_workspace_size(...) bytes."""
    gu_q, gu_s, gu_z = gu
    dn_q, dn_s, dn_z = dn
    _require_cuda(gu_q, gu_s, gu_z, dn_q, dn_s, dn_z, workspace, dev_status)
    for t in (x_host, topk_ids_host, topk_weights_host, out_host):
        if t.is_cuda:
            raise ValueError("w4_moe_layer_host takes host tensors for x, ids, weights and out")
    M, d = x_host.shape
    E, two_m, _ = gu_q.shape
    m = two_m // 2
    k = topk_ids_host.shape[1]
    _check(load_library().w4_moe_layer_host(
        _ptr(x_host), _ptr(topk_ids_host), _ptr(topk_weights_host), M, d, m, E, k, block_m,
        _ptr(gu_q), _ptr(gu_s), _ptr(gu_z), gu_group, _ptr(dn_q), _ptr(dn_s), _ptr(dn_z),
        dn_group, _ptr(workspace), workspace.numel(), _ptr(out_host), _ptr(dev_status),
        _stream(stream)), "w4_moe_layer_host")
    return out_host


def w4_moe_route_align_gather(logits, x, k: int, block_m: int = 16, dev_status=None, out=None,
                              xg=None, ids=None, weights=None, stream=None):
    """Router, alignment and activation gather in one launch, from the logits
    [M, E] fp32.  Returns (topk_ids, topk_weights, align dict, xg)."""
    import torch
    _require_cuda(logits, x, dev_status, xg, ids, weights)
    M, E = logits.shape
    d = x.shape[1]
    cap = w4_moe_align_capacity(M, k, E, block_m)
    dev = x.device
    if out is None:
        out = dict(sorted_ids=_result(cap, torch.int32, dev, stream),
                   block_expert=_result(cap // block_m, torch.int32, dev, stream),
                   expert_offsets=_result(E + 1, torch.int32, dev, stream),
                   num_padded=_result(1, torch.int32, dev, stream))
    out.update(M=M, k=k, E=E, block_m=block_m)
    if xg is None:
        xg = _result((cap, d + SUM_COLS), torch.float16, dev, stream)
    if ids is None:
        ids = _result((M, k), torch.int32, dev, stream)
    if weights is None:
        weights = _result((M, k), torch.float32, dev, stream)
    _check(load_library().w4_moe_route_align_gather(
        _ptr(logits), _ptr(x), M, d, k, E, block_m, _ptr(ids), _ptr(weights),
        _ptr(out["sorted_ids"]), _ptr(out["block_expert"]), _ptr(out["expert_offsets"]),
        _ptr(out["num_padded"]), _ptr(xg), _ptr(dev_status), _stream(stream)),
        "w4_moe_route_align_gather")
    return ids, weights, out, xg


def w4_moe_layer_from_logits(x, logits, k: int, gu, dn, block_m: int = 16, gu_group: int = 128,
                             dn_group: int = 64, workspace=None, out=None, ids=None,
                             weights=None, dev_status=None, stream=None):
    """w4_moe_layer with the router in its first launch: from the logits
    [M, E] fp32.  Returns (out, topk_ids, topk_weights).  For up to 32 tokens
    w4_moe_layer_few_from_logits is the faster one."""
    import torch
    gu_q, gu_s, gu_z = gu
    dn_q, dn_s, dn_z = dn
    _require_cuda(x, logits, gu_q, gu_s, gu_z, dn_q, dn_s, dn_z, workspace, out, ids, weights,
                  dev_status)
    M, d = x.shape
    E, two_m, _ = gu_q.shape
    m = two_m // 2
    need = w4_moe_layer_workspace_size(M, d, m, E, k, block_m)
    if workspace is None:
        workspace = _scratch(need, torch.uint8, x.device, stream)
    if out is None:
        out = _result((M, d), torch.bfloat16, x.device, stream)
    if ids is None:
        ids = _result((M, k), torch.int32, x.device, stream)
    if weights is None:
        weights = _result((M, k), torch.float32, x.device, stream)
    _check(load_library().w4_moe_layer_from_logits(
        _ptr(x), _ptr(logits), M, d, m, E, k, block_m, _ptr(gu_q), _ptr(gu_s), _ptr(gu_z),
        gu_group, _ptr(dn_q), _ptr(dn_s), _ptr(dn_z), dn_group, _ptr(workspace),
        workspace.numel(), _ptr(ids), _ptr(weights), _ptr(out), _ptr(dev_status),
        _stream(stream)), "w4_moe_layer_from_logits")
    return out, ids, weights


def w4_moe_layer_few_workspace_size(M, d, m, E, k) -> int:
    return int(load_library().w4_moe_layer_few_workspace_size(M, d, m, E, k))


def _few_inputs(x, k, gu, dn, gu_group, dn_group, workspace, dev_status, stream):
    """(M, d, m, E, the workspace) of a few-token call, with x, the weights and
    the workspace checked."""
    import torch
    (gq, gs, gz), (dq, ds, dz) = gu, dn
    if x.dim() != 2 or gq.dim() != 3 or gu_group <= 0 or dn_group <= 0:
        raise ValueError("x must be [M, d] and the packed weights [E, rows, columns / 2]")
    M, d = x.shape
    E, two_m, _ = gq.shape
    m = two_m // 2
    u8, f16 = torch.uint8, torch.float16
    g_shape, d_shape = (E, 2 * m, d // gu_group), (E, d, m // dn_group)
    _require(((x, torch.bfloat16, (M, d), "x"),
              (gq, u8, (E, 2 * m, d // 2), "gu's codes"), (gs, f16, g_shape, "gu's scales"),
              (gz, f16, g_shape, "gu's zeros"), (dq, u8, (E, d, m // 2), "dn's codes"),
              (ds, f16, d_shape, "dn's scales"), (dz, f16, d_shape, "dn's zeros")))
    if workspace is None:
        workspace = _scratch(w4_moe_layer_few_workspace_size(M, d, m, E, k), u8, x.device, stream)
    _require_cuda(workspace)
    _require_int32(dev_status)
    return M, d, m, E, workspace


def w4_moe_layer_few(x, topk_ids, topk_weights, gu, dn, gu_group: int = 128, dn_group: int = 64,
                     workspace=None, out=None, dev_status=None, stream=None):
    """The whole routed-expert layer for a few tokens (M <= 32, M k <= 256)
    in one cooperative launch; arguments and result as w4_moe_layer."""
    import torch
    if topk_ids.dim() != 2:
        raise ValueError("topk_ids must be [M, k]")
    k = topk_ids.shape[1]
    M, d, m, E, workspace = _few_inputs(x, k, gu, dn, gu_group, dn_group, workspace, dev_status,
                                        stream)
    _require(((topk_ids, torch.int32, (M, k), "topk_ids"),
              (topk_weights, torch.float32, (M, k), "topk_weights")))
    if out is None:
        out = torch.empty_like(x) if stream is None else \
            _result(x.shape, x.dtype, x.device, stream)
    else:
        _require(((out, torch.bfloat16, (M, d), "out"),))
    _check(load_library().w4_moe_layer_few(
        x.data_ptr(), topk_ids.data_ptr(), topk_weights.data_ptr(), M, d, m, E, k,
        gu[0].data_ptr(), gu[1].data_ptr(), gu[2].data_ptr(), gu_group, dn[0].data_ptr(),
        dn[1].data_ptr(), dn[2].data_ptr(), dn_group, workspace.data_ptr(), workspace.nbytes,
        out.data_ptr(), _ptr(dev_status), _stream(stream)), "w4_moe_layer_few")
    return out


def w4_moe_layer_few_from_logits(x, logits, k: int, gu, dn, gu_group: int = 128,
                                 dn_group: int = 64, workspace=None, out=None, ids=None,
                                 weights=None, dev_status=None, stream=None):
    """w4_moe_layer_few with the router in its launch: from the logits
    [M, E] fp32.  Returns (out, topk_ids, topk_weights)."""
    import torch
    M, d, m, E, workspace = _few_inputs(x, k, gu, dn, gu_group, dn_group, workspace, dev_status,
                                        stream)
    _require(((logits, torch.float32, (M, E), "logits"),))
    if out is None:
        out = torch.empty_like(x) if stream is None else \
            _result(x.shape, x.dtype, x.device, stream)
    else:
        _require(((out, torch.bfloat16, (M, d), "out"),))
    if ids is None:
        ids = _result((M, k), torch.int32, x.device, stream)
    else:
        _require(((ids, torch.int32, (M, k), "ids"),))
    if weights is None:
        weights = _result((M, k), torch.float32, x.device, stream)
    else:
        _require(((weights, torch.float32, (M, k), "weights"),))
    _check(load_library().w4_moe_layer_few_from_logits(
        x.data_ptr(), logits.data_ptr(), M, d, m, E, k, gu[0].data_ptr(), gu[1].data_ptr(),
        gu[2].data_ptr(), gu_group, dn[0].data_ptr(), dn[1].data_ptr(), dn[2].data_ptr(), dn_group,
        workspace.data_ptr(), workspace.nbytes, ids.data_ptr(), weights.data_ptr(), out.data_ptr(),
        _ptr(dev_status), _stream(stream)), "w4_moe_layer_few_from_logits")
    return out, ids, weights


def w4_moe_layer_static_scratch(x, topk_ids, topk_weights, gu, dn, out, block_m: int = 16,
                                gu_group: int = 128, dn_group: int = 64, dev_status=None,
                                stream=None):
    """w4_moe_layer with the intermediates in the library's own static device
    array instead of a workspace: for callers that cannot allocate device
    memory when they run the layer.  Nothing is allocated here either, so the
    caller passes `out` ([M, d] bf16).  Calls that overlap on the GPU share
    the array and race: keep them on one stream."""
    gu_q, gu_s, gu_z = gu
    dn_q, dn_s, dn_z = dn
    _require_cuda(x, topk_ids, topk_weights, gu_q, gu_s, gu_z, dn_q, dn_s, dn_z, out,
                  dev_status)
    M, d = x.shape
    E, two_m, _ = gu_q.shape
    m = two_m // 2
    k = topk_ids.shape[1]
    _check(load_library().w4_moe_layer_static_scratch(
        _ptr(x), _ptr(topk_ids), _ptr(topk_weights), M, d, m, E, k, block_m, _ptr(gu_q),
        _ptr(gu_s), _ptr(gu_z), gu_group, _ptr(dn_q), _ptr(dn_s), _ptr(dn_z), dn_group,
        _ptr(out), _ptr(dev_status), _stream(stream)), "w4_moe_layer_static_scratch")
    return out


def w4_w4a16_linear_workspace_size(M: int, K: int, N: int, group: int = 128) -> int:
    return int(load_library().w4_w4a16_linear_workspace_size(M, K, N, group))


def w4_w4a16_linear(x, q, s, z, group: int = 128, workspace=None, out=None, dev_status=None,
                    stream=None):
    """w4a16_linear: y [M, N] bf16 = x [M, K] bf16 . deq(W)^T with W packed as
    w4_quantize writes it (q [N, K/2] uint8, s/z [N, K/group] fp16).  For up to 32
    rows w4_w4a16_linear_few takes less time."""
    import torch
    _require_cuda(x, q, s, z, workspace, out, dev_status)
    M, K = x.shape
    N = q.shape[0]
    if out is None:
        out = _result((M, N), torch.bfloat16, x.device, stream)
    need = w4_w4a16_linear_workspace_size(M, K, N, group)
    if workspace is None:
        workspace = _scratch(max(need, 256), torch.uint8, x.device, stream)
    _check(load_library().w4_w4a16_linear(
        _ptr(x), M, K, N, _ptr(q), _ptr(s), _ptr(z), group, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(out), _ptr(dev_status),
        _stream(stream)), "w4_w4a16_linear")
    return out


def w4_w4a16_linear_few(x, q, s, z, group: int = 128, out=None, dev_status=None, stream=None):
    """w4_w4a16_linear for up to 32 rows, in one launch without a workspace: y [M, N]
    bf16 = x [M, K] bf16 . deq(W)^T with W packed as w4_quantize writes it."""
    return (_calls_module or _calls()).linear_few(x, q, s, z, group, out, dev_status, stream)


# --------------------------------------------------------------------------
# Beside the layer: RMSNorm and the sampler ("dg-w4-kernels" -- RMSNorm, Sampler)
# --------------------------------------------------------------------------
def w4_rmsnorm(x, weight, eps: float = 1e-6, out=None, stream=None):
    """fused_rmsnorm: y = x / sqrt(mean(x^2) + eps) * weight over the last
    axis; x [..., d] and weight [d] bf16, y bf16."""
    _require_cuda(x, weight, out)
    d = x.shape[-1]
    M = x.numel() // d if d else 0
    if out is None:
        out = _result(x.shape, x.dtype, x.device, stream)
    _check(load_library().w4_rmsnorm(_ptr(x), _ptr(weight), M, d, float(eps), _ptr(out),
                                     _stream(stream)), "w4_rmsnorm")
    return out


def w4_sample_logits_workspace_size(M: int, V: int) -> int:
    return int(load_library().w4_sample_logits_workspace_size(M, V))


def _sampler_ws(logits, workspace, stream):
    import torch
    M, V = logits.shape
    need = w4_sample_logits_workspace_size(M, V)
    if workspace is None:
        workspace = _scratch(max(need, 16), torch.uint8, logits.device, stream)
    return workspace, workspace.numel() * workspace.element_size()


def w4_sample_logits(logits, seed: int = 0, offset: int = 0, entropy=True, sample=True,
                     argmax=True, workspace=None, stream=None):
    """One pass over logits [M, V] fp32: (entropy [M] fp32 nats, Gumbel-max
    sample [M] int64, argmax [M] int64); an output passed as False is skipped
    (None in its place), a tensor is written in place."""
    import torch
    _require_cuda(logits, workspace)
    M, V = logits.shape
    dev = logits.device

    def out(spec, dtype):
        if spec is False or spec is None:
            return None
        if spec is True:
            return _result(M, dtype, dev, stream)
        _require_cuda(spec)
        return spec
    ent = out(entropy, torch.float32)
    smp = out(sample, torch.int64)
    amx = out(argmax, torch.int64)
    ws, ws_bytes = _sampler_ws(logits, workspace, stream)
    _check(load_library().w4_sample_logits(
        _ptr(logits), M, V, seed & (2**64 - 1), offset & (2**64 - 1), _ptr(ent), _ptr(smp),
        _ptr(amx), _ptr(ws), ws_bytes, _stream(stream)), "w4_sample_logits")
    return ent, smp, amx


def w4_fused_entropy(logits, workspace=None, stream=None):
    """fused_entropy: [M, V] fp32 -> [M] fp32 nats, one pass."""
    ent, _, _ = w4_sample_logits(logits, entropy=True, sample=False, argmax=False,
                                 workspace=workspace, stream=stream)
    return ent


def w4_gumbel_argmax_sample(logits, seed: int, offset: int = 0, workspace=None, stream=None):
    """gumbel_argmax_sample: (sample, argmax), both [M] int64, one pass."""
    _, smp, amx = w4_sample_logits(logits, seed, offset, entropy=False, sample=True,
                                   argmax=True, workspace=workspace, stream=stream)
    return smp, amx


# --------------------------------------------------------------------------
# A paged key/value cache: the pool is a tensor [..., P, page_size, Hkv, D] of
# 16-bit values (the leading axes, layers and K / V, are its planes), the state
# three int32 tensors table [B, W] (-1: no page), lens [B] and refs [P].
# --------------------------------------------------------------------------
def _require_int32(*ts):
    """Contiguous int32 CUDA tensors (or None)."""
    int32 = (_torch or _load_torch()).int32
    for t in ts:
        if t is None or (t.is_cuda and t.dtype is int32 and t.is_contiguous()):
            continue
        if not t.is_cuda:
            raise ValueError("tensors passed to the CUDA library must live on the GPU")
        if not t.is_contiguous():
            raise ValueError("tensors passed to the CUDA library must be contiguous")
        raise ValueError("tables, lengths, slots, page lists and status must be int32")


def _kv_state(table, lens, refs, dev_status):
    """(B, W, P) of a cache's state, with its tensors checked."""
    _require_int32(table, lens, refs, dev_status)
    if table.dim() != 2 or refs.dim() != 1 or lens.shape != table.shape[:1]:
        raise ValueError("lens must be [B] and refs [P] for a table [B, W]")
    B, W = table.shape
    return B, W, refs.shape[0]


def _kv_pool(pool, P):
    """(planes, bytes of a page in one plane, page_size) of a pool."""
    _require_cuda(pool)
    if pool.dim() < 4 or pool.shape[-4] != P or pool.element_size() != 2:
        raise ValueError("the pool must be [..., P, page_size, Hkv, D] of 16-bit values")
    page, Hkv, D = pool.shape[-3:]
    page_bytes = page * Hkv * D * 2
    return pool.numel() * 2 // max(P * page_bytes, 1), page_bytes, page


def _kv_lists(first, *others):
    """The length of equally long int32 lists."""
    _require_int32(first, *others)
    shape = first.shape
    if len(shape) != 1:
        raise ValueError("slots and page lists must be one-dimensional and equally long")
    for t in others:
        if t.shape != shape:
            raise ValueError("slots and page lists must be one-dimensional and equally long")
    return shape[0]


def _kv_workspace(workspace, P, n, device, stream):
    import torch
    if workspace is None:
        workspace = _scratch(w4_kv_workspace_size(P, n), torch.uint8, device, stream)
    _require_cuda(workspace)
    return workspace, workspace.nbytes


def w4_kv_workspace_size(P: int, n: int = 0) -> int:
    return int(load_library().w4_kv_workspace_size(P, n))


def w4_kv_reserve(table, lens, refs, slots, new_lens, page_size: int, dev_status=None,
                  stream=None):
    """Grow slots[i] to new_lens[i] tokens; pages are taken lowest free first."""
    B, W, P = _kv_state(table, lens, refs, dev_status)
    n = _kv_lists(slots, new_lens)
    _check(load_library().w4_kv_reserve(_ptr(table), B, W, _ptr(lens), _ptr(refs), P, _ptr(slots),
                                        _ptr(new_lens), n, page_size, _ptr(dev_status),
                                        _stream(stream)), "w4_kv_reserve")


def w4_kv_free(table, lens, refs, slots, dev_status=None, stream=None):
    """Empty slots[i] and let go of its pages."""
    B, W, P = _kv_state(table, lens, refs, dev_status)
    n = _kv_lists(slots)
    _check(load_library().w4_kv_free(_ptr(table), B, W, _ptr(lens), _ptr(refs), P, _ptr(slots), n,
                                     _ptr(dev_status), _stream(stream)), "w4_kv_free")


def w4_kv_fork(pool, table, lens, refs, parents, children, workspace=None, dev_status=None,
               stream=None):
    """Make the empty slots children[i] copies of parents[i]: full pages are
    shared, the last, partly filled one is copied in every plane."""
    B, W, P = _kv_state(table, lens, refs, dev_status)
    planes, page_bytes, page = _kv_pool(pool, P)
    n = _kv_lists(parents, children)
    workspace, nbytes = _kv_workspace(workspace, P, n, pool.device, stream)
    _check(load_library().w4_kv_fork(_ptr(pool), planes, page_bytes, _ptr(table), B, W, _ptr(lens),
                                     _ptr(refs), P, _ptr(parents), _ptr(children), n, page,
                                     _ptr(workspace), nbytes, _ptr(dev_status), _stream(stream)),
           "w4_kv_fork")


def w4_kv_copy_pages(pool, src, dst, dev_status=None, stream=None):
    """Copy page src[i] to page dst[i] in every plane (disjoint pages)."""
    P = pool.shape[-4] if pool.dim() >= 4 else 0
    planes, page_bytes, _ = _kv_pool(pool, P)
    _require_int32(dev_status)
    n = _kv_lists(src, dst)
    _check(load_library().w4_kv_copy_pages(_ptr(pool), planes, page_bytes, P, _ptr(src), _ptr(dst),
                                           n, _ptr(dev_status), _stream(stream)),
           "w4_kv_copy_pages")


def w4_kv_compact(pool, table, refs, table_out=None, refs_out=None, workspace=None,
                  dev_status=None, stream=None):
    """Move the pages in use to the front of the pool.  Returns (table, refs)
    with the pages renamed: table_out and refs_out, by default table and refs
    themselves."""
    table_out = table if table_out is None else table_out
    refs_out = refs if refs_out is None else refs_out
    _require_int32(table, refs, table_out, refs_out, dev_status)
    if table.dim() != 2 or refs.dim() != 1 or table_out.shape != table.shape or \
            refs_out.shape != refs.shape:
        raise ValueError("table_out and refs_out must have the shapes of table and refs")
    B, W = table.shape
    P = refs.shape[0]
    planes, page_bytes, _ = _kv_pool(pool, P)
    workspace, nbytes = _kv_workspace(workspace, P, 0, pool.device, stream)
    _check(load_library().w4_kv_compact(_ptr(pool), planes, page_bytes, _ptr(table), B, W,
                                        _ptr(refs), P, _ptr(table_out), _ptr(refs_out),
                                        _ptr(workspace), nbytes, _ptr(dev_status),
                                        _stream(stream)), "w4_kv_compact")
    return table_out, refs_out


def _rows16(t, dtype, what):
    """A CUDA tensor of the type, contiguous along its last axis.  Returns its strides."""
    if not t.is_cuda:
        raise ValueError("tensors passed to the CUDA library must live on the GPU")
    strides = t.stride()
    if t.dtype is not dtype or not strides or strides[-1] != 1:
        raise ValueError(f"{what} must be {dtype}, contiguous along the last axis")
    return strides


def _kv_planes(k_pages, v_pages):
    """(type, shape [P, page_size, Hkv, D], strides) of one layer's planes."""
    dtype, shape = k_pages.dtype, k_pages.shape
    strides = _rows16(k_pages, dtype, "k_pages")
    if k_pages.dim() != 4 or k_pages.element_size() != 2 or v_pages.shape != shape or \
            _rows16(v_pages, dtype, "v_pages") != strides:
        raise ValueError("k_pages and v_pages must be alike, [P, page_size, Hkv, D] of 16 bits")
    return dtype, shape, strides


def _kv_batch(table, lens, q_offsets):
    """(B, W) of q_offsets [B + 1], with a table and lengths for as many."""
    B = q_offsets.numel() - 1
    if B < 0 or q_offsets.dim() != 1 or table.dim() != 2 or lens.dim() != 1:
        raise ValueError("q_offsets must be [B + 1] for a table [B, W] and lens [B]")
    rows, W = table.shape
    if rows < B or lens.numel() < B:
        raise ValueError("q_offsets must be [B + 1] for a table [B, W] and lens [B]")
    return B, W


def w4_kv_append(k_pages, v_pages, table, lens, k, v, q_offsets, dev_status=None, stream=None):
    """Write the new tokens' keys and values [T, Hkv, D] (any strides of tokens
    and heads) into their pages; slot b's are rows q_offsets[b] ..
    q_offsets[b + 1] and its last tokens."""
    dtype, (P, page, Hkv, D), strides = _kv_planes(k_pages, v_pages)
    ks, vs = _rows16(k, dtype, "k"), _rows16(v, dtype, "v")
    _require_int32(table, lens, q_offsets, dev_status)
    if k.dim() != 3 or k.shape != v.shape or k.shape[1:] != (Hkv, D):
        raise ValueError("k and v must be [T, Hkv, D] of the pages' type")
    B, W = _kv_batch(table, lens, q_offsets)
    if B == 0:
        return
    _check(load_library().w4_kv_append(
        k_pages.data_ptr(), v_pages.data_ptr(), *strides[:3], P, page, Hkv, D, table.data_ptr(), B,
        W, lens.data_ptr(), k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1],
        q_offsets.data_ptr(), k.shape[0], _ptr(dev_status), _stream(stream)), "w4_kv_append")


def w4_kv_keep(pool, table, lens, refs, q_offsets, kept, kept_offsets, lens_out=None,
               dev_status=None, stream=None):
    """Keep the accepted ones of each slot's new tokens: of slot b's last
    q_offsets[b + 1] - q_offsets[b] tokens those that kept[kept_offsets[b]:
    kept_offsets[b + 1]] names (ascending, from 0) move together in every plane,
    the others are taken back.  Returns the new lengths: lens_out, by default
    lens itself."""
    return (_calls_module or _calls()).kv_keep(pool, table, lens, refs, q_offsets, kept, kept_offsets,
                                               lens if lens_out is None else lens_out, dev_status,
                                               stream)


# --------------------------------------------------------------------------
# Norms and rotation of queries and keys
# --------------------------------------------------------------------------
_ROPE_METHODS = {"linear": 0, "base": 1, "parts": 2}


def w4_rope_steps(rot: int, base: float = 10000.0, method: str = "linear", factor: float = 1.0,
                  trained_len: float = 0.0, low: float = 0.0, high: float = 0.0, device="cuda"):
    """The rotation's frequencies base^(-2 i / rot) as a table [rot / 2] int64 for
    w4_qk_norm_rope and w4_kv_append_rope, made once.  For contexts longer than the
    trained one by `factor`: method "linear" divides them by it, "base" raises the
    base, "parts" divides those that turn less than `low` times within trained_len,
    keeps those that turn more than `high` times and mixes between."""
    import torch
    if method not in _ROPE_METHODS:
        raise ValueError(f"method must be one of {sorted(_ROPE_METHODS)}")
    steps = torch.empty(max(rot // 2, 0), dtype=torch.int64)
    _check(load_library().w4_rope_steps(rot, base, _ROPE_METHODS[method], factor, trained_len, low,
                                        high, _ptr(steps)), "w4_rope_steps")
    return steps.to(device)


def w4_qk_norm_rope(q, k, positions, steps, q_weight=None, k_weight=None, eps: float = 1e-6,
                    interleaved: bool = False, amplitude: float = 1.0, q_out=None, k_out=None,
                    stream=None):
    """Queries [T, Hq, D] and keys [T, Hkv, D] (any strides of tokens and heads)
    normed for each head (with a weight [D]) and their first 2 len(steps) values
    rotated by positions [T] int32, in one pass.  Returns (q_out, k_out); they may
    be q and k themselves, and else have no memory in common with an input."""
    return (_calls_module or _calls()).qk_norm_rope(q, k, positions, steps, q_weight, k_weight, eps,
                                                    interleaved, amplitude, q_out, k_out, stream)


def w4_kv_append_rope(k_pages, v_pages, table, lens, q, k, v, q_offsets, steps, positions=None,
                      q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                      amplitude: float = 1.0, q_out=None, dev_status=None, stream=None):
    """w4_qk_norm_rope and w4_kv_append in one pass: returns the queries, writes the
    keys and values [T, Hkv, D] of the slots' last tokens into their pages.
    positions defaults to the tokens' places in their sequences."""
    return (_calls_module or _calls()).kv_append_rope(
        k_pages, v_pages, table, lens, q, k, v, q_offsets, steps, positions, q_weight, k_weight, eps,
        interleaved, amplitude, q_out, dev_status, stream)


def w4_attn_shared_prefix_workspace_size(T: int, B: int, G: int, max_q: int, Hq: int, Hkv: int,
                                         D: int) -> int:
    return int(load_library().w4_attn_shared_prefix_workspace_size(T, B, G, max_q, Hq, Hkv, D))


def w4_attn_shared_prefix(q, k_pages, v_pages, table, lens, q_offsets, group_offsets=None,
                          shared_lens=None, max_q: int = 1, causal: bool = True, scale=None,
                          workspace=None, out=None, dev_status=None, stream=None):
    """Attention of q [T, Hq, D] (any strides of tokens and heads) over one
    layer's pages [P, page_size, Hkv, D]; sequences group_offsets[g] ..
    group_offsets[g + 1] share their first shared_lens[g] tokens, which are read
    once for the group.  scale defaults to 1 / sqrt(D).  Returns out [T, Hq, D]."""
    if _calls_module is None and not _calls_built():
        return _attn_shared_prefix(q, k_pages, v_pages, table, lens, q_offsets, group_offsets,
                                   shared_lens, max_q, causal, scale, workspace, out, dev_status,
                                   stream)
    return (_calls_module or _calls()).attn(q, k_pages, v_pages, table, lens, q_offsets, None, causal,
                                            group_offsets, shared_lens, max_q, scale, workspace, out,
                                            dev_status, stream)


def _attn_shared_prefix(q, k_pages, v_pages, table, lens, q_offsets, group_offsets, shared_lens,
                        max_q, causal, scale, workspace, out, dev_status, stream):
    """The same call of the library where the module has not been built for this torch."""
    torch = _torch or _load_torch()
    dtype, (P, page, Hkv, D), strides = _kv_planes(k_pages, v_pages)
    qs = _rows16(q, dtype, "q")
    _require_int32(table, lens, q_offsets, group_offsets, shared_lens, dev_status)
    if q.dim() != 3 or (dtype is not torch.bfloat16 and dtype is not torch.float16):
        raise ValueError("q must be [T, Hq, D] of the pages' type, bf16 or fp16")
    T, Hq, q_d = q.shape
    if q_d != D:
        raise ValueError("q must be [T, Hq, D] of the pages' type, bf16 or fp16")
    B, W = _kv_batch(table, lens, q_offsets)
    G = 0 if group_offsets is None else group_offsets.numel() - 1
    if G < 0 or (G > 0 and (shared_lens is None or shared_lens.numel() != G)):
        raise ValueError("group_offsets must be [G + 1] and shared_lens [G]")
    if out is not None:
        _require(((out, dtype, (T, Hq, D), "out"),))
    if workspace is not None:
        _require_cuda(workspace)
    device = torch.cuda.current_device()
    for t in (q, k_pages, v_pages, table, lens, q_offsets, group_offsets, shared_lens, workspace, out,
              dev_status):
        if t is not None and t.get_device() != device:
            raise ValueError("tensors passed to the CUDA library must live on the current device")
    if out is None:
        out = _result((T, Hq, D), dtype, q.device, stream)
    if workspace is None:
        workspace = _scratch(
            max(w4_attn_shared_prefix_workspace_size(T, B, G, max_q, Hq, Hkv, D), 256)
            if Hkv and Hq % Hkv == 0 else 256, torch.uint8, q.device, stream)
    _check(load_library().w4_attn_shared_prefix(
        q.data_ptr(), qs[0], qs[1], k_pages.data_ptr(), v_pages.data_ptr(), *strides[:3], P, page,
        table.data_ptr(), W, lens.data_ptr(), q_offsets.data_ptr(), T, B, max_q,
        _ptr(group_offsets), _ptr(shared_lens), G, Hq, Hkv, D,
        0 if dtype is torch.bfloat16 else 1, int(causal), D ** -0.5 if scale is None else scale,
        workspace.data_ptr(), workspace.nbytes, out.data_ptr(), _ptr(dev_status),
        _stream(stream)), "w4_attn_shared_prefix")
    return out


def w4_attn_tree(q, k_pages, v_pages, table, lens, q_offsets, tree, group_offsets=None,
                 shared_lens=None, max_q: int = 1, scale=None, workspace=None, out=None,
                 dev_status=None, stream=None):
    """w4_attn_shared_prefix for trees of drafted tokens: bit j % 32 of word j // 32 of
    row t of tree [T, words] int32 tells whether query t sees its sequence's j-th new
    token; the older ones it sees all.  Returns out [T, Hq, D]."""
    if tree is None:
        raise ValueError("tree must be [T, words], a bit for each of max_q tokens in a row")
    return (_calls_module or _calls()).attn(q, k_pages, v_pages, table, lens, q_offsets, tree, False,
                                            group_offsets, shared_lens, max_q, scale, workspace, out,
                                            dev_status, stream)
