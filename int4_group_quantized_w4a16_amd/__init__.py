"""MI355X (gfx950) W4A16 fused-QKV library (and its W8A16 sibling): thin Python binding over libkaio.so.

Every function here only marshals arguments (shape/dtype/device checks,
output allocation through PyTorch, the current HIP stream) and calls the
C ABI declared in ``include/kaio.h``.  All arithmetic runs in the HIP
kernels; there is no CPU fallback -- if ``libkaio.so`` is missing or the
device is not gfx950 the call raises.

    kaio_qkv_w4a16(x, w_q, w_k, w_v, s_q, s_k, s_v) -> (q, k, v)
    kaio_qkv_w8a16(x, w_q, w_k, w_v, s_q, s_k, s_v) -> (q, k, v)
    kaio_gemm_f16f32(a, b) -> c
    kaio_gemm_f16f32_bwd(a, b, grad) -> (grad_a, grad_b)
    kaio_dequant_group_bwd(dy, scale, group_size) -> dq
    kaio_linear_w4a16(x, w, s, bias=, activation=, residual=) -> y
    kaio_quantize_rows(x) -> (q, scale)
    kaio_linear_w8a8(x, w, w_scale, x_scale=, bias=, activation=, residual=) -> y
    KaioExperts(router, w_gate, s_gate, w_up, s_up, w_down, s_down): the weights of a mixture of experts, for
    kaio_moe_w4a16(x, experts, top_k, normalize=, activation=, residual=) -> y
    KaioPagedKV(k_cache, v_cache, page_table, q_start, lens): a paged cache and its batch, for
    kaio_rope_append(q, k, v, positions, inv_freq, sections, paged) -> q
    kaio_paged_attention(q, paged, max_new, scale, window=, sinks=) -> out
"""
from __future__ import annotations

import ctypes
import os

__all__ = ["DTYPE_CODES", "KaioError", "kaio_qkv_w4a16", "kaio_qkv_w8a16", "kaio_gemm_f16f32", "kaio_gemm_f16f32_bwd",
           "kaio_dequant_group_bwd", "kaio_linear_w4a16", "kaio_quantize_rows",
           "kaio_linear_w8a8", "KaioExperts", "kaio_moe_w4a16", "KaioPagedKV", "kaio_rope_append", "kaio_paged_attention",
           "ACTIVATION_CODES",
           "kaio_last_error", "kaio_version", "lib", "LIB_PATH", "GROUP_SIZE"]

# KAIO_LIBRARY may name another in-tree build of the same library (the host-sanitizer
# build used by the CPU boundary tests); by default the in-tree libkaio.so is loaded.
LIB_PATH = os.environ.get("KAIO_LIBRARY") or os.path.join(os.path.dirname(os.path.abspath(__file__)), "libkaio.so")
GROUP_SIZE = 128

STATUS = {0: "OK", 1: "INVALID_ARGUMENT", 2: "INVALID_PROBLEM", 3: "UNSUPPORTED", 4: "DEVICE", 5: "LAUNCH"}
DTYPE_CODES = {"f32": 0, "bf16": 1, "f16": 2, "f64": 3}
ACTIVATION_CODES = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


class KaioError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"[{STATUS.get(status, status)}] {message}")
        self.status = status
        self.message = message


_lib = None


class _PagedKV(ctypes.Structure):
    """kaio_paged_kv of include/kaio.h."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_cache", "v_cache", "page_table", "q_start", "lens")] + \
               [("dtype", ctypes.c_int32)] + \
               [(n, ctypes.c_uint32) for n in ("pages", "page_size", "kv_heads", "head_dim", "seqs", "table_width")]


class _Experts(ctypes.Structure):
    """kaio_experts of include/kaio.h."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("router", "w_gate", "s_gate", "w_up", "s_up", "w_down", "s_down")] + \
               [(n, ctypes.c_uint32) for n in ("experts", "hidden", "inner", "group_size")]


def lib() -> ctypes.CDLL:
    """The loaded C library (loads on first use; raises if it was never built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m int4_group_quantized_w4a16_amd.build_lib`")
        L = ctypes.CDLL(LIB_PATH)
        vp, u32, i32 = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_int32
        L.kaio_qkv_w4a16.argtypes = [vp] * 10 + [u32] * 4 + [vp]
        L.kaio_qkv_w4a16.restype = ctypes.c_int
        L.kaio_qkv_w8a16.argtypes = [vp] * 10 + [u32] * 4 + [vp]
        L.kaio_qkv_w8a16.restype = ctypes.c_int
        L.kaio_gemm_f16f32.argtypes = [vp, vp, vp, u32, u32, u32, vp]
        L.kaio_gemm_f16f32.restype = ctypes.c_int
        L.kaio_gemm_f16f32_bwd.argtypes = [vp] * 5 + [u32] * 3 + [vp, ctypes.c_size_t, vp]
        L.kaio_gemm_f16f32_bwd.restype = ctypes.c_int
        L.kaio_gemm_f16f32_bwd_noalloc.argtypes = [vp] * 5 + [u32] * 3 + [vp]
        L.kaio_gemm_f16f32_bwd_noalloc.restype = ctypes.c_int
        L.kaio_gemm_f16f32_bwd_workspace_size.argtypes = [u32, u32]
        L.kaio_gemm_f16f32_bwd_workspace_size.restype = ctypes.c_size_t
        L.kaio_dequant_group_bwd.argtypes = [ctypes.c_int, i32, i32, i32, vp, vp, vp, vp, ctypes.c_size_t, vp]
        L.kaio_dequant_group_bwd.restype = ctypes.c_int
        L.kaio_qkv_plan.argtypes = [u32] * 4 + [vp]
        L.kaio_qkv_plan.restype = ctypes.c_int
        L.kaio_linear_w4a16.argtypes = [vp] * 6 + [u32] * 4 + [ctypes.c_int, vp]
        L.kaio_linear_w4a16.restype = ctypes.c_int
        L.kaio_quantize_rows.argtypes = [ctypes.c_int] + [vp] * 3 + [u32] * 2 + [vp]
        L.kaio_quantize_rows.restype = ctypes.c_int
        L.kaio_linear_w8a8.argtypes = [ctypes.c_int] + [vp] * 7 + [u32] * 3 + [ctypes.c_int, vp, ctypes.c_size_t, vp]
        L.kaio_linear_w8a8.restype = ctypes.c_int
        L.kaio_linear_w8a8_workspace_size.argtypes = [u32] * 3 + [i32]
        L.kaio_linear_w8a8_workspace_size.restype = ctypes.c_size_t
        L.kaio_moe_w4a16.argtypes = [vp] * 4 + [u32] * 2 + [i32, ctypes.c_int, vp, ctypes.c_size_t, vp]
        L.kaio_moe_w4a16.restype = ctypes.c_int
        L.kaio_moe_w4a16_workspace_size.argtypes = [vp] + [u32] * 2
        L.kaio_moe_w4a16_workspace_size.restype = ctypes.c_size_t
        L.kaio_rope_append.argtypes = [vp] * 7 + [u32, i32, vp, u32, u32, vp]
        L.kaio_rope_append.restype = ctypes.c_int
        L.kaio_paged_attention.argtypes = [vp] * 3 + [u32] * 3 + [ctypes.c_float, u32, u32, vp, ctypes.c_size_t, vp]
        L.kaio_paged_attention.restype = ctypes.c_int
        L.kaio_paged_attention_workspace_size.argtypes = [vp, u32, u32, u32]
        L.kaio_paged_attention_workspace_size.restype = ctypes.c_size_t
        L.kaio_last_error.argtypes = []
        L.kaio_last_error.restype = ctypes.c_char_p
        L.kaio_version.argtypes = []
        L.kaio_version.restype = ctypes.c_char_p
        _lib = L
    return _lib


_fast = None


def _quick():
    """csrc/torch_binding.cpp, bound to the loaded library: the short way of ordinary calls.  It returns None for
    anything it does not take, which then goes through the checks below.  False where it was never built, or was built
    for another torch than the one that is loaded."""
    global _fast
    if _fast is None:
        L = lib()
        _fast = False
        if os.path.exists(os.path.join(os.path.dirname(os.path.abspath(__file__)), "_binding.so")):
            import warnings
            import torch  # (its libraries come first)
            try:
                from . import _binding as b
            except ImportError as e:
                warnings.warn(f"_binding.so does not load, calls go through ctypes: {e}")
                return _fast
            if getattr(b, "torch_version", None) != torch.__version__:
                warnings.warn("_binding.so was built for another torch, calls go through ctypes: build again")
                return _fast
            b.bind(*[ctypes.cast(f, ctypes.c_void_p).value for f in (
                L.kaio_linear_w4a16, L.kaio_rope_append, L.kaio_paged_attention, L.kaio_paged_attention_workspace_size,
                L.kaio_quantize_rows, L.kaio_linear_w8a8, L.kaio_linear_w8a8_workspace_size, L.kaio_moe_w4a16,
                L.kaio_moe_w4a16_workspace_size)])
            _fast = b
    return _fast


def kaio_last_error() -> str:
    return lib().kaio_last_error().decode()


def kaio_version() -> str:
    return lib().kaio_version().decode()


def kaio_qkv_plan(m: int, n: int, k: int, bits: int = 4) -> dict:
    """The kernel form a QKV call of these sizes runs (kaio_qkv_plan; host only)."""
    plan = (ctypes.c_uint32 * 5)()
    _check(lib().kaio_qkv_plan(m, n, k, bits, plan))
    return {"kernel": ("split_k", "tile", "tile_one_output")[plan[0]], "waves": plan[1], "rows": plan[2],
            "sets": plan[3], "outputs": 1 if plan[0] == 2 else 3, "workgroups": plan[4]}


def _check(status: int):
    if status != 0:
        raise KaioError(status, kaio_last_error())


def _call(device, fn, *args):
    """fn(*args) of the C library, which launches on the current device, on ``device``."""
    import torch
    if torch.cuda.current_device() == device.index:
        _check(fn(*args))
        return
    with torch.cuda.device(device):
        _check(fn(*args))


def _stream(device, stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _allocate(device, stream, make):
    """make() with ``stream`` (if given) current, so that the memory it allocates belongs to the stream that uses it."""
    if stream is None:
        return make()
    import torch
    s = stream if isinstance(stream, torch.cuda.Stream) else \
        torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=device)
    with torch.cuda.stream(s):
        return make()


def _tensor(t, name, dtypes, device=None, rank=2, any_offset=False):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != rank:
        raise ValueError(f"{name} must be rank-{rank}, got shape {tuple(t.shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a HIP device; there is no CPU fallback")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous() or (t.storage_offset() != 0 and not any_offset):
        raise ValueError(f"{name} must be contiguous" + ("" if any_offset else " with zero offset"))
    return t


def _u32_dtypes():
    import torch
    return (torch.int32, torch.uint32) if hasattr(torch, "uint32") else (torch.int32,)


def _qkv(fn, bits, x, w_q, w_k, w_v, s_q, s_k, s_v, q, k, v, stream):
    import torch
    f16 = (torch.float16,)
    _tensor(x, "x", f16)
    dev = x.device
    M, K = x.shape
    per_word = 32 // bits
    ws = [_tensor(t, n, _u32_dtypes(), dev) for t, n in ((w_q, "w_q_packed"), (w_k, "w_k_packed"), (w_v, "w_v_packed"))]
    ss = [_tensor(t, n, f16, dev) for t, n in ((s_q, "scales_q"), (s_k, "scales_k"), (s_v, "scales_v"))]
    if K % GROUP_SIZE:
        raise ValueError(f"K ({K}) must be a multiple of group_size ({GROUP_SIZE})")
    for t, n in zip(ws, ("w_q_packed", "w_k_packed", "w_v_packed")):
        if t.shape[0] != K // per_word:
            raise ValueError(f"{n} has {t.shape[0]} rows, expected K/{per_word} = {K // per_word} (K={K})")
    for t, n in zip(ss, ("scales_q", "scales_k", "scales_v")):
        if t.shape[0] != K // GROUP_SIZE:
            raise ValueError(f"{n} has {t.shape[0]} rows, expected K/{GROUP_SIZE} = {K // GROUP_SIZE} (K={K})")
    Ns = [t.shape[1] for t in ws + ss]
    if len(set(Ns)) != 1:
        raise ValueError(f"N mismatch across weight/scale tensors: {Ns}")
    N = Ns[0]
    outs = []
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        if t is None:
            t = torch.empty((M, N), dtype=torch.float16, device=dev)
        _tensor(t, n, f16, dev)
        if tuple(t.shape) != (M, N):
            raise ValueError(f"output {n} must be [{M}, {N}]")
        outs.append(t)
    for dim in (M, N, K):
        if dim >= 2 ** 32:
            raise ValueError("dimension exceeds u32")
    _call(dev, fn, x.data_ptr(), *[t.data_ptr() for t in ws], *[t.data_ptr() for t in ss], *[t.data_ptr() for t in outs], M,
          N, K, GROUP_SIZE, _stream(dev, stream))
    return tuple(outs)


def kaio_qkv_w4a16(x, w_q, w_k, w_v, s_q, s_k, s_v, q=None, k=None, v=None, stream=None):
    """Fused W4A16 QKV projection; returns (q, k, v), each f16[M, N].

    x f16[M,K]; w_* packed INT4 as int32/uint32 [K/8, N]; s_* f16[K/128, N].
    """
    return _qkv(lib().kaio_qkv_w4a16, 4, x, w_q, w_k, w_v, s_q, s_k, s_v, q, k, v, stream)


def kaio_qkv_w8a16(x, w_q, w_k, w_v, s_q, s_k, s_v, q=None, k=None, v=None, stream=None):
    """Fused W8A16 QKV projection; returns (q, k, v), each f16[M, N].

    x f16[M,K]; w_* packed INT8 as int32/uint32 [K/4, N] (byte i of row r holds k = 4r+i);
    s_* f16[K/128, N].
    """
    return _qkv(lib().kaio_qkv_w8a16, 8, x, w_q, w_k, w_v, s_q, s_k, s_v, q, k, v, stream)


def kaio_gemm_f16f32(a, b, c=None, stream=None):
    """C = A . B with A f16[M,K], B f16[K,N]; returns C f32[M,N]."""
    import torch
    _tensor(a, "a", (torch.float16,))
    _tensor(b, "b", (torch.float16,), a.device)
    M, K = a.shape
    Kb, N = b.shape
    if K != Kb:
        raise ValueError(f"K mismatch between inputs: a is [{M}, {K}], b is [{Kb}, {N}]")
    if c is None:
        c = torch.empty((M, N), dtype=torch.float32, device=a.device)
    _tensor(c, "c", (torch.float32,), a.device)
    if tuple(c.shape) != (M, N):
        raise ValueError(f"c must be [{M}, {N}]")
    _call(a.device, lib().kaio_gemm_f16f32, a.data_ptr(), b.data_ptr(), c.data_ptr(), M, N, K, _stream(a.device, stream))
    return c


def kaio_gemm_f16f32_bwd(a, b, grad, grad_a=None, grad_b=None, workspace=None, stream=None):
    """Backward of C = A . B: returns (grad_a f16[M,K], grad_b f16[K,N]) for grad f32[M,N].

    grad is cast to f16 first; each gradient is accumulated in f32 and rounded to f16.
    ``workspace`` (uint8, at least M*N*2 bytes) is allocated here when not given.
    """
    import torch
    _tensor(a, "a", (torch.float16,))
    _tensor(b, "b", (torch.float16,), a.device)
    _tensor(grad, "grad", (torch.float32,), a.device)
    M, K = a.shape
    Kb, N = b.shape
    if K != Kb or tuple(grad.shape) != (M, N):
        raise ValueError(f"shape mismatch: a [{M}, {K}], b [{Kb}, {N}], grad {list(grad.shape)}")
    if grad_a is None:
        grad_a = torch.empty((M, K), dtype=torch.float16, device=a.device)
    if grad_b is None:
        grad_b = torch.empty((K, N), dtype=torch.float16, device=a.device)
    _tensor(grad_a, "grad_a", (torch.float16,), a.device)
    _tensor(grad_b, "grad_b", (torch.float16,), a.device)
    if tuple(grad_a.shape) != (M, K) or tuple(grad_b.shape) != (K, N):
        raise ValueError(f"grad_a must be [{M}, {K}] and grad_b [{K}, {N}]")
    need = lib().kaio_gemm_f16f32_bwd_workspace_size(M, N)
    if workspace is None:
        workspace = torch.empty((max(need, 16),), dtype=torch.uint8, device=a.device)
    _tensor(workspace, "workspace", (torch.uint8,), a.device, rank=1)
    _call(a.device, lib().kaio_gemm_f16f32_bwd, a.data_ptr(), b.data_ptr(), grad.data_ptr(), grad_a.data_ptr(),
          grad_b.data_ptr(), M, N, K, workspace.data_ptr(), workspace.numel(), _stream(a.device, stream))
    return grad_a, grad_b


def kaio_dequant_group_bwd(dy, scale, group_size, dq=None, stream=None):
    """dq[i, j] = dy[i, j] * scale[i, j // group_size], bit-exact, same dtype as dy."""
    import torch
    codes = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2, torch.float64: 3}
    _tensor(dy, "d_output", tuple(codes))
    _tensor(scale, "scale", (dy.dtype,), dy.device)
    outer, axis = dy.shape
    if group_size <= 0 or axis % group_size:
        raise ValueError("axis_size must be a positive multiple of group_size")
    if tuple(scale.shape) != (outer, axis // group_size):
        raise ValueError("scale shape != [outer, num_groups]")
    if dq is None:
        dq = torch.empty_like(dy)
    _tensor(dq, "d_input", (dy.dtype,), dy.device)
    if tuple(dq.shape) != (outer, axis):
        raise ValueError("d_input shape != [outer, axis_size]")
    if outer >= 2 ** 31 or axis >= 2 ** 31:
        raise ValueError("sizes exceed i32")
    _call(dy.device, lib().kaio_dequant_group_bwd, codes[dy.dtype], outer, axis, group_size, dy.data_ptr(),
          scale.data_ptr(), dq.data_ptr(), None, 0, _stream(dy.device, stream))
    return dq


def kaio_linear_w4a16(x, w, s, bias=None, activation="none", residual=None, y=None, stream=None):
    """y = act(x . (int4(w) * s) + bias) + residual, one rounding to f16; returns y f16[M, N].

    x f16[M,K]; w packed INT4 as int32/uint32 [K/8, N]; s f16[K/128, N]; bias f16[N]; residual f16[M, N];
    activation one of ACTIVATION_CODES.  ``y`` may be ``residual`` itself (updated in place).
    """
    fast = _fast or _quick()
    if fast and stream is None:
        r = fast.linear(x, w, s, bias, ACTIVATION_CODES.get(activation, -1), residual, y)
        if r is not None:
            return r
    import torch
    f16 = (torch.float16,)
    _tensor(x, "x", f16, any_offset=True)
    dev = x.device
    _tensor(w, "w_packed", _u32_dtypes(), dev, any_offset=True)
    _tensor(s, "scales", f16, dev, any_offset=True)
    M, K = x.shape
    N = w.shape[1]
    if K % GROUP_SIZE:
        raise ValueError(f"K ({K}) must be a multiple of group_size ({GROUP_SIZE})")
    if w.shape[0] != K // 8:
        raise ValueError(f"w_packed has {w.shape[0]} rows, expected K/8 = {K // 8} (K={K})")
    if tuple(s.shape) != (K // GROUP_SIZE, N):
        raise ValueError(f"scales must be [{K // GROUP_SIZE}, {N}], got {list(s.shape)}")
    if activation not in ACTIVATION_CODES:
        raise ValueError(f"unknown activation {activation!r}: one of {tuple(ACTIVATION_CODES)}")
    if bias is not None:
        _tensor(bias, "bias", f16, dev, rank=1, any_offset=True)
        if bias.shape[0] != N:
            raise ValueError(f"bias must be [{N}], got {list(bias.shape)}")
    if y is None:
        y = _allocate(dev, stream, lambda: torch.empty((M, N), dtype=torch.float16, device=dev))
    for t, n in ((residual, "residual"), (y, "y")):
        if t is not None:
            _tensor(t, n, f16, dev, any_offset=True)
            if tuple(t.shape) != (M, N):
                raise ValueError(f"{n} must be [{M}, {N}], got {list(t.shape)}")
    for dim in (M, N, K):
        if dim >= 2 ** 32:
            raise ValueError("dimension exceeds u32")
    _call(dev, lib().kaio_linear_w4a16, x.data_ptr(), w.data_ptr(), s.data_ptr(), None if bias is None else bias.data_ptr(),
          None if residual is None else residual.data_ptr(), y.data_ptr(), M, N, K, GROUP_SIZE,
          ACTIVATION_CODES[activation], _stream(dev, stream))
    return y


def _like(t, name, dtypes, device, shape):
    _tensor(t, name, dtypes, device, rank=len(shape), any_offset=True)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t


def _scratch(need, workspace, device, stream):
    """The workspace of a call that needs ``need`` bytes: the caller's, checked, or one of its own."""
    import torch
    if workspace is not None:
        return _tensor(workspace, "workspace", (torch.uint8,), device, rank=1, any_offset=True)
    return _allocate(device, stream, lambda: torch.empty((need,), dtype=torch.uint8, device=device)) if need else None


def _aligned(t, device, stream):
    """t, or a copy of it where it begins (a slice of a larger tensor) off the 16 bytes that the C library asks for."""
    return t if t is None or t.data_ptr() % 16 == 0 else _allocate(device, stream, t.clone)


def _ptr(t):
    return None if t is None else t.data_ptr()


def kaio_quantize_rows(x, q=None, scale=None, stream=None):
    """Rows rounded to 8 bits; returns (q int8[M, K], scale f32[M]).

    x f16 or bf16 [M, K], K a multiple of 16: scale = max |row| / 127, q = round(127 x / max |row|), ties to even.  A row
    with an infinity or a NaN has scale NaN and q 0.  ``scale`` may begin anywhere in a larger tensor (off 16 bytes the
    scales are copied there).
    """
    fast = _fast or _quick()
    if fast and stream is None:
        r = fast.quantize_rows(x, q, scale)
        if r is not None:
            return r
    import torch
    _tensor(x, "x", (torch.float16, torch.bfloat16), any_offset=True)
    dev = x.device
    M, K = x.shape
    if K % 16:
        raise ValueError(f"K ({K}) must be a multiple of 16")
    if q is None:
        q = _allocate(dev, stream, lambda: torch.empty((M, K), dtype=torch.int8, device=dev))
    if scale is None:
        scale = _allocate(dev, stream, lambda: torch.empty((M,), dtype=torch.float32, device=dev))
    _like(q, "q", (torch.int8,), dev, (M, K))
    _like(scale, "scale", (torch.float32,), dev, (M,))
    if max(M, K) >= 2 ** 32:
        raise ValueError("dimension exceeds u32")
    # scales of some rows of a larger tensor may begin anywhere: made elsewhere and copied
    made = scale
    if scale.data_ptr() % 16:
        begin, end = scale.data_ptr(), scale.data_ptr() + 4 * M
        if any(t.data_ptr() < end and begin < t.data_ptr() + t.numel() * t.element_size() for t in (x, q)):
            raise ValueError("output scale overlaps x or q")
        made = _allocate(dev, stream, lambda: torch.empty_like(scale))
    _call(dev, lib().kaio_quantize_rows, 2 if x.dtype == torch.float16 else 1, x.data_ptr(), q.data_ptr(), made.data_ptr(),
          M, K, _stream(dev, stream))
    if made is not scale:
        _allocate(dev, stream, lambda: scale.copy_(made))
    return q, scale


def kaio_linear_w8a8(x, w, w_scale, x_scale=None, bias=None, activation="none", residual=None, y=None, dtype=None,
                     workspace=None, stream=None):
    """y = act(x_scale * w_scale * (x . w^T) + bias) + residual, summed in integers, one rounding; returns y [M, N].

    w int8 [N, K] with w_scale f32 [N], K a multiple of 16.  x int8 [M, K] with x_scale f32 [M], or f16 or bf16 [M, K]
    without, then rounded here as by kaio_quantize_rows.  Scales and bias may begin anywhere in a larger tensor (off 16
    bytes they are copied first).  y, bias [N] and residual [M, N] are in x's dtype; for int8 x in
    ``dtype``, else the dtype of y, residual or bias, the first that is given, else f16.  ``y`` may be ``residual`` itself
    (updated in place).  ``workspace`` (uint8) is allocated here when it is needed and not given.
    """
    fast = _fast or _quick()
    if fast and stream is None and dtype is None:
        r = fast.linear8(x, w, w_scale, x_scale, bias, ACTIVATION_CODES.get(activation, -1), residual, y, workspace)
        if r is not None:
            return r
    import torch
    kinds = (torch.float16, torch.bfloat16)
    _tensor(x, "x", (torch.int8,) if x_scale is not None else kinds, any_offset=True)
    dev = x.device
    M, K = x.shape
    _tensor(w, "w", (torch.int8,), dev, any_offset=True)
    N = w.shape[0]
    if w.shape[1] != K:
        raise ValueError(f"K mismatch between inputs: x is [{M}, {K}], w is [{N}, {w.shape[1]}]")
    if K % 16:
        raise ValueError(f"K ({K}) must be a multiple of 16")
    _like(w_scale, "w_scale", (torch.float32,), dev, (N,))
    if x_scale is not None:
        _like(x_scale, "x_scale", (torch.float32,), dev, (M,))
        if dtype is None:
            dtype = next((t.dtype for t in (y, residual, bias) if isinstance(t, torch.Tensor)), torch.float16)
    elif dtype not in (None, x.dtype):
        raise TypeError(f"dtype must be x's, {x.dtype}, got {dtype}")
    else:
        dtype = x.dtype
    if dtype not in kinds:
        raise TypeError(f"dtype must be one of {kinds}, got {dtype}")
    if activation not in ACTIVATION_CODES:
        raise ValueError(f"unknown activation {activation!r}: one of {tuple(ACTIVATION_CODES)}")
    if bias is not None:
        _like(bias, "bias", (dtype,), dev, (N,))
    if residual is not None:
        _like(residual, "residual", (dtype,), dev, (M, N))
    if y is None:
        y = _allocate(dev, stream, lambda: torch.empty((M, N), dtype=dtype, device=dev))
    _like(y, "y", (dtype,), dev, (M, N))
    if max(M, N, K) >= 2 ** 32:
        raise ValueError("dimension exceeds u32")
    x_scale, w_scale, bias = (_aligned(t, dev, stream) for t in (x_scale, w_scale, bias))
    need = lib().kaio_linear_w8a8_workspace_size(M, N, K, int(x_scale is not None))
    workspace = _scratch(need, workspace, dev, stream)
    _call(dev, lib().kaio_linear_w8a8, 2 if dtype == torch.float16 else 1, x.data_ptr(), _ptr(x_scale), w.data_ptr(),
          w_scale.data_ptr(), _ptr(bias), _ptr(residual), y.data_ptr(), M, N, K, ACTIVATION_CODES[activation],
          _ptr(workspace), 0 if workspace is None else workspace.numel(), _stream(dev, stream))
    return y


class KaioExperts:
    """The weights of a mixture-of-experts feed-forward (kaio_experts of include/kaio.h).

    router          f16 [experts, hidden]
    w_gate, w_up    packed INT4 as int32/uint32 [experts, hidden/8, inner]; s_gate, s_up f16 [experts, hidden/128, inner]
    w_down          packed INT4 as int32/uint32 [experts, inner/8, hidden]; s_down f16 [experts, inner/128, hidden]

    Holds the tensors; made once and kept while they live, as only their addresses and shapes are taken here.
    """

    def __init__(self, router, w_gate, s_gate, w_up, s_up, w_down, s_down):
        import torch
        f16, u32 = (torch.float16,), _u32_dtypes()
        _tensor(router, "router", f16, any_offset=True)
        dev = router.device
        experts, hidden = router.shape
        _tensor(w_gate, "w_gate", u32, dev, rank=3, any_offset=True)
        inner = w_gate.shape[2]
        if hidden % GROUP_SIZE or inner % GROUP_SIZE or not (experts and hidden and inner):
            raise ValueError(f"hidden ({hidden}) and inner ({inner}) must be positive multiples of group_size "
                             f"({GROUP_SIZE}), and there must be experts")
        if max(experts, hidden, inner) >= 2 ** 31:
            raise ValueError("dimension exceeds i32")
        for t, name, k, n in ((w_gate, "gate", hidden, inner), (w_up, "up", hidden, inner), (w_down, "down", inner, hidden)):
            _like(t, "w_" + name, u32, dev, (experts, k // 8, n))
        for t, name, k, n in ((s_gate, "gate", hidden, inner), (s_up, "up", hidden, inner), (s_down, "down", inner, hidden)):
            _like(t, "s_" + name, f16, dev, (experts, k // GROUP_SIZE, n))
        self.router, self.w_gate, self.s_gate, self.w_up, self.s_up, self.w_down, self.s_down = \
            router, w_gate, s_gate, w_up, s_up, w_down, s_down
        self.device, self.experts, self.hidden, self.inner = dev, experts, hidden, inner
        self._c = _Experts(*[t.data_ptr() for t in (router, w_gate, s_gate, w_up, s_up, w_down, s_down)],
                           experts, hidden, inner, GROUP_SIZE)
        self._ref = ctypes.byref(self._c)
        self._addr = ctypes.addressof(self._c)
        self._index = dev.index


def kaio_moe_w4a16(x, experts, top_k, normalize=True, activation="silu", residual=None, y=None, workspace=None, stream=None):
    """A mixture-of-experts feed-forward for a few tokens; returns y f16 [T, hidden].

    x f16 [T, hidden]; each token goes to the ``top_k`` experts of largest <x, router row> (ties: the lowest index), with
    their softmax over all experts as weights, or over the chosen ones with ``normalize``:
    y = sum of weight * (act(x . gate) * (x . up)) . down, + residual.  ``y`` may be ``residual`` itself.  ``workspace``
    (uint8) is allocated here when not given.
    """
    if not isinstance(experts, KaioExperts):
        raise TypeError("experts must be a KaioExperts")
    fast = _fast or _quick()
    if fast and stream is None:
        r = fast.moe(x, experts._addr, experts._index, top_k, bool(normalize), ACTIVATION_CODES.get(activation, -1), residual,
                     y, workspace)
        if r is not None:
            return r
    import torch
    f16 = (torch.float16,)
    dev = experts.device
    _tensor(x, "x", f16, dev, any_offset=True)
    T = x.shape[0]
    _like(x, "x", f16, dev, (T, experts.hidden))
    if not 1 <= top_k <= experts.experts:
        raise ValueError(f"top_k ({top_k}) must be 1 to experts ({experts.experts})")
    if activation not in ACTIVATION_CODES:
        raise ValueError(f"unknown activation {activation!r}: one of {tuple(ACTIVATION_CODES)}")
    if residual is not None:
        _like(residual, "residual", f16, dev, x.shape)
    if y is None:
        y = _allocate(dev, stream, lambda: torch.empty_like(x))
    _like(y, "y", f16, dev, x.shape)
    if T >= 2 ** 32:
        raise ValueError("dimension exceeds u32")
    need = lib().kaio_moe_w4a16_workspace_size(experts._ref, T, top_k)
    workspace = _scratch(need, workspace, dev, stream)
    _call(dev, lib().kaio_moe_w4a16, experts._ref, x.data_ptr(), _ptr(residual), y.data_ptr(), T, top_k,
          int(bool(normalize)), ACTIVATION_CODES[activation], _ptr(workspace),
          0 if workspace is None else workspace.numel(), _stream(dev, stream))
    return y


class KaioPagedKV:
    """A paged key/value cache and the batch that uses it (kaio_paged_kv of include/kaio.h).

    k_cache, v_cache  f16 or bf16 [pages, page_size, kv_heads, head_dim]
    page_table        int32 [seqs, width]; an id outside [0, pages), -1 by custom, is a page that is not there
    q_start           int32 [seqs + 1], ascending: rows of q of each sequence's new tokens
    lens              int32 [seqs]: tokens of each sequence, the new ones last

    The host does not know the lengths, so ``width`` decides how attention shares out its work: short prompts and short
    caches are faster with a table not much wider than its sequences need (include/kaio.h has figures).

    Holds the tensors; made once and kept while they live, as only their addresses and shapes are taken here.
    What page_table, q_start and lens hold is read on the device by each call.
    """

    def __init__(self, k_cache, v_cache, page_table, q_start, lens):
        import torch
        _tensor(k_cache, "k_cache", (torch.float16, torch.bfloat16), rank=4, any_offset=True)
        dev = k_cache.device
        _tensor(v_cache, "v_cache", (k_cache.dtype,), dev, rank=4, any_offset=True)
        if v_cache.shape != k_cache.shape:
            raise ValueError(f"v_cache must be {list(k_cache.shape)}, got {list(v_cache.shape)}")
        if 0 in k_cache.shape[1:]:
            raise ValueError(f"page_size, kv_heads and head_dim must be at least 1, got caches of {list(k_cache.shape)}")
        i32 = (torch.int32,)
        _tensor(page_table, "page_table", i32, dev, any_offset=True)
        _tensor(q_start, "q_start", i32, dev, rank=1, any_offset=True)
        _tensor(lens, "lens", i32, dev, rank=1, any_offset=True)
        seqs = lens.shape[0]
        if page_table.shape[0] != seqs or q_start.shape[0] != seqs + 1:
            raise ValueError(f"page_table has {page_table.shape[0]} rows and q_start {q_start.shape[0]} entries, "
                             f"expected {seqs} and {seqs + 1}")
        if max(*k_cache.shape, seqs, page_table.shape[1]) >= 2 ** 31:
            raise ValueError("dimension exceeds i32")
        self.k_cache, self.v_cache, self.page_table, self.q_start, self.lens = k_cache, v_cache, page_table, q_start, lens
        self.device, self.dtype = dev, k_cache.dtype
        self.pages, self.page_size, self.kv_heads, self.head_dim = k_cache.shape
        self.seqs = seqs
        self._c = _PagedKV(k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), q_start.data_ptr(),
                           lens.data_ptr(), 2 if self.dtype == torch.float16 else 1, *k_cache.shape, seqs,
                           page_table.shape[1])
        self._ref = ctypes.byref(self._c)
        self._addr = ctypes.addressof(self._c)
        self._index = dev.index

    def _heads(self, t, name, heads=None):
        _tensor(t, name, (self.dtype,), self.device, rank=3, any_offset=True)
        if t.shape[2] != self.head_dim or (heads is not None and t.shape[1] != heads):
            raise ValueError(f"{name} must be [tokens, {'heads' if heads is None else heads}, {self.head_dim}], "
                             f"got {list(t.shape)}")
        return t


def _paged(paged):
    if not isinstance(paged, KaioPagedKV):
        raise TypeError("paged must be a KaioPagedKV")
    return paged


def kaio_rope_append(q, k, v, positions, inv_freq, sections, paged, interleaved=False, q_out=None, stream=None):
    """Rotary positions on q and k, k and v written to the paged cache; returns the turned q.

    q [T, q_heads, head_dim], k and v [T, kv_heads, head_dim] in the cache's dtype; positions int32 [axes, T];
    inv_freq float64 [pairs]; sections: how many consecutive pairs each axis turns (their sum is ``pairs``;
    elements past 2 * pairs of a head pass through).  Pair j is elements (2j, 2j+1) when ``interleaved``, else
    (j, j + pairs).  ``q_out`` may be ``q`` itself (turned in place).
    """
    p = _paged(paged)
    fast = _fast or _quick()
    if fast and stream is None:
        r = fast.rope_append(q, k, v, positions, inv_freq, sections, p._addr, p._index, bool(interleaved), q_out)
        if r is not None:
            return r
    import torch
    p._heads(q, "q")
    T = q.shape[0]
    p._heads(k, "k", p.kv_heads)
    p._heads(v, "v", p.kv_heads)
    if k.shape[0] != T or v.shape[0] != T:
        raise ValueError(f"k and v must have q's {T} rows, got {k.shape[0]} and {v.shape[0]}")
    _tensor(positions, "positions", (torch.int32,), p.device, any_offset=True)
    _tensor(inv_freq, "inv_freq", (torch.float64,), p.device, rank=1, any_offset=True)
    axes = len(sections)
    if tuple(positions.shape) != (axes, T):
        raise ValueError(f"positions must be [{axes}, {T}], got {list(positions.shape)}")
    if min(sections, default=0) < 0 or sum(sections) != inv_freq.shape[0]:
        raise ValueError(f"sections {list(sections)} must be counts that add up to the {inv_freq.shape[0]} pairs of inv_freq")
    if q_out is None:
        q_out = _allocate(p.device, stream, lambda: torch.empty_like(q))
    p._heads(q_out, "q_out")
    if q_out.shape != q.shape:
        raise ValueError(f"q_out must be {list(q.shape)}, got {list(q_out.shape)}")
    if T >= 2 ** 31 or q.shape[1] >= 2 ** 31:
        raise ValueError("dimension exceeds i32")
    _call(p.device, lib().kaio_rope_append, p._ref, q.data_ptr(), k.data_ptr(), v.data_ptr(), positions.data_ptr(),
          inv_freq.data_ptr(), (ctypes.c_uint32 * axes)(*sections), axes, int(bool(interleaved)), q_out.data_ptr(), T,
          q.shape[1], _stream(p.device, stream))
    return q_out


def kaio_paged_attention(q, paged, max_new, scale, window=0, sinks=0, out=None, workspace=None, stream=None):
    """Causal attention of the new tokens over the paged cache; returns out, shaped as q.

    q [T, q_heads, head_dim] in the cache's dtype, q_heads a multiple of the cache's heads; ``max_new``: the most
    new tokens a sequence has (it chooses the kernel).  With ``window`` > 0 a row at position p sees positions
    above p - window and the first ``sinks``.  A row that sees nothing is zero.  ``workspace`` (uint8) is
    allocated here when it is needed and not given.
    """
    p = _paged(paged)
    fast = _fast or _quick()
    if fast and stream is None:
        r = fast.attention(q, p._addr, p._index, max_new, scale, window, sinks, out, workspace)
        if r is not None:
            return r
    import torch
    p._heads(q, "q")
    T, hq, _ = q.shape
    if hq % p.kv_heads:
        raise ValueError(f"q has {hq} heads, not a multiple of the cache's {p.kv_heads}")
    if out is None:
        out = _allocate(p.device, stream, lambda: torch.empty_like(q))
    p._heads(out, "out")
    if out.shape != q.shape:
        raise ValueError(f"out must be {list(q.shape)}, got {list(out.shape)}")
    if max_new < 0 or window < 0 or sinks < 0 or max(T, hq, max_new, window, sinks) >= 2 ** 31:
        raise ValueError("max_new, window and sinks must be counts that fit in i32")
    need = lib().kaio_paged_attention_workspace_size(p._ref, T, hq, max_new)
    if workspace is None and need:
        workspace = _allocate(p.device, stream, lambda: torch.empty((need,), dtype=torch.uint8, device=p.device))
    if workspace is not None:
        _tensor(workspace, "workspace", (torch.uint8,), p.device, rank=1, any_offset=True)
    _call(p.device, lib().kaio_paged_attention, p._ref, q.data_ptr(), out.data_ptr(), T, hq, max_new, scale, window, sinks,
          None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.numel(),
          _stream(p.device, stream))
    return out
