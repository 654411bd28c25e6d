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
    KaioPagedKV(k_cache, v_cache, page_table, q_start, lens): a paged cache and its batch, for
    kaio_rope_append(q, k, v, positions, inv_freq, sections, paged) -> q
    kaio_paged_attention(q, paged, max_new, scale, window=, sinks=) -> out
"""
from __future__ import annotations

import ctypes
import os

__all__ = ["DTYPE_CODES", "KaioError", "kaio_qkv_w4a16", "kaio_qkv_w8a16", "kaio_gemm_f16f32", "kaio_gemm_f16f32_bwd",
           "kaio_dequant_group_bwd", "kaio_linear_w4a16", "KaioPagedKV", "kaio_rope_append", "kaio_paged_attention",
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
                L.kaio_linear_w4a16, L.kaio_rope_append, L.kaio_paged_attention, L.kaio_paged_attention_workspace_size)])
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
    _check(fn(x.data_ptr(), *[t.data_ptr() for t in ws], *[t.data_ptr() for t in ss],
              *[t.data_ptr() for t in outs], M, N, K, GROUP_SIZE, _stream(dev, stream)))
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
    _check(lib().kaio_gemm_f16f32(a.data_ptr(), b.data_ptr(), c.data_ptr(), M, N, K, _stream(a.device, stream)))
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
    _check(lib().kaio_gemm_f16f32_bwd(a.data_ptr(), b.data_ptr(), grad.data_ptr(), grad_a.data_ptr(),
                                      grad_b.data_ptr(), M, N, K, workspace.data_ptr(), workspace.numel(),
                                      _stream(a.device, stream)))
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
    _check(lib().kaio_dequant_group_bwd(codes[dy.dtype], outer, axis, group_size, dy.data_ptr(),
                                        scale.data_ptr(), dq.data_ptr(), None, 0, _stream(dy.device, stream)))
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
    _check(lib().kaio_linear_w4a16(x.data_ptr(), w.data_ptr(), s.data_ptr(),
                                   None if bias is None else bias.data_ptr(),
                                   None if residual is None else residual.data_ptr(), y.data_ptr(),
                                   M, N, K, GROUP_SIZE, ACTIVATION_CODES[activation], _stream(dev, stream)))
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
    _check(lib().kaio_rope_append(p._ref, q.data_ptr(), k.data_ptr(), v.data_ptr(), positions.data_ptr(),
                                  inv_freq.data_ptr(), (ctypes.c_uint32 * axes)(*sections), axes, int(bool(interleaved)),
                                  q_out.data_ptr(), T, q.shape[1], _stream(p.device, stream)))
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
    _check(lib().kaio_paged_attention(p._ref, q.data_ptr(), out.data_ptr(), T, hq, max_new, scale, window, sinks,
                                      None if workspace is None else workspace.data_ptr(),
                                      0 if workspace is None else workspace.numel(), _stream(p.device, stream)))
    return out
