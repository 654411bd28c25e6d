// C ABI entry points: host-side validation, device check, dispatch.
// Every check here runs before any HIP call, so argument errors are reported
// the same way with or without a GPU.

#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <string>

#include "launch.hpp"

static_assert(kaio::kGemmBwdScratchBytes == KAIO_GEMM_BWD_NOALLOC_MAX_BYTES,
              "the header's limit must match the static buffer");

namespace {

thread_local std::string g_last_error;

kaio_status fail(kaio_status st, const char* op, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = std::string("kaio::") + op + ": " + buf;
  return st;
}

kaio_status ok() {
  g_last_error.clear();
  return KAIO_OK;
}

// a*b*c as bytes, false when it does not fit comfortably in the address space
bool bytes_of(uint64_t a, uint64_t b, uint64_t c, uint64_t* out) {
  unsigned __int128 v = (unsigned __int128)a * b * c;
  if (v >= ((unsigned __int128)1 << 62)) return false;
  *out = (uint64_t)v;
  return true;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
  const char* name;
};

// first pair (output, other) whose byte ranges intersect; empty ranges never do
const Range* overlap(const Range* outs, int nouts, const Range* ins, int nins, const Range** other) {
  for (int i = 0; i < nouts; ++i) {
    if (outs[i].lo == outs[i].hi) continue;
    for (int j = 0; j < nins; ++j) {
      if (ins[j].lo == ins[j].hi) continue;
      if (outs[i].lo < ins[j].hi && ins[j].lo < outs[i].hi) { *other = &ins[j]; return &outs[i]; }
    }
    for (int j = i + 1; j < nouts; ++j) {
      if (outs[j].lo == outs[j].hi) continue;
      if (outs[i].lo < outs[j].hi && outs[j].lo < outs[i].hi) { *other = &outs[j]; return &outs[i]; }
    }
  }
  return nullptr;
}

Range range(const void* p, uint64_t bytes, const char* name) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{lo, lo + (uintptr_t)bytes, name};
}

// Device check, cached per device ordinal: the current device must be gfx950.
constexpr int kMaxDevices = 64;
std::atomic<int> g_device_state[kMaxDevices];  // 0 unknown, 1 ok, 2 bad

kaio_status check_device(const char* op) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess || dev < 0)
    return fail(KAIO_ERR_DEVICE, op, "no HIP device available (%s); there is no CPU fallback",
                hipGetErrorString(e));
  if (dev >= kMaxDevices) return fail(KAIO_ERR_DEVICE, op, "device ordinal %d out of range", dev);
  int st = g_device_state[dev].load(std::memory_order_acquire);
  if (st == 0) {
    hipDeviceProp_t prop;
    e = hipGetDeviceProperties(&prop, dev);
    if (e != hipSuccess)
      return fail(KAIO_ERR_DEVICE, op, "hipGetDeviceProperties failed: %s", hipGetErrorString(e));
    st = (std::strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? 1 : 2;
    g_device_state[dev].store(st, std::memory_order_release);
  }
  if (st != 1) {
    hipDeviceProp_t prop;
    const char* arch = (hipGetDeviceProperties(&prop, dev) == hipSuccess) ? prop.gcnArchName : "?";
    return fail(KAIO_ERR_DEVICE, op, "device %d is %s; this library is built for gfx950 (MI355X) only",
                dev, arch);
  }
  return KAIO_OK;
}

kaio_status launched(const char* op, hipError_t e) {
  if (e != hipSuccess) return fail(KAIO_ERR_LAUNCH, op, "launch failed: %s", hipGetErrorString(e));
  return ok();
}

// kaio_gemm_f16f32_bwd and its allocation-free variant (noalloc: f16(grad) goes
// to the library's static per-device buffer instead of the caller's workspace).
kaio_status gemm_bwd(const char* op, const void* a, const void* b, const float* grad, void* grad_a,
                     void* grad_b, uint32_t m, uint32_t n, uint32_t k, bool noalloc, void* workspace,
                     size_t workspace_bytes, void* stream) {
  uint64_t a_bytes = 0, b_bytes = 0, g_bytes = 0, g16_bytes = 0;
  const uint64_t wgs_a = (uint64_t)((m + kaio::kGemmBM - 1) / kaio::kGemmBM) *
                         ((k + kaio::kGemmBN - 1) / kaio::kGemmBN);
  const uint64_t wgs_b = (uint64_t)((k + kaio::kGemmBM - 1) / kaio::kGemmBM) *
                         ((n + kaio::kGemmBN - 1) / kaio::kGemmBN);
  if (!bytes_of(m, k, 2, &a_bytes) || !bytes_of(k, n, 2, &b_bytes) || !bytes_of(m, n, 4, &g_bytes) ||
      !bytes_of(m, n, 2, &g16_bytes) || wgs_a > kaio::kMaxWorkgroups || wgs_b > kaio::kMaxWorkgroups)
    return fail(KAIO_ERR_INVALID_PROBLEM, op, "problem too large for one launch (m=%u, n=%u, k=%u)", m, n, k);
  if (noalloc && g16_bytes > kaio::kGemmBwdScratchBytes)
    return fail(KAIO_ERR_UNSUPPORTED, op,
                "f16(grad) needs m*n*2 = %llu bytes, more than the static buffer of %llu bytes "
                "(use kaio_gemm_f16f32_bwd with a workspace)",
                (unsigned long long)g16_bytes, (unsigned long long)kaio::kGemmBwdScratchBytes);
  if (k == 0) return ok();
  if (m > 0 && !grad_a) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "output grad_a is null");
  if (n > 0 && !grad_b) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "output grad_b is null");
  const bool empty = m == 0 || n == 0;   // both gradients are the empty sum
  if (!empty) {
    if (!a) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "input a is null");
    if (!b) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "input b is null");
    if (!grad) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "input grad is null");
    if (!noalloc && !workspace) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "workspace is null");
    if (!noalloc && workspace_bytes < g16_bytes)
      return fail(KAIO_ERR_INVALID_ARGUMENT, op, "workspace_bytes (%zu) < %llu needed", workspace_bytes,
                  (unsigned long long)g16_bytes);
  }
  if (m > 0 && !aligned16(grad_a)) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "output grad_a is not 16-byte aligned");
  if (n > 0 && !aligned16(grad_b)) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "output grad_b is not 16-byte aligned");
  if (!empty) {
    if (!aligned16(a)) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "input a is not 16-byte aligned");
    if (!aligned16(b)) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "input b is not 16-byte aligned");
    if (!aligned16(grad)) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "input grad is not 16-byte aligned");
    if (!noalloc && !aligned16(workspace)) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "workspace is not 16-byte aligned");
  }
  // written: grad_a, grad_b, and (when not empty) the workspace
  const Range ro[3] = {range(grad_a, a_bytes, "grad_a"), range(grad_b, b_bytes, "grad_b"),
                       range(empty || noalloc ? nullptr : workspace, empty || noalloc ? 0 : g16_bytes,
                             "workspace")};
  const Range ri[3] = {range(empty ? nullptr : a, empty ? 0 : a_bytes, "a"),
                       range(empty ? nullptr : b, empty ? 0 : b_bytes, "b"),
                       range(empty ? nullptr : grad, empty ? 0 : g_bytes, "grad")};
  const Range* other = nullptr;
  if (const Range* o = overlap(ro, 3, ri, 3, &other))
    return fail(KAIO_ERR_INVALID_ARGUMENT, op, "%s overlaps %s", o->name, other->name);
  if (kaio_status st = check_device(op)) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (empty) {
    if (m > 0)
      if (hipError_t e = kaio::launch_fill_zero(grad_a, a_bytes, s)) return launched(op, e);
    if (n > 0)
      if (hipError_t e = kaio::launch_fill_zero(grad_b, b_bytes, s)) return launched(op, e);
    return launched(op, hipSuccess);
  }
  if (noalloc)
    return launched(op, kaio::launch_gemm_f16f32_bwd_noalloc(
                            static_cast<const uint16_t*>(a), static_cast<const uint16_t*>(b), grad,
                            static_cast<uint16_t*>(grad_a), static_cast<uint16_t*>(grad_b), m, n, k, s));
  return launched(op, kaio::launch_gemm_f16f32_bwd(
                          static_cast<const uint16_t*>(a), static_cast<const uint16_t*>(b), grad,
                          static_cast<uint16_t*>(grad_a), static_cast<uint16_t*>(grad_b),
                          static_cast<uint16_t*>(workspace), m, n, k, s));
}

// kaio_qkv_w4a16 (bits 4: u32[k/8, n] weights) and kaio_qkv_w8a16 (bits 8:
// u32[k/4, n] weights): the same validation, the same kernels templated on
// the weight width.
kaio_status qkv(const char* op, uint32_t bits, const void* x, const uint32_t* w_q, const uint32_t* w_k,
                const uint32_t* w_v, const void* s_q, const void* s_k, const void* s_v, void* q, void* k_out,
                void* v, uint32_t m, uint32_t n, uint32_t k, uint32_t group_size, void* stream) {
  if (group_size != 128)
    return fail(KAIO_ERR_UNSUPPORTED, op, "group_size (%u) must be 128 (locked by the kernel contract)",
                group_size);
  if (k % 128 != 0)
    return fail(KAIO_ERR_INVALID_PROBLEM, op, "K (%u) must be a multiple of group_size (128)", k);
  if (m == 0 || n == 0) return ok();

  uint64_t out_bytes = 0, x_bytes = 0, w_bytes = 0, s_bytes = 0;
  const bool decode = kaio::qkv_split_k(m, k, bits);
  const uint64_t wgs = decode ? 3ull * ((n + kaio::decode_bn(m) - 1) / kaio::decode_bn(m))
                              : kaio::prefill_wgs(kaio::tile_form(m, n, k, bits), m, n);
  if (!bytes_of(m, n, 2, &out_bytes) || !bytes_of(m, k, 2, &x_bytes) || !bytes_of(k / (32 / bits), n, 4, &w_bytes) ||
      !bytes_of(k / 128, n, 2, &s_bytes) || wgs > kaio::kMaxWorkgroups || n >= kaio::kMaxN ||
      k >= kaio::kMaxK)
    return fail(KAIO_ERR_INVALID_PROBLEM, op, "problem too large for one launch (m=%u, n=%u, k=%u)", m, n, k);

  const void* ins[7] = {x, w_q, w_k, w_v, s_q, s_k, s_v};
  static const char* in_names[7] = {"x", "w_q_packed", "w_k_packed", "w_v_packed",
                                    "scales_q", "scales_k", "scales_v"};
  void* outs[3] = {q, k_out, v};
  static const char* out_names[3] = {"q", "k", "v"};
  for (int i = 0; i < 3; ++i)
    if (!outs[i]) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "output %s is null", out_names[i]);
  if (k > 0)
    for (int i = 0; i < 7; ++i)
      if (!ins[i]) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "input %s is null", in_names[i]);
  for (int i = 0; i < 3; ++i)
    if (!aligned16(outs[i]))
      return fail(KAIO_ERR_INVALID_ARGUMENT, op, "output %s is not 16-byte aligned", out_names[i]);
  if (k > 0)
    for (int i = 0; i < 7; ++i)
      if (!aligned16(ins[i]))
        return fail(KAIO_ERR_INVALID_ARGUMENT, op, "input %s is not 16-byte aligned", in_names[i]);

  const Range ro[3] = {range(q, out_bytes, "q"), range(k_out, out_bytes, "k"), range(v, out_bytes, "v")};
  const Range ri[7] = {range(x, x_bytes, "x"),           range(w_q, w_bytes, "w_q_packed"),
                       range(w_k, w_bytes, "w_k_packed"), range(w_v, w_bytes, "w_v_packed"),
                       range(s_q, s_bytes, "scales_q"),   range(s_k, s_bytes, "scales_k"),
                       range(s_v, s_bytes, "scales_v")};
  const Range* other = nullptr;
  if (const Range* o = overlap(ro, 3, ri, 7, &other))
    return fail(KAIO_ERR_INVALID_ARGUMENT, op, "output %s overlaps %s", o->name, other->name);

  if (kaio_status st = check_device(op)) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();  // start from a clean error state
  if (k == 0) {
    for (int i = 0; i < 3; ++i)
      if (hipError_t e = kaio::launch_fill_zero(outs[i], out_bytes, s)) return launched(op, e);
    return ok();
  }
  kaio::QkvProblem p;
  p.x = static_cast<const uint16_t*>(x);
  p.w[0] = w_q; p.w[1] = w_k; p.w[2] = w_v;
  p.s[0] = static_cast<const uint16_t*>(s_q);
  p.s[1] = static_cast<const uint16_t*>(s_k);
  p.s[2] = static_cast<const uint16_t*>(s_v);
  p.out[0] = static_cast<uint16_t*>(q);
  p.out[1] = static_cast<uint16_t*>(k_out);
  p.out[2] = static_cast<uint16_t*>(v);
  p.m = m; p.n = n; p.k = k;
  p.bits = bits;
  return launched(op, decode ? kaio::launch_qkv_decode(p, s) : kaio::launch_qkv_prefill(p, s));
}

bool aligned_to(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// an enum parameter's code, read from its bytes (a C caller may pass any int)
template <typename E>
int code_of(const E& e) {
  static_assert(sizeof(E) == sizeof(int), "enums are passed as ints");
  int code = 0;
  std::memcpy(&code, &e, sizeof code);
  return code;
}

// The checks of a paged cache that need no pointers: dtype and sizes.
kaio_status check_paged_sizes(const char* op, const kaio_paged_kv* kv) {
  if (!kv) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "kv is null");
  if (kv->dtype != KAIO_DTYPE_F16 && kv->dtype != KAIO_DTYPE_BF16)
    return fail(KAIO_ERR_UNSUPPORTED, op, "unsupported dtype %d (f16, bf16)", kv->dtype);
  if (kv->page_size == 0 || kv->kv_heads == 0 || kv->head_dim == 0)
    return fail(KAIO_ERR_INVALID_PROBLEM, op, "page_size (%u), kv_heads (%u) and head_dim (%u) must be > 0",
                kv->page_size, kv->kv_heads, kv->head_dim);
  return KAIO_OK;
}

bool paged_fits(const kaio_paged_kv* kv, uint64_t* cache_bytes, uint64_t* table_bytes) {
  const uint64_t slots = (uint64_t)kv->pages * kv->page_size;
  return slots < (1ull << 31) && (uint64_t)kv->kv_heads * kv->head_dim < (1ull << 31) &&
         bytes_of(slots, (uint64_t)kv->kv_heads * kv->head_dim, 2, cache_bytes) &&
         bytes_of(kv->seqs, kv->table_width, 4, table_bytes) && kv->seqs < (1u << 31);
}

kaio_status check_paged_pointers(const char* op, const kaio_paged_kv* kv) {
  const bool cache = kv->pages > 0, table = kv->seqs > 0 && kv->table_width > 0;
  const struct { const void* p; const char* name; bool used; uintptr_t align; } all[5] = {
      {kv->k_cache, "k_cache", cache, 16}, {kv->v_cache, "v_cache", cache, 16},
      {kv->page_table, "page_table", table, 4}, {kv->q_start, "q_start", kv->seqs > 0, 4},
      {kv->lens, "lens", kv->seqs > 0, 4}};
  for (const auto& a : all)
    if (a.used && !a.p) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "%s is null", a.name);
  for (const auto& a : all)
    if (a.used && !aligned_to(a.p, a.align))
      return fail(KAIO_ERR_INVALID_ARGUMENT, op, "%s is not %u-byte aligned", a.name, (unsigned)a.align);
  return KAIO_OK;
}

kaio::PagedKV paged_of(const kaio_paged_kv* kv, uint32_t tokens) {
  kaio::PagedKV p;
  p.k = static_cast<uint16_t*>(kv->k_cache);
  p.v = static_cast<uint16_t*>(kv->v_cache);
  p.table = kv->page_table;
  p.q_start = kv->q_start;
  p.lens = kv->lens;
  p.pages = kv->pages;
  p.kv_heads = kv->kv_heads;
  p.head_dim = kv->head_dim;
  p.seqs = kv->seqs;
  p.width = kv->table_width;
  const uint64_t cap = (uint64_t)kv->table_width * kv->page_size;
  p.cap = cap < 0x7FFFFFFFull ? (uint32_t)cap : 0x7FFFFFFFu;
  p.page = kaio::FastDiv::of(kv->page_size);
  p.tokens = tokens;
  return p;
}

kaio::AttentionPlan attention_plan_of(const kaio_paged_kv* kv, uint32_t tokens, uint32_t q_heads, uint32_t max_new,
                                      uint32_t window = 0, uint32_t sinks = 0) {
  return kaio::attention_plan(kv->kv_heads, q_heads, kv->head_dim, kv->seqs,
                              (uint64_t)kv->table_width * kv->page_size, tokens, max_new, window, sinks);
}

}  // namespace

extern "C" {

kaio_status kaio_qkv_w4a16(const void* x, const uint32_t* w_q, const uint32_t* w_k, const uint32_t* w_v,
                           const void* s_q, const void* s_k, const void* s_v, void* q, void* k_out,
                           void* v, uint32_t m, uint32_t n, uint32_t k, uint32_t group_size,
                           void* stream) {
  return qkv("qkv_w4a16", 4, x, w_q, w_k, w_v, s_q, s_k, s_v, q, k_out, v, m, n, k, group_size, stream);
}

kaio_status kaio_qkv_w8a16(const void* x, const uint32_t* w_q, const uint32_t* w_k, const uint32_t* w_v,
                           const void* s_q, const void* s_k, const void* s_v, void* q, void* k_out,
                           void* v, uint32_t m, uint32_t n, uint32_t k, uint32_t group_size,
                           void* stream) {
  return qkv("qkv_w8a16", 8, x, w_q, w_k, w_v, s_q, s_k, s_v, q, k_out, v, m, n, k, group_size, stream);
}

kaio_status kaio_gemm_f16f32(const void* a, const void* b, float* c, uint32_t m, uint32_t n, uint32_t k,
                             void* stream) {
  static const char* op = "gemm_f16f32";
  if (m == 0 || n == 0) return ok();
  uint64_t c_bytes = 0, a_bytes = 0, b_bytes = 0;
  const uint64_t wgs = (uint64_t)((m + kaio::kGemmBM - 1) / kaio::kGemmBM) *
                       ((n + kaio::kGemmBN - 1) / kaio::kGemmBN);
  if (!bytes_of(m, n, 4, &c_bytes) || !bytes_of(m, k, 2, &a_bytes) || !bytes_of(k, n, 2, &b_bytes) ||
      wgs > kaio::kMaxWorkgroups)
    return fail(KAIO_ERR_INVALID_PROBLEM, op, "problem too large for one launch (m=%u, n=%u, k=%u)", m, n, k);
  if (!c) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "output c is null");
  if (k > 0 && !a) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "input a is null");
  if (k > 0 && !b) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "input b is null");
  if (!aligned16(c)) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "output c is not 16-byte aligned");
  if (k > 0 && !aligned16(a)) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "input a is not 16-byte aligned");
  if (k > 0 && !aligned16(b)) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "input b is not 16-byte aligned");
  const Range ro[1] = {range(c, c_bytes, "c")};
  const Range ri[2] = {range(a, a_bytes, "a"), range(b, b_bytes, "b")};
  const Range* other = nullptr;
  if (const Range* o = overlap(ro, 1, ri, 2, &other))
    return fail(KAIO_ERR_INVALID_ARGUMENT, op, "output %s overlaps %s", o->name, other->name);
  if (kaio_status st = check_device(op)) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (k == 0) return launched(op, kaio::launch_fill_zero(c, c_bytes, s));
  return launched(op, kaio::launch_gemm_f16f32(static_cast<const uint16_t*>(a),
                                               static_cast<const uint16_t*>(b), c, m, n, k, s));
}

size_t kaio_gemm_f16f32_bwd_workspace_size(uint32_t m, uint32_t n) { return (size_t)m * n * 2; }

kaio_status kaio_gemm_f16f32_bwd(const void* a, const void* b, const float* grad, void* grad_a, void* grad_b,
                                 uint32_t m, uint32_t n, uint32_t k, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  return gemm_bwd("gemm_f16f32_bwd", a, b, grad, grad_a, grad_b, m, n, k, false, workspace, workspace_bytes,
                  stream);
}

kaio_status kaio_gemm_f16f32_bwd_noalloc(const void* a, const void* b, const float* grad, void* grad_a,
                                         void* grad_b, uint32_t m, uint32_t n, uint32_t k, void* stream) {
  return gemm_bwd("gemm_f16f32_bwd_noalloc", a, b, grad, grad_a, grad_b, m, n, k, true, nullptr, 0, stream);
}

kaio_status kaio_dequant_group_bwd(kaio_dtype dtype, int32_t outer, int32_t axis, int32_t group_size,
                                   const void* dy, const void* scale, void* dq, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  static const char* op = "dequant_group_bwd";
  (void)workspace;
  (void)workspace_bytes;
  // A C caller may pass any int here.  In C++ reading an enum object that holds a value
  // outside the enumeration's range is undefined, so the code is taken from the
  // parameter's bytes and only a validated code is turned back into a kaio_dtype.
  static_assert(sizeof(kaio_dtype) == sizeof(int), "kaio_dtype is passed as an int");
  int code = 0;
  std::memcpy(&code, &dtype, sizeof code);
  size_t esz = 0;
  switch (code) {
    case KAIO_DTYPE_F32: esz = 4; break;
    case KAIO_DTYPE_BF16: esz = 2; break;
    case KAIO_DTYPE_F16: esz = 2; break;
    case KAIO_DTYPE_F64: esz = 8; break;
    default:
      return fail(KAIO_ERR_UNSUPPORTED, op, "unsupported dtype %d (f32, bf16, f16, f64)", code);
  }
  const kaio_dtype dt = static_cast<kaio_dtype>(code);
  if (outer < 0 || axis < 0)
    return fail(KAIO_ERR_INVALID_PROBLEM, op, "outer_size (%d) and axis_size (%d) must be non-negative",
                outer, axis);
  if (group_size <= 0) return fail(KAIO_ERR_INVALID_PROBLEM, op, "group_size (%d) must be > 0", group_size);
  if (axis % group_size != 0)
    return fail(KAIO_ERR_INVALID_PROBLEM, op, "axis_size (%d) must be a multiple of group_size (%d)", axis,
                group_size);
  const uint64_t total = (uint64_t)outer * (uint64_t)axis;
  if (total == 0) return ok();
  uint64_t bytes = 0;
  if (!bytes_of(outer, axis, esz, &bytes))
    return fail(KAIO_ERR_INVALID_PROBLEM, op, "problem too large (outer=%d, axis=%d)", outer, axis);
  if (!dy) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "d_output is null");
  if (!scale) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "scale is null");
  if (!dq) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "d_input is null");
  const void* ptrs[3] = {dy, scale, dq};
  static const char* names[3] = {"d_output", "scale", "d_input"};
  for (int i = 0; i < 3; ++i)
    if (reinterpret_cast<uintptr_t>(ptrs[i]) % esz != 0)
      return fail(KAIO_ERR_INVALID_ARGUMENT, op, "%s is not aligned to its element size (%zu)", names[i], esz);
  const Range ro[1] = {range(dq, bytes, "d_input")};
  const Range ri[2] = {range(dy, bytes, "d_output"),
                       range(scale, (uint64_t)outer * (uint64_t)(axis / group_size) * esz, "scale")};
  const Range* other = nullptr;
  if (const Range* o = overlap(ro, 1, ri, 2, &other))
    return fail(KAIO_ERR_INVALID_ARGUMENT, op, "output %s overlaps %s", o->name, other->name);
  if (kaio_status st = check_device(op)) return st;
  (void)hipGetLastError();
  return launched(op, kaio::launch_dequant_group_bwd(dt, outer, axis, group_size, dy, scale, dq,
                                                     static_cast<hipStream_t>(stream)));
}

kaio_status kaio_qkv_plan(uint32_t m, uint32_t n, uint32_t k, uint32_t bits, uint32_t plan[5]) {
  static const char* op = "qkv_plan";
  if (bits != 4 && bits != 8) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "bits (%u) must be 4 or 8", bits);
  if (!plan) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "plan is null");
  if (k % 128 != 0)
    return fail(KAIO_ERR_INVALID_PROBLEM, op, "K (%u) must be a multiple of group_size (128)", k);
  for (int i = 0; i < 5; ++i) plan[i] = 0;
  if (m == 0 || n == 0) return ok();
  if (kaio::qkv_split_k(m, k, bits)) {
    const uint32_t bn = kaio::decode_bn(m);
    plan[2] = bn;
    plan[3] = 1;
    plan[4] = (uint32_t)(3ull * ((n + bn - 1) / bn));
  } else {
    const kaio::PrefillForm f = kaio::tile_form(m, n, k, bits);
    plan[0] = f.outs == 1 ? 2 : 1;
    plan[1] = f.waves;
    plan[2] = f.bm;
    plan[3] = f.sets;
    const uint64_t wgs = kaio::prefill_wgs(f, m, n);
    plan[4] = wgs > 0xFFFFFFFFull ? 0xFFFFFFFFu : (uint32_t)wgs;
  }
  return ok();
}

kaio_status kaio_linear_w4a16(const void* x, const uint32_t* w, const void* s, const void* bias,
                              const void* residual, void* y, uint32_t m, uint32_t n, uint32_t k,
                              uint32_t group_size, kaio_activation activation, void* stream) {
  static const char* op = "linear_w4a16";
  if (group_size != 128)
    return fail(KAIO_ERR_UNSUPPORTED, op, "group_size (%u) must be 128 (locked by the kernel contract)", group_size);
  const int act = code_of(activation);
  if (act < KAIO_ACT_NONE || act > KAIO_ACT_SILU) return fail(KAIO_ERR_UNSUPPORTED, op, "unknown activation %d", act);
  if (k % 128 != 0)
    return fail(KAIO_ERR_INVALID_PROBLEM, op, "K (%u) must be a multiple of group_size (128)", k);
  if (m == 0 || n == 0) return ok();
  uint64_t out_bytes = 0, x_bytes = 0, w_bytes = 0, s_bytes = 0;
  const uint64_t wgs = kaio::linear_wgs(m, n);
  if (!bytes_of(m, n, 2, &out_bytes) || !bytes_of(m, k, 2, &x_bytes) || !bytes_of(k / 8, n, 4, &w_bytes) ||
      !bytes_of(k / 128, n, 2, &s_bytes) || wgs > kaio::kMaxWorkgroups || n >= kaio::kMaxN || k >= kaio::kMaxK)
    return fail(KAIO_ERR_INVALID_PROBLEM, op, "problem too large for one launch (m=%u, n=%u, k=%u)", m, n, k);
  if (!y) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "output y is null");
  const struct { const void* p; const char* name; } ins[5] = {
      {x, "x"}, {w, "w_packed"}, {s, "scales"}, {bias, "bias"}, {residual, "residual"}};
  if (k > 0)
    for (int i = 0; i < 3; ++i)
      if (!ins[i].p) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "input %s is null", ins[i].name);
  if (!aligned16(y)) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "output y is not 16-byte aligned");
  for (int i = k > 0 ? 0 : 3; i < 5; ++i)
    if (!aligned16(ins[i].p)) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "input %s is not 16-byte aligned", ins[i].name);
  const Range ro[1] = {range(y, out_bytes, "y")};
  const Range ri[5] = {range(x, k > 0 ? x_bytes : 0, "x"), range(w, w_bytes, "w_packed"), range(s, s_bytes, "scales"),
                       range(bias, bias ? (uint64_t)n * 2 : 0, "bias"),
                       range(residual, residual && residual != y ? out_bytes : 0, "residual")};
  const Range* other = nullptr;
  if (const Range* o = overlap(ro, 1, ri, 5, &other))
    return fail(KAIO_ERR_INVALID_ARGUMENT, op, "output %s overlaps %s", o->name, other->name);
  if (kaio_status st = check_device(op)) return st;
  (void)hipGetLastError();
  kaio::LinearProblem p;
  p.x = static_cast<const uint16_t*>(x);
  p.w = w;
  p.s = static_cast<const uint16_t*>(s);
  p.bias = static_cast<const uint16_t*>(bias);
  p.residual = static_cast<const uint16_t*>(residual);
  p.y = static_cast<uint16_t*>(y);
  p.m = m; p.n = n; p.k = k;
  p.act = act;
  return launched(op, kaio::launch_linear_w4a16(p, static_cast<hipStream_t>(stream)));
}

kaio_status kaio_rope_append(const kaio_paged_kv* kv, const void* q, const void* k, const void* v,
                             const int32_t* positions, const double* inv_freq, const uint32_t* sections,
                             uint32_t axes, int32_t interleaved, void* q_out, uint32_t tokens, uint32_t q_heads,
                             void* stream) {
  static const char* op = "rope_append";
  if (kaio_status st = check_paged_sizes(op, kv)) return st;
  if (axes < 1 || axes > kaio::kMaxAxes)
    return fail(KAIO_ERR_UNSUPPORTED, op, "axes (%u) must be 1 to %u", axes, kaio::kMaxAxes);
  if (kv->head_dim > 1024) return fail(KAIO_ERR_UNSUPPORTED, op, "head_dim (%u) must be at most 1024", kv->head_dim);
  if (!sections) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "sections is null");
  uint64_t half = 0;
  kaio::RopeAppend p;
  for (uint32_t a = 0; a < kaio::kMaxAxes; ++a) {
    p.first_pair[a] = (uint32_t)(half > 0xFFFFFFFFull ? 0xFFFFFFFFull : half);
    if (a < axes) half += sections[a];
  }
  if (2 * half > kv->head_dim)
    return fail(KAIO_ERR_INVALID_PROBLEM, op, "sections turn %llu pairs: head_dim (%u) has %u",
                (unsigned long long)half, kv->head_dim, kv->head_dim / 2);
  if (tokens == 0) return ok();
  uint64_t cache_bytes = 0, table_bytes = 0, q_bytes = 0, kv_bytes = 0;
  const uint64_t heads = (uint64_t)q_heads + 2ull * kv->kv_heads;
  if (!paged_fits(kv, &cache_bytes, &table_bytes) || tokens >= (1u << 31) ||
      !bytes_of(tokens, (uint64_t)q_heads * kv->head_dim, 2, &q_bytes) ||
      !bytes_of(tokens, (uint64_t)kv->kv_heads * kv->head_dim, 2, &kv_bytes) ||
      heads * kv->head_dim >= (1ull << 31) || tokens > kaio::kMaxWorkgroups)
    return fail(KAIO_ERR_INVALID_PROBLEM, op, "problem too large for one launch (tokens=%u, heads=%llu, slots=%llu)",
                tokens, (unsigned long long)heads, (unsigned long long)kv->pages * kv->page_size);
  if (kaio_status st = check_paged_pointers(op, kv)) return st;
  const struct { const void* p; const char* name; bool used; uintptr_t align; } all[6] = {
      {q, "input q", q_heads > 0, 16}, {k, "input k", true, 16}, {v, "input v", true, 16},
      {q_out, "output q_out", q_heads > 0, 16}, {positions, "positions", half > 0, 4}, {inv_freq, "inv_freq", half > 0, 8}};
  for (const auto& a : all)
    if (a.used && !a.p) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "%s is null", a.name);
  for (const auto& a : all)
    if (a.used && !aligned_to(a.p, a.align))
      return fail(KAIO_ERR_INVALID_ARGUMENT, op, "%s is not %u-byte aligned", a.name, (unsigned)a.align);
  const Range ro[3] = {range(q_out, q_bytes, "q_out"), range(kv->k_cache, cache_bytes, "k_cache"),
                       range(kv->v_cache, cache_bytes, "v_cache")};
  const Range ri[8] = {range(q, q != q_out ? q_bytes : 0, "q"), range(k, kv_bytes, "k"), range(v, kv_bytes, "v"),
                       range(positions, half ? (uint64_t)axes * tokens * 4 : 0, "positions"),
                       range(inv_freq, half * 8, "inv_freq"), range(kv->page_table, table_bytes, "page_table"),
                       range(kv->q_start, kv->seqs ? ((uint64_t)kv->seqs + 1) * 4 : 0, "q_start"),
                       range(kv->lens, (uint64_t)kv->seqs * 4, "lens")};
  const Range* other = nullptr;
  if (const Range* o = overlap(ro, 3, ri, 8, &other))
    return fail(KAIO_ERR_INVALID_ARGUMENT, op, "output %s overlaps %s", o->name, other->name);
  if (kaio_status st = check_device(op)) return st;
  (void)hipGetLastError();
  p.kv = paged_of(kv, tokens);
  p.q = static_cast<const uint16_t*>(q);
  p.k_new = static_cast<const uint16_t*>(k);
  p.v_new = static_cast<const uint16_t*>(v);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.axes = axes;
  p.half = (uint32_t)half;
  p.q_heads = q_heads;
  p.per_head = kaio::FastDiv::of(kv->head_dim >= 16 ? kv->head_dim / 16 : 1);
  p.bf16 = kv->dtype == KAIO_DTYPE_BF16;
  p.interleaved = interleaved != 0;
  return launched(op, kaio::launch_rope_append(p, static_cast<hipStream_t>(stream)));
}

size_t kaio_paged_attention_workspace_size(const kaio_paged_kv* kv, uint32_t tokens, uint32_t q_heads,
                                           uint32_t max_new) {
  if (!kv || kv->kv_heads == 0 || q_heads % kv->kv_heads != 0 || kv->page_size == 0 || tokens == 0) return 0;
  return attention_plan_of(kv, tokens, q_heads, max_new).workspace;
}

kaio_status kaio_paged_attention(const kaio_paged_kv* kv, const void* q, void* out, uint32_t tokens, uint32_t q_heads,
                                 uint32_t max_new, float scale, uint32_t window, uint32_t sinks, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  static const char* op = "paged_attention";
  if (kaio_status st = check_paged_sizes(op, kv)) return st;
  if (q_heads % kv->kv_heads != 0)
    return fail(KAIO_ERR_INVALID_PROBLEM, op, "q_heads (%u) must be a multiple of kv_heads (%u)", q_heads, kv->kv_heads);
  if (!std::isfinite(scale)) return fail(KAIO_ERR_INVALID_PROBLEM, op, "scale must be finite");
  if (kv->head_dim > 256) return fail(KAIO_ERR_UNSUPPORTED, op, "head_dim (%u) must be at most 256", kv->head_dim);
  if (tokens == 0 || q_heads == 0) return ok();
  if (max_new == 0) return fail(KAIO_ERR_INVALID_PROBLEM, op, "max_new must be > 0");
  uint64_t cache_bytes = 0, table_bytes = 0, q_bytes = 0;
  if (!paged_fits(kv, &cache_bytes, &table_bytes) || (uint64_t)tokens * q_heads > kaio::kMaxWorkgroups ||
      (uint64_t)kv->seqs * kv->kv_heads > kaio::kMaxWorkgroups / 2 ||
      !bytes_of(tokens, (uint64_t)q_heads * kv->head_dim, 2, &q_bytes))
    return fail(KAIO_ERR_INVALID_PROBLEM, op, "problem too large for one launch (tokens=%u, q_heads=%u, seqs=%u, slots=%llu)",
                tokens, q_heads, kv->seqs, (unsigned long long)kv->pages * kv->page_size);
  if (kaio_status st = check_paged_pointers(op, kv)) return st;
  const kaio::AttentionPlan plan = attention_plan_of(kv, tokens, q_heads, max_new, window, sinks);
  const uint64_t need = plan.workspace;
  if (!q) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "input q is null");
  if (!out) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "output out is null");
  if (need && !workspace) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "workspace is null");
  if (workspace_bytes < need)
    return fail(KAIO_ERR_INVALID_ARGUMENT, op, "workspace_bytes (%zu) < %llu needed", workspace_bytes,
                (unsigned long long)need);
  if (!aligned16(q)) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "input q is not 16-byte aligned");
  if (!aligned16(out)) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "output out is not 16-byte aligned");
  if (need && !aligned16(workspace)) return fail(KAIO_ERR_INVALID_ARGUMENT, op, "workspace is not 16-byte aligned");
  const Range ro[2] = {range(out, q_bytes, "out"), range(need ? workspace : nullptr, need, "workspace")};
  const Range ri[6] = {range(q, q_bytes, "q"), range(kv->k_cache, cache_bytes, "k_cache"),
                       range(kv->v_cache, cache_bytes, "v_cache"), range(kv->page_table, table_bytes, "page_table"),
                       range(kv->q_start, kv->seqs ? ((uint64_t)kv->seqs + 1) * 4 : 0, "q_start"),
                       range(kv->lens, (uint64_t)kv->seqs * 4, "lens")};
  const Range* other = nullptr;
  if (const Range* o = overlap(ro, 2, ri, 6, &other))
    return fail(KAIO_ERR_INVALID_ARGUMENT, op, "%s overlaps %s", o->name, other->name);
  if (kaio_status st = check_device(op)) return st;
  (void)hipGetLastError();
  kaio::PagedAttention p;
  p.kv = paged_of(kv, tokens);
  p.q = static_cast<const uint16_t*>(q);
  p.out = static_cast<uint16_t*>(out);
  p.workspace = need ? workspace : nullptr;
  p.q_heads = q_heads;
  p.group = kaio::FastDiv::of(q_heads / kv->kv_heads);
  p.max_new = max_new;
  p.scale = scale;
  p.window = window;
  p.sinks = sinks;
  p.bf16 = kv->dtype == KAIO_DTYPE_BF16;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (plan.rows) return launched(op, kaio::launch_attention_rows(p, st));
  const hipError_t e = plan.stream ? kaio::launch_attention_stream(p, plan, st) : kaio::launch_attention_tile(p, plan, st);
  if (e != hipSuccess || !plan.split) return launched(op, e);
  return launched(op, kaio::launch_attention_join(p, plan, st));
}

const char* kaio_last_error(void) { return g_last_error.c_str(); }

const char* kaio_version(void) { return "kaio-mi355x 0.1.0 gfx950"; }

}  // extern "C"
