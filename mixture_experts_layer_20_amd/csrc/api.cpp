// libmoe C-ABI: argument validation, workspace carving and kernel launches.
// Every entry point checks its arguments on the host before enqueuing anything, never
// synchronises, never allocates, and reports errors through status codes.
#include "libmoe.h"

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <memory>
#include <mutex>
#include <new>
#include <string>

#include "block_step.h"
#include "common.h"
#include "mxfp8.h"
#include "train_step.h"

namespace {

thread_local std::string g_err;

moe_status_t fail(moe_status_t st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_err = buf;
  return st;
}

moe_status_t hip_check(hipError_t e, const char* what) {
  if (e == hipSuccess) return MOE_OK;
  return fail(MOE_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

constexpr int64_t kMaxInt = 0x7fffffff;

#define CHECK(cond, st, ...)                 \
  do {                                       \
    if (!(cond)) return fail(st, __VA_ARGS__); \
  } while (0)

// Device tensors, index arrays and workspaces are accessed with vector loads and stores of up to
// 16 bytes (the GEMMs also with 16-byte direct-to-LDS loads) at offsets from each base pointer
// that are multiples of the access size, so every device pointer must be 16-byte aligned (hipMalloc
// and PyTorch allocations are 256-byte aligned).  NULL passes.
bool aligned16(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) & 15) return false;
  return true;
}

#define CHECK_ALIGN16(...)                                                   \
  CHECK(aligned16({__VA_ARGS__}), MOE_ERR_INVALID_VALUE,                    \
        "device pointers must be 16-byte aligned (" #__VA_ARGS__ ")")

moe_status_t check_dtype(moe_dtype_t dt) {
  CHECK(dt == MOE_F32 || dt == MOE_BF16, MOE_ERR_INVALID_VALUE, "dt must be MOE_F32 or MOE_BF16");
  return MOE_OK;
}

moe_status_t check_tokens(int64_t T, int64_t d, int32_t E, int32_t k) {
  CHECK(T >= 0, MOE_ERR_INVALID_VALUE, "T must be >= 0 (got %lld)", (long long)T);
  CHECK(d > 0, MOE_ERR_INVALID_VALUE, "d must be > 0 (got %lld)", (long long)d);
  CHECK(E > 0, MOE_ERR_INVALID_VALUE, "E must be > 0 (got %d)", E);
  CHECK(k > 0 && k <= E, MOE_ERR_INVALID_VALUE, "k must be in [1, E] (got k=%d, E=%d)", k, E);
  CHECK(E <= 256, MOE_ERR_UNSUPPORTED, "E > 256 is not supported (got %d)", E);
  CHECK(k <= 8, MOE_ERR_UNSUPPORTED, "k > 8 is not supported (got %d)", k);
  CHECK(d <= kMaxInt && T <= kMaxInt, MOE_ERR_UNSUPPORTED, "T and d must fit in int32");
  CHECK(T * k <= kMaxInt - 8, MOE_ERR_UNSUPPORTED, "T*k must be < 2^31");
  CHECK(T * (int64_t)E <= kMaxInt, MOE_ERR_UNSUPPORTED, "T*E must be < 2^31");
  return MOE_OK;
}

moe_status_t check_mlp(int32_t G, int64_t M, int64_t d, int64_t f, moe_dtype_t dt) {
  moe_status_t st = check_dtype(dt);
  if (st != MOE_OK) return st;
  CHECK(G > 0, MOE_ERR_INVALID_VALUE, "G must be > 0 (got %d)", G);
  CHECK(M >= 0, MOE_ERR_INVALID_VALUE, "M must be >= 0 (got %lld)", (long long)M);
  CHECK(d > 0 && f > 0, MOE_ERR_INVALID_VALUE, "d and f must be > 0");
  CHECK(d % 128 == 0 && f % 128 == 0, MOE_ERR_UNSUPPORTED,
        "d and f must be multiples of 128 (got d=%lld, f=%lld)", (long long)d, (long long)f);
  CHECK(M <= kMaxInt / 2 && d <= 65536 && f <= 65536 && G <= 1024, MOE_ERR_UNSUPPORTED,
        "sizes out of the supported range");
  CHECK(((M + 127) / 128 + G) * (2 * f / 64 + d / 64) < kMaxInt, MOE_ERR_UNSUPPORTED, "grid too large");
  return MOE_OK;
}

inline size_t align256(size_t b) { return (b + 255) / 256 * 256; }
inline size_t esize(moe_dtype_t dt) { return dt == MOE_BF16 ? 2 : 4; }
inline hipStream_t S(moe_stream_t s) { return reinterpret_cast<hipStream_t>(s); }

moe_status_t run_gemm(int mode, const moe::GemmArgs& a, moe_dtype_t dt, moe_stream_t s,
                      const char* what) {
  CHECK_ALIGN16(a.a, a.b0, a.b1, a.aux0, a.aux1, a.out0, a.out1, a.out2, a.offsets, a.tile_prefix);
  if (a.nseg == 2) CHECK_ALIGN16(a.s1.a, a.s1.b0, a.s1.b1, a.s1.aux0, a.s1.aux1, a.s1.out0, a.s1.out1, a.s1.out2,
                                 a.s1.offsets);
  return hip_check(moe::launch_grouped_gemm(mode, a, dt == MOE_BF16, S(s)), what);
}

moe::GemmArgs base_args(const int32_t* offsets, int32_t G, int64_t M, int64_t d, int64_t f, void* ws,
                        size_t ws_bytes) {
  moe::GemmArgs a{};
  a.offsets = offsets;
  a.tile_prefix = reinterpret_cast<int32_t*>(ws);
  a.ws_bytes = ws_bytes;
  a.G = G;
  a.M = (int)M;
  a.d = (int)d;
  a.f = (int)f;
  return a;
}

// ---------------------------------------------------------------------------------------------
// Scratch for the entry point that allocates nothing (moe_permute_noalloc): a file-scope device
// array that each GPU holds from the library's load until the process ends.  In host code the
// array's name only stands in for the symbol; its device address, different on every GPU, comes
// from hipGetSymbolAddress, taken once per device with that device current, and only that address
// is ever handed to a kernel.
constexpr size_t kScratchBytes = size_t(4) << 20;
static __device__ __align__(256) unsigned char scratch[kScratchBytes];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices] = {};

// The current device's scratch address (looked up on the first call on that device).
moe_status_t scratch_address(void** out) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(MOE_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
  CHECK(dev >= 0 && dev < kMaxDevices, MOE_ERR_UNSUPPORTED, "device %d is beyond the %d devices supported", dev,
        kMaxDevices);
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (g_scratch_ptr[dev] == nullptr) {
    void* ptr = nullptr;
    e = hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch));
    if (e != hipSuccess || ptr == nullptr)
      return fail(MOE_ERR_HIP, "hipGetSymbolAddress(scratch): %s", hipGetErrorString(e));
    g_scratch_ptr[dev] = ptr;
  }
  *out = g_scratch_ptr[dev];
  return MOE_OK;
}

}  // namespace

extern "C" {

const char* moe_status_string(moe_status_t st) {
  switch (st) {
    case MOE_OK: return "MOE_OK";
    case MOE_ERR_INVALID_VALUE: return "MOE_ERR_INVALID_VALUE";
    case MOE_ERR_UNSUPPORTED: return "MOE_ERR_UNSUPPORTED";
    case MOE_ERR_WORKSPACE: return "MOE_ERR_WORKSPACE";
    case MOE_ERR_HIP: return "MOE_ERR_HIP";
    default: return "MOE_ERR_UNKNOWN";
  }
}

const char* moe_last_error(void) { return g_err.c_str(); }

const char* moe_version(void) { return "libmoe 0.1 gfx950"; }

// ---------------------------------------------------------------------------------------------

moe_status_t moe_route(const void* x, const void* w_router, const float* bias, float* logits,
                       int64_t T, int64_t d, int32_t E, int32_t k, int32_t renormalize,
                       moe_dtype_t dt, int32_t* topk_idx, float* topk_gate, moe_stream_t stream) {
  g_err.clear();
  moe_status_t st = check_dtype(dt);
  if (st != MOE_OK) return st;
  if ((st = check_tokens(T, d, E, k)) != MOE_OK) return st;
  CHECK(renormalize == 0 || renormalize == 1, MOE_ERR_INVALID_VALUE, "renormalize must be 0 or 1");
  CHECK(!w_router || x, MOE_ERR_INVALID_VALUE, "x is NULL with a learned router");
  CHECK(w_router || !bias, MOE_ERR_INVALID_VALUE, "bias given without a learned router");
  if (T == 0) return MOE_OK;
  CHECK(logits && topk_idx && topk_gate, MOE_ERR_INVALID_VALUE, "logits/topk_idx/topk_gate is NULL");
  CHECK_ALIGN16(x, w_router, bias, logits, topk_idx, topk_gate);
  if (w_router) {
    st = hip_check(moe::launch_router_logits(x, w_router, bias, logits, (int)T, (int)d, E,
                                             dt == MOE_BF16, S(stream)),
                   "router logits");
    if (st != MOE_OK) return st;
  }
  return hip_check(moe::launch_topk_gate(logits, (int)T, E, k, renormalize, topk_idx, topk_gate, S(stream)),
                   "top-k");
}

size_t moe_permute_workspace_size(int64_t T, int32_t E, int32_t k) {
  if (T < 0 || E <= 0 || k <= 0) return 0;
  return moe::permute_ws_bytes(T, E, k);
}

moe_status_t moe_permute(const void* x, const int32_t* topk_idx, int64_t T, int64_t d, int32_t E,
                         int32_t k, moe_dtype_t dt, int32_t* counts, int32_t* offsets,
                         int32_t* dest_pos, int32_t* src_row, void* x_perm, void* ws,
                         size_t ws_bytes, moe_stream_t stream) {
  g_err.clear();
  moe_status_t st = check_dtype(dt);
  if (st != MOE_OK) return st;
  if ((st = check_tokens(T, d, E, k)) != MOE_OK) return st;
  CHECK(counts && offsets, MOE_ERR_INVALID_VALUE, "counts/offsets is NULL");
  CHECK(T == 0 || (topk_idx && dest_pos && src_row), MOE_ERR_INVALID_VALUE,
        "topk_idx/dest_pos/src_row is NULL");
  CHECK(!x_perm || x || T == 0, MOE_ERR_INVALID_VALUE, "x is NULL while x_perm is requested");
  CHECK(!x_perm || d % 8 == 0, MOE_ERR_UNSUPPORTED, "the row gather needs d %% 8 == 0 (got %lld)",
        (long long)d);
  const size_t need = moe::permute_ws_bytes(T, E, k);
  CHECK(ws && ws_bytes >= need, MOE_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need,
        ws ? ws_bytes : (size_t)0);
  CHECK_ALIGN16(x, topk_idx, counts, offsets, dest_pos, src_row, x_perm, ws);
  return hip_check(moe::launch_permute(x, topk_idx, (int)T, (int)d, E, k, dt == MOE_BF16, counts,
                                       offsets, dest_pos, src_row, x_perm, ws, S(stream)),
                   "permute");
}

size_t moe_permute_noalloc_max_scratch(void) { return kScratchBytes; }

moe_status_t moe_permute_noalloc(const void* x, const int32_t* topk_idx, int64_t T, int64_t d, int32_t E, int32_t k,
                                 moe_dtype_t dt, int32_t* counts, int32_t* offsets, int32_t* dest_pos,
                                 int32_t* src_row, void* x_perm, moe_stream_t stream) {
  g_err.clear();
  moe_status_t st = check_dtype(dt);
  if (st != MOE_OK) return st;
  if ((st = check_tokens(T, d, E, k)) != MOE_OK) return st;
  CHECK(counts && offsets, MOE_ERR_INVALID_VALUE, "counts/offsets is NULL");
  CHECK(T == 0 || (topk_idx && dest_pos && src_row), MOE_ERR_INVALID_VALUE,
        "topk_idx/dest_pos/src_row is NULL");
  CHECK(!x_perm || x || T == 0, MOE_ERR_INVALID_VALUE, "x is NULL while x_perm is requested");
  CHECK(!x_perm || d % 8 == 0, MOE_ERR_UNSUPPORTED, "the row gather needs d %% 8 == 0 (got %lld)",
        (long long)d);
  const size_t need = moe::permute_ws_bytes(T, E, k);
  CHECK(need <= kScratchBytes, MOE_ERR_UNSUPPORTED,
        "T*k = %lld with E = %d needs %zu bytes of scratch; moe_permute_noalloc holds %zu (use moe_permute)",
        (long long)(T * k), E, need, kScratchBytes);
  CHECK_ALIGN16(x, topk_idx, counts, offsets, dest_pos, src_row, x_perm);
  void* ws = nullptr;
  if ((st = scratch_address(&ws)) != MOE_OK) return st;
  // Every scratch element the kernels read they first write in the same call (chunk counts,
  // chunk bases, local ranks), so nothing needs clearing.
  return hip_check(moe::launch_permute(x, topk_idx, (int)T, (int)d, E, k, dt == MOE_BF16, counts,
                                       offsets, dest_pos, src_row, x_perm, ws, S(stream)),
                   "permute (no allocation)");
}

// ---------------------------------------------------------------------------------------------

size_t moe_grouped_mlp_fwd_workspace_size(int64_t M, int32_t G, int64_t d, int64_t f) {
  (void)M; (void)d; (void)f;
  if (G <= 0) return 0;
  return moe::gemm_ws_bytes(G);
}

size_t moe_grouped_mlp_bwd_workspace_size(int64_t M, int32_t G, int64_t d, int64_t f) {
  if (G <= 0 || M < 0 || f <= 0 || d <= 0) return 0;
  // Tile prefix and split-K partials first, dAB (sized for fp32 so one workspace serves both
  // element types) at the end.
  return moe::gemm_ws_bytes(G) + align256(moe::gemm_partial_bytes(G, M, (int)d, (int)f)) +
         align256((size_t)M * 2 * f * 4);
}

#define MLP_COMMON_CHECKS(need)                                                              \
  g_err.clear();                                                                             \
  moe_status_t st = check_mlp(G, M, d, f, dt);                                               \
  if (st != MOE_OK) return st;                                                               \
  CHECK(offsets, MOE_ERR_INVALID_VALUE, "offsets is NULL");                                  \
  CHECK(ws && ws_bytes >= (need), MOE_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", \
        (size_t)(need), ws ? ws_bytes : (size_t)0);

moe_status_t moe_expert_gate_up_fwd(const void* x_in, const int32_t* offsets, int32_t G,
                                    int64_t M, int64_t d, int64_t f, const void* w1,
                                    const void* w3, moe_dtype_t dt, void* a_stash, void* b_stash,
                                    void* h, void* ws, size_t ws_bytes, moe_stream_t stream) {
  MLP_COMMON_CHECKS(moe::gemm_ws_bytes(G));
  CHECK(w1 && w3 && (M == 0 || (x_in && h)), MOE_ERR_INVALID_VALUE, "x_in/w1/w3/h is NULL");
  CHECK((a_stash == nullptr) == (b_stash == nullptr), MOE_ERR_INVALID_VALUE,
        "a_stash and b_stash must both be given or both be NULL");
  moe::GemmArgs a = base_args(offsets, G, M, d, f, ws, ws_bytes);
  a.a = x_in; a.b0 = w1; a.b1 = w3; a.out0 = a_stash; a.out1 = b_stash; a.out2 = h;
  return run_gemm(moe::GEMM_UP_FWD, a, dt, stream, "gate/up GEMM");
}

moe_status_t moe_expert_down_fwd(const void* h, const int32_t* offsets, int32_t G, int64_t M,
                                 int64_t d, int64_t f, const void* w2, moe_dtype_t dt, void* y,
                                 void* ws, size_t ws_bytes, moe_stream_t stream) {
  MLP_COMMON_CHECKS(moe::gemm_ws_bytes(G));
  CHECK(w2 && (M == 0 || (h && y)), MOE_ERR_INVALID_VALUE, "h/w2/y is NULL");
  moe::GemmArgs a = base_args(offsets, G, M, d, f, ws, ws_bytes);
  a.a = h; a.b0 = w2; a.out0 = y;
  return run_gemm(moe::GEMM_DOWN_FWD, a, dt, stream, "down GEMM");
}

moe_status_t moe_expert_down_bwd(const void* dy, const void* a_stash, const void* b_stash,
                                 const int32_t* offsets, int32_t G, int64_t M, int64_t d,
                                 int64_t f, const void* w2, moe_dtype_t dt, void* dab, void* ws,
                                 size_t ws_bytes, moe_stream_t stream) {
  MLP_COMMON_CHECKS(moe::gemm_ws_bytes(G));
  CHECK(w2 && (M == 0 || (dy && a_stash && b_stash && dab)), MOE_ERR_INVALID_VALUE,
        "dy/a/b/w2/dab is NULL");
  moe::GemmArgs a = base_args(offsets, G, M, d, f, ws, ws_bytes);
  a.a = dy; a.b0 = w2; a.aux0 = a_stash; a.aux1 = b_stash; a.out0 = dab;
  return run_gemm(moe::GEMM_DOWN_BWD, a, dt, stream, "down dgrad GEMM");
}

moe_status_t moe_expert_down_wgrad(const void* dy, const void* h, const int32_t* offsets,
                                   int32_t G, int64_t M, int64_t d, int64_t f, moe_dtype_t dt,
                                   void* dw2, void* ws, size_t ws_bytes, moe_stream_t stream) {
  MLP_COMMON_CHECKS(moe::gemm_ws_bytes(G));
  CHECK(dw2 && (M == 0 || (dy && h)), MOE_ERR_INVALID_VALUE, "dy/h/dw2 is NULL");
  moe::GemmArgs a = base_args(offsets, G, M, d, f, ws, ws_bytes);
  a.a = dy; a.b0 = h; a.out0 = dw2;
  return run_gemm(moe::GEMM_DOWN_WGRAD, a, dt, stream, "down wgrad GEMM");
}

moe_status_t moe_expert_gate_up_dgrad(const void* dab, const int32_t* offsets, int32_t G,
                                      int64_t M, int64_t d, int64_t f, const void* w1,
                                      const void* w3, moe_dtype_t dt, void* dx_in, void* ws,
                                      size_t ws_bytes, moe_stream_t stream) {
  MLP_COMMON_CHECKS(moe::gemm_ws_bytes(G));
  CHECK(w1 && w3 && (M == 0 || (dab && dx_in)), MOE_ERR_INVALID_VALUE, "dab/w1/w3/dx_in is NULL");
  moe::GemmArgs a = base_args(offsets, G, M, d, f, ws, ws_bytes);
  a.a = dab; a.b0 = w1; a.b1 = w3; a.out0 = dx_in;
  return run_gemm(moe::GEMM_UP_DGRAD, a, dt, stream, "gate/up dgrad GEMM");
}

moe_status_t moe_expert_gate_up_wgrad(const void* dab, const void* x_in, const int32_t* offsets,
                                      int32_t G, int64_t M, int64_t d, int64_t f, moe_dtype_t dt,
                                      void* dw1, void* dw3, void* ws, size_t ws_bytes,
                                      moe_stream_t stream) {
  MLP_COMMON_CHECKS(moe::gemm_ws_bytes(G));
  CHECK(dw1 && dw3 && (M == 0 || (dab && x_in)), MOE_ERR_INVALID_VALUE, "dab/x_in/dw1/dw3 is NULL");
  moe::GemmArgs a = base_args(offsets, G, M, d, f, ws, ws_bytes);
  a.a = dab; a.b0 = x_in; a.out0 = dw1; a.out1 = dw3;
  return run_gemm(moe::GEMM_UP_WGRAD, a, dt, stream, "gate/up wgrad GEMM");
}

size_t moe_expert_stage_workspace_size(const moe_expert_set_t* sets, int32_t nsets, int64_t d) {
  if (!sets || nsets < 1 || nsets > 2 || d <= 0) return 0;
  size_t need = 0;
  for (int i = 0; i < nsets; ++i) {
    const moe_expert_set_t& e = sets[i];
    if (e.G <= 0 || e.M < 0 || e.f <= 0) return 0;
    need = std::max(need, moe::gemm_ws_bytes(e.G) + align256(moe::gemm_partial_bytes(e.G, e.M, (int)d, (int)e.f)));
  }
  if (nsets == 2)
    need = std::max(need, moe::gemm_ws_bytes(sets[0].G) +
                              align256(moe::gemm_sets_partial_bytes(sets[0].G, sets[0].M, sets[1].G, sets[1].M,
                                                                    (int)d, (int)sets[1].f)));
  return need;
}

namespace {

// The GEMM operands of one expert set for a stage, or an error when a member the stage needs is
// missing.
moe_status_t stage_operands(moe_stage_t stage, const moe_expert_set_t& e, moe::GemmArgs& a) {
  const bool rows = e.M > 0;
  switch (stage) {
    case MOE_STAGE_GATE_UP_FWD:
      CHECK(e.w1 && e.w3 && (!rows || (e.x && e.h)), MOE_ERR_INVALID_VALUE, "x/w1/w3/h is NULL");
      CHECK((e.a == nullptr) == (e.b == nullptr), MOE_ERR_INVALID_VALUE,
            "a and b must both be given or both be NULL");
      a.a = e.x; a.b0 = e.w1; a.b1 = e.w3; a.out0 = e.a; a.out1 = e.b; a.out2 = e.h;
      return MOE_OK;
    case MOE_STAGE_DOWN_FWD:
      CHECK(e.w2 && (!rows || (e.h && e.y)), MOE_ERR_INVALID_VALUE, "h/w2/y is NULL");
      a.a = e.h; a.b0 = e.w2; a.out0 = e.y;
      return MOE_OK;
    case MOE_STAGE_DOWN_BWD:
      CHECK(e.w2 && (!rows || (e.dy && e.a && e.b && e.dab)), MOE_ERR_INVALID_VALUE, "dy/a/b/w2/dab is NULL");
      a.a = e.dy; a.b0 = e.w2; a.aux0 = e.a; a.aux1 = e.b; a.out0 = e.dab;
      return MOE_OK;
    case MOE_STAGE_GATE_UP_DGRAD:
      CHECK(e.w1 && e.w3 && (!rows || (e.dab && e.dx)), MOE_ERR_INVALID_VALUE, "dab/w1/w3/dx is NULL");
      a.a = e.dab; a.b0 = e.w1; a.b1 = e.w3; a.out0 = e.dx;
      return MOE_OK;
    case MOE_STAGE_DOWN_WGRAD:
      CHECK(e.dw2 && (!rows || (e.dy && e.h)), MOE_ERR_INVALID_VALUE, "dy/h/dw2 is NULL");
      a.a = e.dy; a.b0 = e.h; a.out0 = e.dw2;
      return MOE_OK;
    case MOE_STAGE_GATE_UP_WGRAD:
      CHECK(e.dw1 && e.dw3 && (!rows || (e.dab && e.x)), MOE_ERR_INVALID_VALUE, "dab/x/dw1/dw3 is NULL");
      a.a = e.dab; a.b0 = e.x; a.out0 = e.dw1; a.out1 = e.dw3;
      return MOE_OK;
  }
  return fail(MOE_ERR_INVALID_VALUE, "unknown stage %d", (int)stage);
}

}  // namespace

moe_status_t moe_expert_stage(moe_stage_t stage, const moe_expert_set_t* sets, int32_t nsets, int64_t d,
                              moe_dtype_t dt, void* ws, size_t ws_bytes, moe_stream_t stream) {
  g_err.clear();
  CHECK(sets && (nsets == 1 || nsets == 2), MOE_ERR_INVALID_VALUE, "nsets must be 1 or 2 (got %d)", (int)nsets);
  CHECK((int)stage >= 0 && (int)stage <= 5, MOE_ERR_INVALID_VALUE, "unknown stage %d", (int)stage);
  size_t need = 0;
  moe::GemmArgs a{};
  for (int i = 0; i < nsets; ++i) {
    const moe_expert_set_t& e = sets[i];
    moe_status_t st = check_mlp(e.G, e.M, d, e.f, dt);
    if (st != MOE_OK) return st;
    CHECK(e.offsets, MOE_ERR_INVALID_VALUE, "offsets of set %d is NULL", i);
    need = std::max(need, moe::gemm_ws_bytes(e.G));
    moe::GemmArgs s = base_args(e.offsets, e.G, e.M, d, e.f, ws, ws_bytes);
    if ((st = stage_operands(stage, e, s)) != MOE_OK) return st;
    if (i == 0) {
      a = s;
    } else {
      a.nseg = 2;
      a.s1 = moe::GemmSeg{s.a, s.b0, s.b1, s.aux0, s.aux1, s.out0, s.out1, s.out2, s.offsets, s.G, s.M, s.f};
    }
  }
  CHECK(ws && ws_bytes >= need, MOE_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need,
        ws ? ws_bytes : (size_t)0);
  static const char* names[6] = {"gate/up GEMM", "down GEMM", "down dgrad GEMM", "gate/up dgrad GEMM",
                                 "down wgrad GEMM", "gate/up wgrad GEMM"};
  return run_gemm((int)stage, a, dt, stream, names[(int)stage]);
}

moe_status_t moe_grouped_mlp_fwd(const void* x_in, const int32_t* offsets, int32_t G, int64_t M,
                                 int64_t d, int64_t f, const void* w1, const void* w3,
                                 const void* w2, moe_dtype_t dt, void* a_stash, void* b_stash,
                                 void* h, void* y, void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_status_t st = moe_expert_gate_up_fwd(x_in, offsets, G, M, d, f, w1, w3, dt, a_stash, b_stash,
                                           h, ws, ws_bytes, stream);
  if (st != MOE_OK) return st;
  return moe_expert_down_fwd(h, offsets, G, M, d, f, w2, dt, y, ws, ws_bytes, stream);
}

moe_status_t moe_grouped_mlp_bwd(const void* dy, const void* x_in, const void* a, const void* b,
                                 const void* h, const int32_t* offsets, int32_t G, int64_t M,
                                 int64_t d, int64_t f, const void* w1, const void* w3,
                                 const void* w2, moe_dtype_t dt, void* dx_in, void* dw1, void* dw3,
                                 void* dw2, void* ws, size_t ws_bytes, moe_stream_t stream) {
  MLP_COMMON_CHECKS(moe_grouped_mlp_bwd_workspace_size(M, G, d, f));
  CHECK(w1 && w3 && w2 && dw1 && dw3 && dw2, MOE_ERR_INVALID_VALUE, "weight or gradient pointer is NULL");
  CHECK(M == 0 || (dy && x_in && a && b && h && dx_in), MOE_ERR_INVALID_VALUE,
        "activation pointer is NULL");
  const size_t dab_bytes = align256((size_t)M * 2 * f * 4);
  const size_t gws = moe_grouped_mlp_bwd_workspace_size(M, G, d, f) - dab_bytes;
  void* dab = reinterpret_cast<char*>(ws) + gws;
  if ((st = moe_expert_down_bwd(dy, a, b, offsets, G, M, d, f, w2, dt, dab, ws, gws, stream)) != MOE_OK)
    return st;
  if ((st = moe_expert_down_wgrad(dy, h, offsets, G, M, d, f, dt, dw2, ws, gws, stream)) != MOE_OK)
    return st;
  if ((st = moe_expert_gate_up_dgrad(dab, offsets, G, M, d, f, w1, w3, dt, dx_in, ws, gws, stream)) != MOE_OK)
    return st;
  return moe_expert_gate_up_wgrad(dab, x_in, offsets, G, M, d, f, dt, dw1, dw3, ws, gws, stream);
}

// ---------------------------------------------------------------------------------------------

moe_status_t moe_combine(const void* y_perm, const float* topk_gate, const int32_t* dest_pos,
                         const void* shared_out, int64_t T, int64_t d, int32_t k, moe_dtype_t dt,
                         void* out, moe_stream_t stream) {
  g_err.clear();
  moe_status_t st = check_dtype(dt);
  if (st != MOE_OK) return st;
  if ((st = check_tokens(T, d, k, k)) != MOE_OK) return st;
  CHECK(d % 8 == 0, MOE_ERR_UNSUPPORTED, "d must be a multiple of 8 (got %lld)", (long long)d);
  if (T == 0) return MOE_OK;
  CHECK(y_perm && topk_gate && dest_pos && out, MOE_ERR_INVALID_VALUE, "y_perm/topk_gate/dest_pos/out is NULL");
  CHECK_ALIGN16(y_perm, topk_gate, dest_pos, shared_out, out);
  return hip_check(moe::launch_combine(y_perm, topk_gate, dest_pos, shared_out, (int)T, (int)d, k,
                                       dt == MOE_BF16, out, S(stream)),
                   "combine");
}

moe_status_t moe_combine_bwd(const void* dout, const void* y_perm, const float* topk_gate,
                             const int32_t* dest_pos, int64_t T, int64_t d, int32_t k,
                             moe_dtype_t dt, void* dy_perm, float* dgate, moe_stream_t stream) {
  g_err.clear();
  moe_status_t st = check_dtype(dt);
  if (st != MOE_OK) return st;
  if ((st = check_tokens(T, d, k, k)) != MOE_OK) return st;
  CHECK(d % 8 == 0, MOE_ERR_UNSUPPORTED, "d must be a multiple of 8 (got %lld)", (long long)d);
  if (T == 0) return MOE_OK;
  CHECK(dout && topk_gate && dest_pos && dy_perm, MOE_ERR_INVALID_VALUE, "dout/topk_gate/dest_pos/dy_perm is NULL");
  CHECK(!dgate || y_perm, MOE_ERR_INVALID_VALUE, "y_perm is NULL while dgate is requested");
  CHECK_ALIGN16(dout, y_perm, topk_gate, dest_pos, dy_perm, dgate);
  return hip_check(moe::launch_combine_bwd(dout, y_perm, topk_gate, dest_pos, (int)T, (int)d, k,
                                           dt == MOE_BF16, dy_perm, dgate, S(stream)),
                   "combine backward");
}

moe_status_t moe_permute_bwd(const void* dx_perm, const int32_t* dest_pos, const void* dx_add0,
                             const void* dx_add1, int64_t T, int64_t d, int32_t k,
                             moe_dtype_t dt, void* dx, moe_stream_t stream) {
  g_err.clear();
  moe_status_t st = check_dtype(dt);
  if (st != MOE_OK) return st;
  if ((st = check_tokens(T, d, k, k)) != MOE_OK) return st;
  CHECK(d % 8 == 0, MOE_ERR_UNSUPPORTED, "d must be a multiple of 8 (got %lld)", (long long)d);
  if (T == 0) return MOE_OK;
  CHECK(dx_perm && dest_pos && dx, MOE_ERR_INVALID_VALUE, "dx_perm/dest_pos/dx is NULL");
  CHECK_ALIGN16(dx_perm, dest_pos, dx_add0, dx_add1, dx);
  return hip_check(moe::launch_permute_bwd(dx_perm, dest_pos, dx_add0, dx_add1, (int)T, (int)d, k,
                                           dt == MOE_BF16, dx, S(stream)),
                   "permute backward");
}

size_t moe_route_bwd_workspace_size(int64_t T, int64_t d, int32_t E, int32_t k) {
  if (T < 0 || d <= 0 || E <= 0 || k <= 0) return 0;
  return moe::route_bwd_ws_bytes(T, d, E, k);
}

moe_status_t moe_route_bwd(const float* dgate, const float* topk_gate, const int32_t* topk_idx,
                           const int32_t* offsets, const int32_t* src_row, const void* x,
                           const void* w_router, int64_t T, int64_t d, int32_t E, int32_t k,
                           int32_t renormalize, moe_dtype_t dt, float* dw_router, void* dx_router,
                           void* ws, size_t ws_bytes, moe_stream_t stream) {
  g_err.clear();
  moe_status_t st = check_dtype(dt);
  if (st != MOE_OK) return st;
  if ((st = check_tokens(T, d, E, k)) != MOE_OK) return st;
  CHECK(renormalize == 0 || renormalize == 1, MOE_ERR_INVALID_VALUE, "renormalize must be 0 or 1");
  CHECK(renormalize == 1, MOE_ERR_UNSUPPORTED, "router backward supports renormalized gates only");
  CHECK(offsets && w_router && dw_router, MOE_ERR_INVALID_VALUE, "offsets/w_router/dw_router is NULL");
  CHECK(T == 0 || (dgate && topk_gate && topk_idx && src_row && x && dx_router), MOE_ERR_INVALID_VALUE,
        "a per-token pointer is NULL");
  const size_t need = moe::route_bwd_ws_bytes(T, d, E, k);
  CHECK(ws && ws_bytes >= need, MOE_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need,
        ws ? ws_bytes : (size_t)0);
  CHECK_ALIGN16(dgate, topk_gate, topk_idx, offsets, src_row, x, w_router, dw_router, dx_router, ws);
  return hip_check(moe::launch_route_bwd(dgate, topk_gate, topk_idx, offsets, src_row, x, w_router,
                                         (int)T, (int)d, E, k, dt == MOE_BF16, dw_router, dx_router,
                                         ws, S(stream)),
                   "router backward");
}

size_t moe_router_aux_workspace_size(int64_t T, int32_t E) {
  if (T < 0 || E <= 0) return 0;
  return moe::router_aux_ws_bytes(T, E);
}

moe_status_t moe_router_aux(const float* logits, const int32_t* counts, int64_t T, int32_t E, int32_t k,
                            float weight, float* loss, float* prob_mean, float* load_frac, void* ws,
                            size_t ws_bytes, moe_stream_t stream) {
  g_err.clear();
  moe_status_t st = check_tokens(T, 1, E, k);
  if (st != MOE_OK) return st;
  CHECK(counts && loss && prob_mean && load_frac, MOE_ERR_INVALID_VALUE, "counts/loss/prob_mean/load_frac is NULL");
  CHECK(T == 0 || logits, MOE_ERR_INVALID_VALUE, "logits is NULL");
  const size_t need = moe::router_aux_ws_bytes(T, E);
  CHECK(ws && ws_bytes >= need, MOE_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need,
        ws ? ws_bytes : (size_t)0);
  CHECK_ALIGN16(logits, counts, loss, prob_mean, load_frac, ws);
  return hip_check(moe::launch_router_aux(logits, counts, (int)T, E, k, weight, loss, prob_mean, load_frac, ws,
                                          S(stream)),
                   "router statistics");
}

size_t moe_router_aux_bwd_workspace_size(int64_t T, int64_t d, int32_t E) {
  if (T < 0 || d <= 0 || E <= 0) return 0;
  return moe::router_aux_bwd_ws_bytes(T, d, E);
}

moe_status_t moe_router_aux_bwd(const float* logits, const float* load_frac, const void* x, const void* w_router,
                                int64_t T, int64_t d, int32_t E, float weight, moe_dtype_t dt, float* dw_router,
                                void* dx_router, void* ws, size_t ws_bytes, moe_stream_t stream) {
  g_err.clear();
  moe_status_t st = check_dtype(dt);
  if (st != MOE_OK) return st;
  if ((st = check_tokens(T, d, E, 1)) != MOE_OK) return st;
  CHECK(d % 8 == 0, MOE_ERR_UNSUPPORTED, "d must be a multiple of 8 (got %lld)", (long long)d);
  CHECK(load_frac && w_router && dw_router, MOE_ERR_INVALID_VALUE, "load_frac/w_router/dw_router is NULL");
  CHECK(T == 0 || (logits && x && dx_router), MOE_ERR_INVALID_VALUE, "logits/x/dx_router is NULL");
  const size_t need = moe::router_aux_bwd_ws_bytes(T, d, E);
  CHECK(ws && ws_bytes >= need, MOE_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need,
        ws ? ws_bytes : (size_t)0);
  CHECK_ALIGN16(logits, load_frac, x, w_router, dw_router, dx_router, ws);
  return hip_check(moe::launch_router_aux_bwd(logits, load_frac, x, w_router, (int)T, (int)d, E, weight,
                                              dt == MOE_BF16, dw_router, dx_router, ws, S(stream)),
                   "router load-balancing backward");
}

// ---------------------------------------------------------------------------------------------
// Norms around the block

namespace {

constexpr int64_t kNormMaxWidth = 16384;

moe_status_t check_norm(int64_t T, int64_t d, moe_dtype_t dt) {
  moe_status_t st = check_dtype(dt);
  if (st != MOE_OK) return st;
  CHECK(T >= 0, MOE_ERR_INVALID_VALUE, "T must be >= 0 (got %lld)", (long long)T);
  CHECK(d > 0, MOE_ERR_INVALID_VALUE, "d must be > 0 (got %lld)", (long long)d);
  CHECK(d % 8 == 0 && d <= kNormMaxWidth, MOE_ERR_UNSUPPORTED,
        "d must be a multiple of 8, at most %lld (got %lld)", (long long)kNormMaxWidth, (long long)d);
  CHECK(T <= kMaxInt / 2, MOE_ERR_UNSUPPORTED, "T must be < 2^30 (got %lld)", (long long)T);
  return MOE_OK;
}

// eps >= 0 (a NaN fails the comparison).
#define CHECK_EPS(eps) CHECK((eps) >= 0.0f, MOE_ERR_INVALID_VALUE, "eps must be >= 0")

moe_status_t check_gate(const void* gate, int64_t& gate_rows, int64_t T) {
  if (!gate) {
    gate_rows = 1;
    return MOE_OK;
  }
  CHECK(gate_rows >= 1, MOE_ERR_INVALID_VALUE, "gate_rows must be >= 1 (got %lld)", (long long)gate_rows);
  gate_rows = std::min(gate_rows, std::max<int64_t>(T, 1));
  return MOE_OK;
}

}  // namespace

moe_status_t moe_norm_in(const void* x, const void* w, int64_t T, int64_t d, float eps, moe_dtype_t dt, void* xn,
                         float* rstd, moe_stream_t stream) {
  g_err.clear();
  moe_status_t st = check_norm(T, d, dt);
  if (st != MOE_OK) return st;
  CHECK_EPS(eps);
  if (T == 0) return MOE_OK;
  CHECK(x && w && xn, MOE_ERR_INVALID_VALUE, "x/w/xn is NULL");
  CHECK_ALIGN16(x, w, xn, rstd);
  return hip_check(moe::launch_norm_in(x, w, (int)T, (int)d, eps, dt == MOE_BF16, xn, rstd, S(stream)), "norm before");
}

moe_status_t moe_norm_out(const void* y, const void* x, const void* w, const void* gate, int64_t gate_rows,
                          float res_scale, float eps, int64_t T, int64_t d, moe_dtype_t dt, void* out, float* rstd,
                          moe_stream_t stream) {
  g_err.clear();
  moe_status_t st = check_norm(T, d, dt);
  if (st != MOE_OK) return st;
  CHECK_EPS(eps);
  if ((st = check_gate(gate, gate_rows, T)) != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  CHECK(y && x && w && out, MOE_ERR_INVALID_VALUE, "y/x/w/out is NULL");
  CHECK_ALIGN16(y, x, w, gate, out, rstd);
  return hip_check(moe::launch_norm_out(y, nullptr, nullptr, nullptr, 0, x, w, gate, (int)gate_rows, res_scale, eps,
                                        (int)T, (int)d, dt == MOE_BF16, nullptr, out, rstd, S(stream)),
                   "norm after");
}

moe_status_t moe_combine_norm_out(const void* y_perm, const float* topk_gate, const int32_t* dest_pos,
                                  const void* shared_out, const void* x, const void* w, const void* gate,
                                  int64_t gate_rows, float res_scale, float eps, int64_t T, int64_t d, int32_t k,
                                  moe_dtype_t dt, void* y, void* out, float* rstd, moe_stream_t stream) {
  g_err.clear();
  moe_status_t st = check_norm(T, d, dt);
  if (st != MOE_OK) return st;
  CHECK(k > 0, MOE_ERR_INVALID_VALUE, "k must be > 0 (got %d)", k);
  CHECK(k <= 8, MOE_ERR_UNSUPPORTED, "k > 8 is not supported (got %d)", k);
  CHECK(T * k <= kMaxInt - 8, MOE_ERR_UNSUPPORTED, "T*k must be < 2^31");
  CHECK_EPS(eps);
  if ((st = check_gate(gate, gate_rows, T)) != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  CHECK(y_perm && topk_gate && dest_pos, MOE_ERR_INVALID_VALUE, "y_perm/topk_gate/dest_pos is NULL");
  CHECK(x && w && out, MOE_ERR_INVALID_VALUE, "x/w/out is NULL");
  CHECK_ALIGN16(y_perm, topk_gate, dest_pos, shared_out, x, w, gate, y, out, rstd);
  return hip_check(moe::launch_norm_out(y_perm, topk_gate, dest_pos, shared_out, k, x, w, gate, (int)gate_rows,
                                        res_scale, eps, (int)T, (int)d, dt == MOE_BF16, y, out, rstd, S(stream)),
                   "combine and norm after");
}

size_t moe_norm_bwd_workspace_size(int64_t T, int64_t d) {
  if (T < 0 || d <= 0 || d > kNormMaxWidth || T > kMaxInt / 2) return 0;
  return align256(moe::norm_bwd_ws_bytes(T, (int)d));
}

moe_status_t moe_norm_out_bwd(const void* dout, const void* y, const void* w, const void* gate, int64_t gate_rows,
                              const float* rstd, int64_t T, int64_t d, moe_dtype_t dt, void* dy, float* dw,
                              float* dgate, void* ws, size_t ws_bytes, moe_stream_t stream) {
  g_err.clear();
  moe_status_t st = check_norm(T, d, dt);
  if (st != MOE_OK) return st;
  if ((st = check_gate(gate, gate_rows, T)) != MOE_OK) return st;
  CHECK(w && dw && (T == 0 || (dout && y && rstd && dy)), MOE_ERR_INVALID_VALUE, "dout/y/w/rstd/dy/dw is NULL");
  CHECK((gate == nullptr) == (dgate == nullptr), MOE_ERR_INVALID_VALUE,
        "gate and dgate must both be given or both be NULL");
  const size_t need = moe_norm_bwd_workspace_size(T, d);
  CHECK(need == 0 || (ws && ws_bytes >= need), MOE_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need,
        ws ? ws_bytes : (size_t)0);
  CHECK_ALIGN16(dout, y, w, gate, rstd, dy, dw, dgate, ws);
  return hip_check(moe::launch_norm_out_bwd(dout, y, w, gate, (int)gate_rows, rstd, (int)T, (int)d, dt == MOE_BF16, dy,
                                            dw, dgate, ws, S(stream)),
                   "norm after, backward");
}

moe_status_t moe_norm_in_bwd(const void* dxn, const void* x, const void* w, const float* rstd, const void* dres,
                             float res_scale, int64_t T, int64_t d, moe_dtype_t dt, void* dx, float* dw, void* ws,
                             size_t ws_bytes, moe_stream_t stream) {
  g_err.clear();
  moe_status_t st = check_norm(T, d, dt);
  if (st != MOE_OK) return st;
  CHECK(w && dw && (T == 0 || (dxn && x && rstd && dx)), MOE_ERR_INVALID_VALUE, "dxn/x/w/rstd/dx/dw is NULL");
  const size_t need = moe_norm_bwd_workspace_size(T, d);
  CHECK(need == 0 || (ws && ws_bytes >= need), MOE_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need,
        ws ? ws_bytes : (size_t)0);
  CHECK_ALIGN16(dxn, x, w, rstd, dres, dx, dw, ws);
  return hip_check(moe::launch_norm_in_bwd(dxn, x, w, rstd, dres, res_scale, (int)T, (int)d, dt == MOE_BF16, dx, dw, ws,
                                           S(stream)),
                   "norm before, backward");
}

// ---------------------------------------------------------------------------------------------
// Softmax cross entropy over a vocabulary

namespace {

constexpr int64_t kVocabMax = int64_t(1) << 22;

moe_status_t check_vocab(int64_t T, int64_t d, int64_t V, moe_dtype_t dt) {
  moe_status_t st = check_dtype(dt);
  if (st != MOE_OK) return st;
  CHECK(T >= 0, MOE_ERR_INVALID_VALUE, "T must be >= 0 (got %lld)", (long long)T);
  CHECK(d > 0 && V > 0, MOE_ERR_INVALID_VALUE, "d and V must be > 0 (got d=%lld, V=%lld)", (long long)d, (long long)V);
  CHECK(d % 8 == 0 && d <= 65536, MOE_ERR_UNSUPPORTED, "d must be a multiple of 8, at most 65536 (got %lld)",
        (long long)d);
  CHECK(T <= kVocabMax && V <= kVocabMax, MOE_ERR_UNSUPPORTED, "T and V must be at most 2^22 (got T=%lld, V=%lld)",
        (long long)T, (long long)V);
  // Tiles of 64 x 64 outputs with 256 threads each: a grid has fewer than 2^32 threads.
  const int64_t most = int64_t(1) << 35;
  CHECK(T * V <= most && V * d <= most && T * d <= most, MOE_ERR_UNSUPPORTED,
        "T V, V d and T d must be at most 2^35 (got T=%lld, d=%lld, V=%lld)", (long long)T, (long long)d, (long long)V);
  return MOE_OK;
}

}  // namespace

size_t moe_vocab_loss_workspace_size(int64_t T, int64_t d, int64_t V, moe_dtype_t dt) {
  if (check_vocab(T, d, V, dt) != MOE_OK) return 0;
  return align256(moe::vocab_loss_ws_bytes(T, d, V, dt == MOE_BF16));
}

moe_status_t moe_vocab_loss(const void* h, const void* w, const int32_t* target, int64_t T, int64_t d, int64_t V,
                            moe_dtype_t dt, float* loss, float* lse, void* ws, size_t ws_bytes, moe_stream_t stream) {
  g_err.clear();
  moe_status_t st = check_vocab(T, d, V, dt);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  CHECK(h && w && target && loss && lse, MOE_ERR_INVALID_VALUE, "h/w/target/loss/lse is NULL");
  const size_t need = moe_vocab_loss_workspace_size(T, d, V, dt);
  CHECK(ws && ws_bytes >= need, MOE_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need,
        ws ? ws_bytes : (size_t)0);
  CHECK_ALIGN16(h, w, target, loss, lse, ws);
  return hip_check(moe::launch_vocab_loss(h, w, target, (int)T, (int)d, (int)V, dt == MOE_BF16, loss, lse, ws, S(stream)),
                   "vocabulary loss");
}

moe_status_t moe_vocab_loss_plan(int64_t T, int64_t d, int64_t V, moe_dtype_t dt, moe_vocab_loss_plan_t* plan) {
  g_err.clear();
  moe_status_t st = check_vocab(T, d, V, dt);
  if (st != MOE_OK) return st;
  CHECK(plan, MOE_ERR_INVALID_VALUE, "plan is NULL");
  const moe::VocabPlan p = moe::vocab_loss_plan((int)T, (int)d, (int)V, dt == MOE_BF16);
  *plan = moe_vocab_loss_plan_t{p.piece_words, p.pieces, p.fwd_tile, p.logits_tile, p.dh_tile, p.dw_tile, p.dh_splits, p.dw_splits};
  return MOE_OK;
}

size_t moe_vocab_loss_bwd_workspace_size(int64_t T, int64_t d, int64_t V, moe_dtype_t dt) {
  if (check_vocab(T, d, V, dt) != MOE_OK) return 0;
  return align256(moe::vocab_loss_bwd_ws_bytes(T, d, V, dt == MOE_BF16));
}

moe_status_t moe_vocab_loss_bwd(const void* h, const void* w, const int32_t* target, const float* lse,
                                const float* dloss, int64_t T, int64_t d, int64_t V, moe_dtype_t dt, void* dh, void* dw,
                                void* ws, size_t ws_bytes, moe_stream_t stream) {
  g_err.clear();
  moe_status_t st = check_vocab(T, d, V, dt);
  if (st != MOE_OK) return st;
  CHECK(w && dw && (T == 0 || (h && target && lse && dloss && dh)), MOE_ERR_INVALID_VALUE,
        "h/w/target/lse/dloss/dh/dw is NULL");
  const size_t need = moe_vocab_loss_bwd_workspace_size(T, d, V, dt);
  CHECK(need == 0 || (ws && ws_bytes >= need), MOE_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need,
        ws ? ws_bytes : (size_t)0);
  CHECK_ALIGN16(h, w, target, lse, dloss, dh, dw, ws);
  return hip_check(moe::launch_vocab_loss_bwd(h, w, target, lse, dloss, (int)T, (int)d, (int)V, dt == MOE_BF16, dh, dw,
                                              ws, S(stream)),
                   "vocabulary loss, backward");
}

// ---------------------------------------------------------------------------------------------
// Gradient norm and clipping

namespace {

// The list in the launchers' form, and its checks.  `scale`: the call writes out.
struct GradList {
  std::unique_ptr<moe::GradItem[]> items;
  long long chunks = 0;
};

constexpr int64_t kGradMaxElements = int64_t(1) << 41;   // a chunk then has fewer than 2^31

moe_status_t grad_list(const moe_grad_t* grads, int32_t count, bool scale, GradList& list) {
  CHECK(count >= 0, MOE_ERR_INVALID_VALUE, "count must be >= 0 (got %d)", count);
  CHECK(count == 0 || grads, MOE_ERR_INVALID_VALUE, "grads is NULL");
  CHECK(count <= 1 << 20, MOE_ERR_UNSUPPORTED, "count must be at most 2^20 (got %d)", count);
  list.items.reset(new (std::nothrow) moe::GradItem[std::max(count, 1)]);
  CHECK(list.items, MOE_ERR_UNSUPPORTED, "no host memory for a list of %d gradients", count);
  int64_t total = 0;
  for (int i = 0; i < count; ++i) {
    const moe_grad_t& g = grads[i];
    moe_status_t st = check_dtype(g.dt);
    if (st != MOE_OK) return st;
    CHECK(g.n >= 0, MOE_ERR_INVALID_VALUE, "gradient %d has n = %lld", i, (long long)g.n);
    CHECK(g.n <= kGradMaxElements - total, MOE_ERR_UNSUPPORTED, "more than 2^41 gradient elements");
    total += g.n;
    CHECK(g.n == 0 || (g.grad && (!scale || g.out)), MOE_ERR_INVALID_VALUE, "gradient %d: grad/out is NULL", i);
    CHECK(aligned16({g.grad, scale ? g.out : nullptr}), MOE_ERR_INVALID_VALUE,
          "device pointers must be 16-byte aligned (gradient %d)", i);
    list.items[i] = moe::GradItem{g.grad, g.out, (long long)g.n, g.dt == MOE_BF16};
  }
  list.chunks = moe::grad_chunks(list.items.get(), count);
  if (!scale) return MOE_OK;
  // No output may overlap another tensor of the list: sweep the address ranges in order of their
  // starts, keeping the furthest end of an output and of any range so far.
  struct Range {
    uintptr_t begin, end;
    bool out;
  };
  std::unique_ptr<Range[]> r(new (std::nothrow) Range[2 * (size_t)std::max(count, 1)]);
  CHECK(r, MOE_ERR_UNSUPPORTED, "no host memory for a list of %d gradients", count);
  size_t n = 0;
  for (int i = 0; i < count; ++i) {
    if (grads[i].n == 0) continue;
    const size_t bytes = (size_t)grads[i].n * esize(grads[i].dt);
    const uintptr_t o = reinterpret_cast<uintptr_t>(grads[i].out), g = reinterpret_cast<uintptr_t>(grads[i].grad);
    r[n++] = Range{o, o + bytes, true};
    if (g != o) r[n++] = Range{g, g + bytes, false};
  }
  std::sort(r.get(), r.get() + n, [](const Range& a, const Range& b) { return a.begin < b.begin; });
  uintptr_t end_out = 0, end_any = 0;
  for (size_t i = 0; i < n; ++i) {
    CHECK(r[i].begin >= end_out && (!r[i].out || r[i].begin >= end_any), MOE_ERR_INVALID_VALUE,
          "an out overlaps another tensor of the list");
    end_any = std::max(end_any, r[i].end);
    if (r[i].out) end_out = std::max(end_out, r[i].end);
  }
  return MOE_OK;
}

moe_status_t check_max_norm(float max_norm) {
  CHECK(max_norm > 0.0f, MOE_ERR_INVALID_VALUE, "max_norm must be > 0");
  return MOE_OK;
}

// Partial sums, and one double for a total behind them.
size_t grad_ws_bytes(long long chunks) { return align256(((size_t)chunks + 1) * sizeof(double)); }

}  // namespace

size_t moe_grad_workspace_size(const moe_grad_t* grads, int32_t count) {
  GradList list;
  if (grad_list(grads, count, false, list) != MOE_OK) return 0;
  return grad_ws_bytes(list.chunks);
}

moe_status_t moe_grad_norm(const moe_grad_t* grads, int32_t count, double* sumsq, float* norm, void* ws,
                           size_t ws_bytes, moe_stream_t stream) {
  g_err.clear();
  GradList list;
  moe_status_t st = grad_list(grads, count, false, list);
  if (st != MOE_OK) return st;
  CHECK(sumsq, MOE_ERR_INVALID_VALUE, "sumsq is NULL");
  const size_t need = grad_ws_bytes(list.chunks);
  CHECK(ws && ws_bytes >= need, MOE_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need,
        ws ? ws_bytes : (size_t)0);
  CHECK_ALIGN16(sumsq, norm, ws);
  double* partial = reinterpret_cast<double*>(ws);
  st = hip_check(moe::launch_grad_sumsq(list.items.get(), count, partial, S(stream)), "gradient sum of squares");
  if (st != MOE_OK) return st;
  return hip_check(moe::launch_grad_total(partial, (int)list.chunks, sumsq, norm, S(stream)), "gradient norm");
}

moe_status_t moe_grad_scale(const moe_grad_t* grads, int32_t count, const double* sumsq, float max_norm, float* norm,
                            moe_stream_t stream) {
  g_err.clear();
  GradList list;
  moe_status_t st = grad_list(grads, count, true, list);
  if (st != MOE_OK) return st;
  if ((st = check_max_norm(max_norm)) != MOE_OK) return st;
  CHECK(sumsq, MOE_ERR_INVALID_VALUE, "sumsq is NULL");
  CHECK_ALIGN16(sumsq, norm);
  if (list.chunks == 0) {   // nothing to scale: the norm alone
    if (!norm) return MOE_OK;
    return hip_check(moe::launch_grad_total(sumsq, 1, nullptr, norm, S(stream)), "gradient norm");
  }
  return hip_check(moe::launch_grad_scale(list.items.get(), count, const_cast<double*>(sumsq), 1, max_norm, norm, S(stream)),
                   "gradient scaling");
}

moe_status_t moe_grad_clip(const moe_grad_t* grads, int32_t count, float max_norm, float* norm, void* ws,
                           size_t ws_bytes, moe_stream_t stream) {
  g_err.clear();
  GradList list;
  moe_status_t st = grad_list(grads, count, true, list);
  if (st != MOE_OK) return st;
  if ((st = check_max_norm(max_norm)) != MOE_OK) return st;
  const size_t need = grad_ws_bytes(list.chunks);
  CHECK(ws && ws_bytes >= need, MOE_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need,
        ws ? ws_bytes : (size_t)0);
  CHECK_ALIGN16(norm, ws);
  double* partial = reinterpret_cast<double*>(ws);
  if (list.chunks == 0) {   // no elements: a norm of zero
    if (!norm) return MOE_OK;
    return hip_check(moe::launch_grad_total(partial, 0, nullptr, norm, S(stream)), "gradient norm");
  }
  st = hip_check(moe::launch_grad_sumsq(list.items.get(), count, partial, S(stream)), "gradient sum of squares");
  if (st != MOE_OK) return st;
  return hip_check(moe::launch_grad_scale(list.items.get(), count, partial, (int)list.chunks, max_norm, norm, S(stream)),
                   "gradient scaling");
}

// ---------------------------------------------------------------------------------------------
// MXFP8

moe_status_t moe_mx_quantize_rows(const void* x, int64_t R, int64_t K, int64_t ldx, uint8_t* codes,
                                  uint8_t* scales, moe_stream_t stream) {
  g_err.clear();
  CHECK(R >= 0 && K > 0, MOE_ERR_INVALID_VALUE, "R must be >= 0 and K > 0 (got R=%lld, K=%lld)", (long long)R,
        (long long)K);
  CHECK(K % 32 == 0, MOE_ERR_UNSUPPORTED, "K must be a multiple of 32 (got %lld)", (long long)K);
  CHECK(ldx >= K && ldx % 8 == 0, MOE_ERR_INVALID_VALUE, "ldx must be >= K and a multiple of 8 (got %lld)",
        (long long)ldx);
  CHECK(K <= kMaxInt && R <= kMaxInt, MOE_ERR_UNSUPPORTED, "R and K must fit in int32");
  if (R == 0) return MOE_OK;
  CHECK(x && codes && scales, MOE_ERR_INVALID_VALUE, "x/codes/scales is NULL");
  CHECK_ALIGN16(x, codes, scales);
  return hip_check(moe::launch_mx_quant_rows(x, R, (int)K, ldx, codes, scales, S(stream)), "MXFP8 row quantization");
}

int64_t moe_mx_quantize_cols_ld(int64_t R, int32_t G, int32_t kpad) {
  if (R < 0 || G <= 0 || kpad <= 0) return 0;
  // Only a non-empty group adds padding, at most kpad - 1 rows.
  return (R + std::min<int64_t>(G, R) * (kpad - 1)) / kpad * kpad;
}

moe_status_t moe_mx_quantize_cols(const void* x, int64_t R, int64_t N, int64_t ldx, const int32_t* offsets,
                                  int32_t G, int64_t group_rows, int32_t kpad, uint8_t* codes, uint8_t* scales,
                                  int64_t ldc, int32_t* kbase, moe_stream_t stream) {
  g_err.clear();
  CHECK(R >= 0 && N > 0, MOE_ERR_INVALID_VALUE, "R must be >= 0 and N > 0");
  CHECK(N % 2 == 0 && ldx >= N && ldx % 2 == 0, MOE_ERR_UNSUPPORTED, "N and ldx must be even, ldx >= N");
  CHECK(G > 0 && G <= 1024, MOE_ERR_INVALID_VALUE, "G must be in [1, 1024] (got %d)", G);
  CHECK(kpad > 0 && kpad % 128 == 0, MOE_ERR_UNSUPPORTED, "kpad must be a positive multiple of 128 (got %d)",
        kpad);
  CHECK(ldc % 128 == 0 && ldc >= 0, MOE_ERR_INVALID_VALUE, "ldc must be a multiple of 128 (got %lld)",
        (long long)ldc);
  CHECK(R <= kMaxInt && N <= kMaxInt && ldc <= kMaxInt, MOE_ERR_UNSUPPORTED, "sizes must fit in int32");
  int64_t need;
  if (offsets) {
    need = moe_mx_quantize_cols_ld(R, G, kpad);
  } else {
    CHECK(group_rows >= 0 && R == (int64_t)G * group_rows, MOE_ERR_INVALID_VALUE,
          "without offsets R must equal G * group_rows (got R=%lld, G=%d, group_rows=%lld)", (long long)R, G,
          (long long)group_rows);
    need = (int64_t)G * ((group_rows + kpad - 1) / kpad * kpad);
  }
  CHECK(ldc >= need, MOE_ERR_INVALID_VALUE, "ldc must be >= %lld (got %lld)", (long long)need, (long long)ldc);
  CHECK(kbase && (ldc == 0 || (codes && scales)), MOE_ERR_INVALID_VALUE, "kbase/codes/scales is NULL");
  CHECK(R == 0 || x, MOE_ERR_INVALID_VALUE, "x is NULL");
  CHECK_ALIGN16(x, offsets, codes, scales, kbase);
  return hip_check(moe::launch_mx_quant_cols(x, R, (int)N, ldx, offsets, G, group_rows, kpad, codes, scales, ldc,
                                             kbase, S(stream)),
                   "MXFP8 column quantization");
}

size_t moe_mx_gemm_workspace_size(int32_t G) {
  if (G <= 0) return 0;
  return align256((size_t)(G + 1) * sizeof(int32_t));
}

moe_status_t moe_mx_gemm_rows(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes,
                              const uint8_t* b_scales, int64_t b_row_stride, int64_t b_group_stride,
                              const uint8_t* b2_codes, const uint8_t* b2_scales, int64_t b2_k, const int32_t* offsets,
                              int32_t G, int64_t M, int64_t N, int64_t K, int32_t epilogue, void* out0, void* out1,
                              void* out2, const void* aux0, const void* aux1, uint8_t* q_codes, uint8_t* q_scales,
                              void* ws, size_t ws_bytes, moe_stream_t stream) {
  g_err.clear();
  CHECK(epilogue >= MOE_MX_EPI_STORE && epilogue <= MOE_MX_EPI_SWIGLU_BWD, MOE_ERR_INVALID_VALUE,
        "unknown epilogue %d", epilogue);
  CHECK(G > 0 && G <= 1024, MOE_ERR_INVALID_VALUE, "G must be in [1, 1024] (got %d)", G);
  CHECK(M >= 0 && N > 0 && K > 0, MOE_ERR_INVALID_VALUE, "M must be >= 0, N and K > 0");
  const int oc = epilogue == MOE_MX_EPI_SWIGLU ? 64 : 128;
  CHECK(K % 128 == 0 && N % oc == 0, MOE_ERR_UNSUPPORTED, "K must be a multiple of 128 and N of %d", oc);
  // Columns one source holds: all K, or the two parts of a K split.
  const int64_t span = (b2_codes && epilogue != MOE_MX_EPI_SWIGLU) ? std::max<int64_t>(b2_k, K - b2_k) : K;
  CHECK(b_row_stride >= span && b_row_stride % 128 == 0 && b_group_stride >= 0 && b_group_stride % 128 == 0,
        MOE_ERR_INVALID_VALUE, "B strides must be multiples of 128, the row stride >= the columns of a source");
  CHECK(M <= kMaxInt && N <= kMaxInt / 2 && K <= kMaxInt, MOE_ERR_UNSUPPORTED, "sizes must fit in int32");
  CHECK(((M + 127) / 128 + G) * (N / oc) < kMaxInt, MOE_ERR_UNSUPPORTED, "grid too large");
  CHECK(a_codes && a_scales && b_codes && b_scales && offsets, MOE_ERR_INVALID_VALUE, "an operand pointer is NULL");
  CHECK((b2_codes == nullptr) == (b2_scales == nullptr), MOE_ERR_INVALID_VALUE,
        "b2_codes and b2_scales must both be given or both be NULL");
  if (epilogue == MOE_MX_EPI_SWIGLU) {
    CHECK(b2_codes, MOE_ERR_INVALID_VALUE, "the SwiGLU epilogue needs the up-projection rows in b2");
  } else if (b2_codes) {
    CHECK(b2_k > 0 && b2_k < K && b2_k % 128 == 0, MOE_ERR_INVALID_VALUE,
          "b2_k must be a multiple of 128 in (0, K) (got %lld)", (long long)b2_k);
  }
  if (epilogue == MOE_MX_EPI_STORE) CHECK(out0, MOE_ERR_INVALID_VALUE, "out0 is NULL");
  if (epilogue == MOE_MX_EPI_SWIGLU) CHECK(out2, MOE_ERR_INVALID_VALUE, "out2 is NULL");
  if (epilogue == MOE_MX_EPI_SWIGLU_BWD) CHECK(out0 && aux0 && aux1, MOE_ERR_INVALID_VALUE, "out0/aux0/aux1 is NULL");
  CHECK((q_codes == nullptr) == (q_scales == nullptr), MOE_ERR_INVALID_VALUE,
        "q_codes and q_scales must both be given or both be NULL");
  CHECK(!q_codes || epilogue != MOE_MX_EPI_STORE, MOE_ERR_INVALID_VALUE,
        "quantized outputs are produced by the SwiGLU epilogues only");
  const size_t need = moe_mx_gemm_workspace_size(G);
  CHECK(ws && ws_bytes >= need, MOE_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need,
        ws ? ws_bytes : (size_t)0);
  if (M == 0) return MOE_OK;
  CHECK_ALIGN16(a_codes, a_scales, b_codes, b_scales, b2_codes, b2_scales, offsets, out0, out1, out2, aux0, aux1, q_codes, q_scales, ws);
  moe::MxGemmArgs a{};
  a.a = a_codes;
  a.as = a_scales;
  a.lda = K;
  a.b = b_codes;
  a.bs = b_scales;
  a.ldb = b_row_stride;
  a.b_gstride = b_group_stride;
  a.b2 = b2_codes;
  a.bs2 = b2_scales;
  a.ksplit = (epilogue != MOE_MX_EPI_SWIGLU && b2_codes) ? (int)b2_k : 0;
  a.kparts = 1;
  a.offsets = offsets;
  a.tile_prefix = reinterpret_cast<int32_t*>(ws);
  a.G = G;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.out0 = out0;
  a.out1 = out1;
  a.out2 = out2;
  a.aux0 = aux0;
  a.aux1 = aux1;
  a.qc = q_codes;
  a.qs = q_scales;
  return hip_check(moe::launch_mx_gemm(epilogue, false, a, S(stream)), "MXFP8 grouped GEMM (rows)");
}

size_t moe_mx_gemm_k_workspace_size(int32_t G, int64_t M, int64_t N) {
  if (G <= 0 || M <= 0 || N <= 0 || M > kMaxInt || N > kMaxInt || G > 1024) return 0;
  return moe::mx_k_workspace_bytes(G, (int)M, (int)N);
}

moe_status_t moe_mx_gemm_k(const uint8_t* a_codes, const uint8_t* a_scales, int64_t lda, const uint8_t* b_codes,
                           const uint8_t* b_scales, int64_t ldb, const int32_t* kbase, int32_t G, int64_t M,
                           int64_t N, int64_t split, void* out0, void* out1, void* ws, size_t ws_bytes,
                           moe_stream_t stream) {
  g_err.clear();
  CHECK(G > 0 && G <= 1024, MOE_ERR_INVALID_VALUE, "G must be in [1, 1024] (got %d)", G);
  CHECK(M > 0 && N > 0 && split >= 0 && split <= M, MOE_ERR_INVALID_VALUE, "M, N must be > 0, split in [0, M]");
  CHECK(M % 128 == 0 && N % 128 == 0, MOE_ERR_UNSUPPORTED, "M and N must be multiples of 128");
  CHECK(lda > 0 && ldb > 0 && lda % 128 == 0 && ldb % 128 == 0, MOE_ERR_INVALID_VALUE,
        "lda and ldb must be positive multiples of 128");
  CHECK(M <= kMaxInt && N <= kMaxInt && lda <= kMaxInt && ldb <= kMaxInt, MOE_ERR_UNSUPPORTED,
        "sizes must fit in int32");
  CHECK((int64_t)G * (M / 128) * (N / 128) < kMaxInt, MOE_ERR_UNSUPPORTED, "grid too large");
  CHECK(a_codes && a_scales && b_codes && b_scales && kbase, MOE_ERR_INVALID_VALUE, "an operand pointer is NULL");
  CHECK((split == 0 || out0) && (split == M || out1), MOE_ERR_INVALID_VALUE, "out0/out1 is NULL");
  const size_t need = moe::mx_k_workspace_bytes(G, (int)M, (int)N);
  CHECK(need == 0 || (ws && ws_bytes >= need), MOE_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need,
        ws ? ws_bytes : (size_t)0);
  CHECK_ALIGN16(a_codes, a_scales, b_codes, b_scales, kbase, out0, out1, ws);
  moe::MxGemmArgs a{};
  a.a = a_codes;
  a.as = a_scales;
  a.lda = lda;
  a.b = b_codes;
  a.bs = b_scales;
  a.ldb = ldb;
  a.offsets = kbase;
  a.G = G;
  a.M = (int)M;
  a.N = (int)N;
  a.out0 = out0;
  a.out1 = out1;
  a.split = (int)split;
  a.kparts = moe::mx_k_parts(G, (int)M, (int)N);
  a.partial = reinterpret_cast<float*>(ws);
  return hip_check(moe::launch_mx_gemm(MOE_MX_EPI_STORE, true, a, S(stream)), "MXFP8 grouped GEMM (K)");
}

// ---------------------------------------------------------------------------------------------
// Routing by scores

namespace {

moe_status_t check_scores(int32_t score, int32_t renormalize, float scale) {
  CHECK(score == MOE_SCORE_SOFTMAX || score == MOE_SCORE_SIGMOID, MOE_ERR_INVALID_VALUE,
        "score must be MOE_SCORE_SOFTMAX or MOE_SCORE_SIGMOID (got %d)", score);
  CHECK(renormalize == 0 || renormalize == 1, MOE_ERR_INVALID_VALUE, "renormalize must be 0 or 1");
  CHECK(std::isfinite(scale), MOE_ERR_INVALID_VALUE, "scale must be finite");
  return MOE_OK;
}

bool dense_scores(int32_t score, int32_t renormalize) {
  return moe::route_scores_dense(score == MOE_SCORE_SIGMOID, renormalize != 0);
}

moe::RouteScores route_scores(const float* logits, const float* bias, int64_t T, int32_t E, int32_t k, int32_t groups,
                              int32_t topk_groups, int32_t score, int32_t renormalize, float scale) {
  moe::RouteScores r{};
  r.logits = logits;
  r.bias = bias;
  r.T = (int)T;
  r.E = E;
  r.k = k;
  r.groups = groups;
  r.topk_groups = topk_groups;
  r.sigmoid = score == MOE_SCORE_SIGMOID;
  r.renormalize = renormalize != 0;
  r.scale = scale;
  return r;
}

}  // namespace

moe_status_t moe_route_balanced(const void* x, const void* w_router, float* logits, const float* select_bias,
                                int64_t T, int64_t d, int32_t E, int32_t k, int32_t groups, int32_t topk_groups,
                                int32_t score, int32_t renormalize, float scale, moe_dtype_t dt, int32_t* topk_idx,
                                float* topk_gate, moe_stream_t stream) {
  g_err.clear();
  moe_status_t st = check_dtype(dt);
  if (st != MOE_OK) return st;
  if ((st = check_tokens(T, d, E, k)) != MOE_OK) return st;
  if ((st = check_scores(score, renormalize, scale)) != MOE_OK) return st;
  CHECK(groups >= 1 && E % groups == 0, MOE_ERR_INVALID_VALUE, "groups must divide E (got groups=%d, E=%d)", groups, E);
  CHECK(topk_groups >= 1 && topk_groups <= groups, MOE_ERR_INVALID_VALUE,
        "topk_groups must be in [1, groups] (got %d of %d)", topk_groups, groups);
  CHECK(k <= topk_groups * (E / groups), MOE_ERR_INVALID_VALUE, "k = %d, but %d open groups have %d experts", k,
        topk_groups, topk_groups * (E / groups));
  CHECK(moe::route_scores_fits(T, E), MOE_ERR_UNSUPPORTED, "T = %lld is too large for a launch", (long long)T);
  CHECK(!w_router || x, MOE_ERR_INVALID_VALUE, "x is NULL with a learned router");
  if (T == 0) return MOE_OK;
  CHECK(logits && topk_idx && topk_gate, MOE_ERR_INVALID_VALUE, "logits/topk_idx/topk_gate is NULL");
  CHECK_ALIGN16(x, w_router, logits, select_bias, topk_idx, topk_gate);
  if (w_router) {
    st = hip_check(moe::launch_router_logits(x, w_router, nullptr, logits, (int)T, (int)d, E, dt == MOE_BF16, S(stream)),
                   "router logits");
    if (st != MOE_OK) return st;
  }
  return hip_check(moe::launch_route_scores(route_scores(logits, select_bias, T, E, k, groups, topk_groups, score,
                                                         renormalize, scale),
                                            topk_idx, topk_gate, S(stream)),
                   "routing by scores");
}

size_t moe_route_balanced_bwd_workspace_size(int64_t T, int64_t d, int32_t E, int32_t k, int32_t score,
                                             int32_t renormalize) {
  if (check_tokens(T, d, E, k) != MOE_OK || check_scores(score, renormalize, 1.0f) != MOE_OK) return 0;
  return moe::route_scores_bwd_ws_bytes(T, d, E, k, dense_scores(score, renormalize));
}

moe_status_t moe_route_balanced_bwd(const float* dgate, const float* logits, const int32_t* topk_idx,
                                    const int32_t* offsets, const int32_t* src_row, const void* x,
                                    const void* w_router, int64_t T, int64_t d, int32_t E, int32_t k, int32_t score,
                                    int32_t renormalize, float scale, moe_dtype_t dt, float* dw_router,
                                    void* dx_router, void* ws, size_t ws_bytes, moe_stream_t stream) {
  g_err.clear();
  moe_status_t st = check_dtype(dt);
  if (st != MOE_OK) return st;
  if ((st = check_tokens(T, d, E, k)) != MOE_OK) return st;
  if ((st = check_scores(score, renormalize, scale)) != MOE_OK) return st;
  const bool dense = dense_scores(score, renormalize);
  CHECK(!dense || d % 8 == 0, MOE_ERR_UNSUPPORTED,
        "softmax scores without renormalization need d %% 8 == 0 (got %lld)", (long long)d);
  CHECK(moe::route_scores_bwd_fits(T, d, E, k, dense, dt == MOE_BF16), MOE_ERR_UNSUPPORTED,
        "T = %lld and d = %lld are too large for a launch", (long long)T, (long long)d);
  CHECK(dw_router && offsets && w_router, MOE_ERR_INVALID_VALUE, "dw_router/offsets/w_router is NULL");
  CHECK(T == 0 || (dgate && logits && topk_idx && src_row && x && dx_router), MOE_ERR_INVALID_VALUE,
        "dgate/logits/topk_idx/src_row/x/dx_router is NULL");
  const size_t need = moe::route_scores_bwd_ws_bytes(T, d, E, k, dense);
  CHECK(ws && ws_bytes >= need, MOE_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need,
        ws ? ws_bytes : (size_t)0);
  CHECK_ALIGN16(dgate, logits, topk_idx, offsets, src_row, x, w_router, dw_router, dx_router, ws);
  return hip_check(moe::launch_route_scores_bwd(route_scores(logits, nullptr, T, E, k, 1, 1, score, renormalize, scale),
                                                dgate, topk_idx, offsets, src_row, x, w_router, (int)d, dt == MOE_BF16,
                                                dw_router, dx_router, ws, S(stream)),
                   "backward of routing by scores");
}

moe_status_t moe_route_bias_update(const int32_t* counts, int32_t E, float rate, const float* bias, float* bias_out,
                                   moe_stream_t stream) {
  g_err.clear();
  CHECK(E > 0, MOE_ERR_INVALID_VALUE, "E must be > 0 (got %d)", E);
  CHECK(E <= 256, MOE_ERR_UNSUPPORTED, "E > 256 is not supported (got %d)", E);
  CHECK(std::isfinite(rate), MOE_ERR_INVALID_VALUE, "rate must be finite");
  CHECK(counts && bias && bias_out, MOE_ERR_INVALID_VALUE, "counts/bias/bias_out is NULL");
  CHECK_ALIGN16(counts, bias, bias_out);
  return hip_check(moe::launch_route_bias(counts, E, rate, bias, bias_out, S(stream)), "bias update");
}

// ---------------------------------------------------------------------------------------------
// Products in 8-bit floating point, a scale for each block of 128

moe_status_t moe_fp8_quantize_rows(const void* x, int64_t R, int64_t K, int64_t ldx, uint8_t* codes, float* scales,
                                   moe_stream_t stream) {
  g_err.clear();
  CHECK(R >= 0 && K > 0, MOE_ERR_INVALID_VALUE, "R must be >= 0 and K > 0 (got R=%lld, K=%lld)", (long long)R,
        (long long)K);
  CHECK(K % 128 == 0, MOE_ERR_UNSUPPORTED, "K must be a multiple of 128 (got %lld)", (long long)K);
  CHECK(ldx >= K && ldx % 8 == 0, MOE_ERR_INVALID_VALUE, "ldx must be >= K and a multiple of 8 (got %lld)",
        (long long)ldx);
  CHECK(K <= kMaxInt && R <= kMaxInt && ldx <= kMaxInt, MOE_ERR_UNSUPPORTED, "R, K and ldx must fit in int32");
  if (R == 0) return MOE_OK;
  CHECK(x && codes && scales, MOE_ERR_INVALID_VALUE, "x/codes/scales is NULL");
  CHECK_ALIGN16(x, codes, scales);
  return hip_check(moe::launch_fp8_quant_rows(x, R, (int)K, ldx, codes, scales, S(stream)), "8-bit row quantization");
}

moe_status_t moe_fp8_quantize_weights(const void* w, int32_t G, int64_t N, int64_t K, uint8_t* codes, float* scales,
                                      uint8_t* codes_t, float* scales_t, moe_stream_t stream) {
  g_err.clear();
  CHECK(G > 0 && N > 0 && K > 0, MOE_ERR_INVALID_VALUE, "G, N and K must be > 0");
  CHECK(N % 128 == 0 && K % 128 == 0, MOE_ERR_UNSUPPORTED, "N and K must be multiples of 128 (got N=%lld, K=%lld)",
        (long long)N, (long long)K);
  CHECK(N <= kMaxInt && K <= kMaxInt && (N / 128) * (K / 128) <= (1 << 23) / G, MOE_ERR_UNSUPPORTED,
        "more than 2^23 blocks");
  CHECK(w && codes && scales, MOE_ERR_INVALID_VALUE, "w/codes/scales is NULL");
  CHECK((codes_t == nullptr) == (scales_t == nullptr), MOE_ERR_INVALID_VALUE,
        "codes_t and scales_t must both be given or both be NULL");
  CHECK_ALIGN16(w, codes, scales, codes_t, scales_t);
  return hip_check(moe::launch_fp8_quant_weights(w, G, (int)N, (int)K, codes, scales, codes_t, scales_t, S(stream)),
                   "8-bit weight quantization");
}

namespace {

moe_status_t check_fp8_sizes(int32_t G, int64_t M, int64_t N, int64_t K) {
  CHECK(G > 0 && G <= 1024, MOE_ERR_INVALID_VALUE, "G must be in [1, 1024] (got %d)", G);
  CHECK(M >= 0 && N > 0 && K > 0, MOE_ERR_INVALID_VALUE, "M must be >= 0, N and K > 0");
  CHECK(N % 128 == 0 && K % 128 == 0, MOE_ERR_UNSUPPORTED, "N and K must be multiples of 128 (got N=%lld, K=%lld)",
        (long long)N, (long long)K);
  CHECK(M <= kMaxInt / 2 && N <= 1 << 20 && K <= 1 << 20, MOE_ERR_UNSUPPORTED, "sizes out of the supported range");
  CHECK(((M + 127) / 128 + G) * (N / 64) < (1 << 24), MOE_ERR_UNSUPPORTED, "more than 2^24 output tiles");
  return MOE_OK;
}

}  // namespace

size_t moe_fp8_gemm_workspace_size(int32_t G, int64_t M, int64_t N, int64_t K) {
  check_fp8_sizes(G, M, N, K);
  return 0;   // no product needs one yet
}

moe_status_t moe_fp8_gemm_rows(const uint8_t* a_codes, const float* a_scales, const uint8_t* b_codes,
                               const float* b_scales, const uint8_t* b2_codes, const float* b2_scales, int64_t b2_k,
                               const int32_t* offsets, int32_t G, int64_t M, int64_t N, int64_t K, int32_t epilogue,
                               void* out0, void* out1, void* out2, const void* aux0, const void* aux1, void* ws,
                               size_t ws_bytes, moe_stream_t stream) {
  g_err.clear();
  CHECK(epilogue >= MOE_MX_EPI_STORE && epilogue <= MOE_MX_EPI_SWIGLU_BWD, MOE_ERR_INVALID_VALUE,
        "unknown epilogue %d", epilogue);
  moe_status_t st = check_fp8_sizes(G, M, N, K);
  if (st != MOE_OK) return st;
  CHECK((b2_codes == nullptr) == (b2_scales == nullptr), MOE_ERR_INVALID_VALUE,
        "b2_codes and b2_scales must both be given or both be NULL");
  if (epilogue == MOE_MX_EPI_SWIGLU) {
    CHECK(b2_codes, MOE_ERR_INVALID_VALUE, "the SwiGLU epilogue needs the up-projection rows in b2");
  } else if (b2_codes) {
    CHECK(b2_k > 0 && b2_k < K && b2_k % 128 == 0, MOE_ERR_INVALID_VALUE,
          "b2_k must be a multiple of 128 in (0, K) (got %lld)", (long long)b2_k);
  }
  (void)ws_bytes;   // none is needed yet
  if (M == 0) return MOE_OK;
  CHECK(a_codes && a_scales && b_codes && b_scales && offsets, MOE_ERR_INVALID_VALUE, "an operand pointer is NULL");
  if (epilogue == MOE_MX_EPI_STORE) CHECK(out0, MOE_ERR_INVALID_VALUE, "out0 is NULL");
  if (epilogue == MOE_MX_EPI_SWIGLU) CHECK(out2, MOE_ERR_INVALID_VALUE, "out2 is NULL");
  if (epilogue == MOE_MX_EPI_SWIGLU_BWD)
    CHECK(out0 && aux0 && aux1, MOE_ERR_INVALID_VALUE, "out0/aux0/aux1 is NULL");
  CHECK_ALIGN16(a_codes, a_scales, b_codes, b_scales, b2_codes, b2_scales, offsets, out0, out1, out2, aux0, aux1, ws);
  moe::Fp8GemmArgs a{};
  a.a = a_codes;
  a.as = a_scales;
  a.b = b_codes;
  a.bs = b_scales;
  a.b2 = b2_codes;
  a.bs2 = b2_scales;
  a.ksplit = (epilogue != MOE_MX_EPI_SWIGLU && b2_codes) ? (int)b2_k : 0;
  a.offsets = offsets;
  a.G = G;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.out0 = out0;
  a.out1 = out1;
  a.out2 = out2;
  a.aux0 = aux0;
  a.aux1 = aux1;
  return hip_check(moe::launch_fp8_gemm(epilogue, a, S(stream)), "8-bit grouped GEMM");
}

// ---------------------------------------------------------------------------------------------
// AdamW

namespace {

// One bijective round of the hash that the kernel's random bits come from.
uint32_t mix32(uint32_t h) {
  h ^= h >> 16;
  h *= 0x9D2B4F35u;
  h ^= h >> 15;
  h *= 0xC5A1E6B7u;
  return h ^ (h >> 16);
}

constexpr int64_t kAdamWMost = int64_t(1) << 34;   // elements of a tensor: runs of 8 are counted in 32 bits

moe_status_t check_adamw(const moe_adamw_t* t, int32_t count, int32_t state_bits) {
  CHECK(count >= 0, MOE_ERR_INVALID_VALUE, "count must be >= 0 (got %d)", count);
  CHECK(count == 0 || t, MOE_ERR_INVALID_VALUE, "tensors is NULL");
  CHECK(count <= 1 << 20, MOE_ERR_UNSUPPORTED, "count must be at most 2^20 (got %d)", count);
  CHECK(state_bits == 32 || state_bits == 8, MOE_ERR_INVALID_VALUE, "state_bits must be 32 or 8 (got %d)", state_bits);
  int64_t total = 0;
  for (int i = 0; i < count; ++i) {
    const moe_adamw_t& a = t[i];
    moe_status_t st = check_dtype(a.dt);
    if (st == MOE_OK) st = check_dtype(a.grad_dt);
    if (st != MOE_OK) return st;
    CHECK(a.n >= 0, MOE_ERR_INVALID_VALUE, "tensor %d has n = %lld", i, (long long)a.n);
    CHECK(a.n <= kAdamWMost, MOE_ERR_UNSUPPORTED, "tensor %d has more than 2^34 elements", i);
    CHECK(a.n <= kGradMaxElements - total, MOE_ERR_UNSUPPORTED, "more than 2^41 elements");
    total += a.n;
    CHECK(a.weight_decay >= 0 && std::isfinite(a.weight_decay), MOE_ERR_INVALID_VALUE,
          "tensor %d: weight_decay must be finite and >= 0", i);
    if (a.n == 0) continue;
    CHECK((a.param || a.master) && a.grad && a.m && a.v && a.param_out && a.m_out && a.v_out, MOE_ERR_INVALID_VALUE,
          "tensor %d: param/grad/m/v or an out is NULL", i);
    const bool scaled = state_bits == 8;
    CHECK((a.scale != nullptr) == scaled && (a.scale_out != nullptr) == scaled, MOE_ERR_INVALID_VALUE,
          "tensor %d: scale and scale_out go with 8-bit states, and only with them", i);
    CHECK((a.master == nullptr) == (a.master_out == nullptr), MOE_ERR_INVALID_VALUE,
          "tensor %d: master and master_out must both be given or both be NULL", i);
    CHECK(!a.master || a.dt == MOE_BF16, MOE_ERR_INVALID_VALUE, "tensor %d: a float parameter has no master copy", i);
    CHECK(aligned16({a.param, a.grad, a.m, a.v, a.scale, a.master, a.param_out, a.m_out, a.v_out, a.scale_out,
                     a.master_out}),
          MOE_ERR_INVALID_VALUE, "device pointers must be 16-byte aligned (tensor %d)", i);
  }
  return MOE_OK;
}

}  // namespace

moe_status_t moe_adamw_check(const moe_adamw_t* tensors, int32_t count, int32_t state_bits) {
  g_err.clear();
  moe_status_t st = check_adamw(tensors, count, state_bits);
  if (st != MOE_OK) return st;
  // Address ranges in order of their starts, with the furthest end of an output and of any range so far;
  // an output in the place of its input is one range.
  struct Range {
    uintptr_t begin, end;
    bool out;
  };
  std::unique_ptr<Range[]> r(new (std::nothrow) Range[11 * (size_t)std::max(count, 1)]);
  CHECK(r, MOE_ERR_UNSUPPORTED, "no host memory for a list of %d tensors", count);
  size_t n = 0;
  for (int i = 0; i < count; ++i) {
    const moe_adamw_t& a = tensors[i];
    if (a.n == 0) continue;
    const size_t state = (size_t)a.n * (state_bits / 8), blocks = 2 * (((size_t)a.n + 127) / 128) * sizeof(float);
    auto add = [&](const void* in, const void* out, size_t bytes) {
      const uintptr_t o = reinterpret_cast<uintptr_t>(out), p = reinterpret_cast<uintptr_t>(in);
      if (out) r[n++] = Range{o, o + bytes, true};
      if (in && in != out) r[n++] = Range{p, p + bytes, false};
    };
    add(a.param, a.param_out, (size_t)a.n * esize(a.dt));
    add(a.grad, nullptr, (size_t)a.n * esize(a.grad_dt));
    add(a.m, a.m_out, state);
    add(a.v, a.v_out, state);
    add(a.scale, a.scale_out, blocks);
    add(a.master, a.master_out, (size_t)a.n * sizeof(float));
  }
  std::sort(r.get(), r.get() + n, [](const Range& a, const Range& b) { return a.begin < b.begin; });
  uintptr_t end_out = 0, end_any = 0;
  for (size_t i = 0; i < n; ++i) {
    CHECK(r[i].begin >= end_out && (!r[i].out || r[i].begin >= end_any), MOE_ERR_INVALID_VALUE,
          "an out overlaps another tensor of the list");
    end_any = std::max(end_any, r[i].end);
    if (r[i].out) end_out = std::max(end_out, r[i].end);
  }
  return MOE_OK;
}

moe_status_t moe_adamw(const moe_adamw_t* tensors, int32_t count, const moe_adamw_step_t* step, const double* sumsq,
                       float max_norm, moe_stream_t stream) {
  g_err.clear();
  CHECK(step, MOE_ERR_INVALID_VALUE, "step is NULL");
  moe_status_t st = check_adamw(tensors, count, step->state_bits);
  if (st != MOE_OK) return st;
  CHECK(step->lr >= 0 && std::isfinite(step->lr), MOE_ERR_INVALID_VALUE, "lr must be finite and >= 0");
  CHECK(step->beta1 >= 0 && step->beta1 < 1 && step->beta2 >= 0 && step->beta2 < 1, MOE_ERR_INVALID_VALUE,
        "beta1 and beta2 must be in [0, 1)");
  CHECK((float)step->eps >= 1.17549435e-38f && std::isfinite((float)step->eps), MOE_ERR_INVALID_VALUE,
        "eps must be a normal float > 0");
  CHECK(step->step >= 1, MOE_ERR_INVALID_VALUE, "step must be >= 1 (got %lld)", (long long)step->step);
  const float step_size = (float)(step->lr / (1.0 - std::pow(step->beta1, (double)step->step)));
  CHECK(std::isfinite(step_size), MOE_ERR_INVALID_VALUE, "lr / (1 - beta1^step) must be finite as a float");
  if (sumsq && (st = check_max_norm(max_norm)) != MOE_OK) return st;
  CHECK_ALIGN16(sumsq);
  if (count == 0) return MOE_OK;
  std::unique_ptr<moe::AdamWItem[]> items(new (std::nothrow) moe::AdamWItem[count]);
  CHECK(items, MOE_ERR_UNSUPPORTED, "no host memory for a list of %d tensors", count);
  for (int i = 0; i < count; ++i) {
    const moe_adamw_t& a = tensors[i];
    CHECK(std::isfinite((float)(step->lr * a.weight_decay)), MOE_ERR_INVALID_VALUE,
          "tensor %d: lr weight_decay must be finite as a float", i);
    items[i] = moe::AdamWItem{a.param,     a.grad,       a.m,          a.v,
                              a.scale,     a.master,     a.param_out,  a.m_out,
                              a.v_out,     a.scale_out,  a.master_out, (long long)a.n,
                              a.dt == MOE_BF16, a.grad_dt == MOE_BF16, (float)(1.0 - step->lr * a.weight_decay),
                              mix32(step->seed + 0x9E3779B9u * (uint32_t)(i + 1))};
  }
  moe::AdamWStep s{};
  s.beta1 = (float)step->beta1;
  s.one_minus_beta1 = (float)(1.0 - step->beta1);
  s.beta2 = (float)step->beta2;
  s.one_minus_beta2 = (float)(1.0 - step->beta2);
  s.inv_sqrt_bc2 = (float)(1.0 / std::sqrt(1.0 - std::pow(step->beta2, (double)step->step)));
  s.step_size = step_size;
  s.eps = (float)step->eps;
  s.sumsq = sumsq;
  s.max_norm = max_norm;
  return hip_check(moe::launch_adamw(items.get(), count, s, step->state_bits == 8, S(stream)), "AdamW");
}

// ---------------------------------------------------------------------------------------------

size_t moe_workspace_bytes(int32_t op, int64_t T, int64_t d, int32_t E, int32_t k, int64_t f, int64_t fs) {
  g_err.clear();
  if (check_tokens(T, d, E, k) != MOE_OK) return 0;
  if (f <= 0 || fs < 0) {
    fail(MOE_ERR_INVALID_VALUE, "f must be > 0 and fs >= 0 (got f=%lld, fs=%lld)", (long long)f, (long long)fs);
    return 0;
  }
  const int64_t Tk = T * k;
  // The routed experts and (fs > 0) the shared expert as expert sets, sizes only.
  moe_expert_set_t sets[2] = {};
  sets[0].G = E;
  sets[0].M = Tk;
  sets[0].f = f;
  sets[1].G = 1;
  sets[1].M = T;
  sets[1].f = fs;
  const int nsets = fs > 0 ? 2 : 1;
  switch (op) {
    case MOE_OP_ROUTE:
    case MOE_OP_COMBINE:
    case MOE_OP_COMBINE_BWD:
    case MOE_OP_PERMUTE_BWD: return 0;
    case MOE_OP_PERMUTE: return moe_permute_workspace_size(T, E, k);
    case MOE_OP_GROUPED_MLP_FWD: return moe_grouped_mlp_fwd_workspace_size(Tk, E, d, f);
    case MOE_OP_GROUPED_MLP_BWD: return moe_grouped_mlp_bwd_workspace_size(Tk, E, d, f);
    case MOE_OP_ROUTE_BWD: return moe_route_bwd_workspace_size(T, d, E, k);
    case MOE_OP_EXPERT_STAGE: return moe_expert_stage_workspace_size(sets, nsets, d);
    case MOE_OP_ROUTER_AUX: return moe_router_aux_workspace_size(T, E);
    case MOE_OP_ROUTER_AUX_BWD: return moe_router_aux_bwd_workspace_size(T, d, E);
    case MOE_OP_MX_GEMM_ROWS: return moe_mx_gemm_workspace_size(E);
    case MOE_OP_MX_GEMM_K: {
      size_t need = std::max(moe_mx_gemm_k_workspace_size(E, d, f), moe_mx_gemm_k_workspace_size(E, 2 * f, d));
      if (fs > 0)
        need = std::max(need, std::max(moe_mx_gemm_k_workspace_size(1, d, fs),
                                       moe_mx_gemm_k_workspace_size(1, 2 * fs, d)));
      return need;
    }
    case MOE_OP_NORM_BWD: return moe_norm_bwd_workspace_size(T, d);
    case MOE_OP_ROUTE_BALANCED_BWD:
      return std::max(moe_route_balanced_bwd_workspace_size(T, d, E, k, MOE_SCORE_SIGMOID, 1),
                      moe_route_balanced_bwd_workspace_size(T, d, E, k, MOE_SCORE_SOFTMAX, 0));
    case MOE_OP_FP8_GEMM_ROWS: {
      size_t need = 0;
      for (int q = 0; q < nsets; ++q) {
        const moe_expert_set_t& e = sets[q];
        need = std::max({need, moe_fp8_gemm_workspace_size(e.G, e.M, e.f, d), moe_fp8_gemm_workspace_size(e.G, e.M, d, e.f),
                         moe_fp8_gemm_workspace_size(e.G, e.M, d, 2 * e.f)});
      }
      return need;
    }
    default:
      fail(MOE_ERR_INVALID_VALUE, "unknown op %d", op);
      return 0;
  }
}

}  // extern "C"
