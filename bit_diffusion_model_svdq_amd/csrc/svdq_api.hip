// C ABI entry points for the device side: argument validation, workspace
// carving, kernel dispatch.  Host-side packing lives in pack.cpp.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <atomic>
#include <mutex>

#include "svdq_internal.h"

namespace svdq {

static thread_local char g_err[512] = "";

svdq_status fail(svdq_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return st;
}

svdq_status hip_check(hipError_t e, const char* what) {
  if (e == hipSuccess) return SVDQ_OK;
  return fail(SVDQ_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

int device_cu_count() {
  static std::atomic<int> cached[64];   // zero-initialized: 0 = not read yet
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
      n = 256;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

static size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

WorkspaceLayout workspace_layout(int M, int K, int N, int r) {
  WorkspaceLayout l;
  const size_t qx_bytes = align256((size_t)M * (K / 2));
  const size_t sx_bytes = align256((size_t)M * (K / kGroup) * 4);
  l.t_slices = k1_plan(M, K, r, false).slices;
  const size_t t_bytes = align256((size_t)l.t_slices * M * r * 4);
  const size_t part_bytes = N > 0 ? align256(gemm_split_bytes(M, K, N)) : 0;
  l.qx = 0;
  l.sx = qx_bytes;
  l.T = qx_bytes + sx_bytes;
  l.part = part_bytes ? qx_bytes + sx_bytes + t_bytes : 0;
  l.bytes = qx_bytes + sx_bytes + t_bytes + part_bytes;
  return l;
}

Workspace carve_workspace(void* base, int M, int K, int N, int r) {
  const WorkspaceLayout l = workspace_layout(M, K, N, r);
  uint8_t* p = static_cast<uint8_t*>(base);
  Workspace w;
  w.qx = p + l.qx;
  w.sx = reinterpret_cast<float*>(p + l.sx);
  w.T = r > 0 ? reinterpret_cast<float*>(p + l.T) : nullptr;
  w.t_slices = l.t_slices;
  w.part = l.part ? reinterpret_cast<float*>(p + l.part) : nullptr;
  w.bytes = l.bytes;
  return w;
}

// MXFP4 workspace: qx [M, K/2] | sx k-tiled E8M0 bytes [ceil(K/256)][sx_rows][8]
// | T [slices, M, r].
WorkspaceLayout workspace_layout_mx(int M, int K, int N, int r) {
  WorkspaceLayout l;
  l.sx_rows = (M + 1) & ~1;
  const size_t qx_bytes = align256((size_t)M * (K / 2));
  const size_t sx_bytes = align256((size_t)((K + 255) / 256) * l.sx_rows * 8);
  l.t_slices = k1_plan(M, K, r, false).slices;
  const size_t t_bytes = align256((size_t)l.t_slices * M * r * 4);
  const size_t part_bytes = N > 0 ? align256(mxfp4_gemm_split_bytes(M, K, N)) : 0;
  l.qx = 0;
  l.sx = qx_bytes;
  l.T = qx_bytes + sx_bytes;
  l.part = part_bytes ? qx_bytes + sx_bytes + t_bytes : 0;
  l.bytes = qx_bytes + sx_bytes + t_bytes + part_bytes;
  return l;
}

MxWorkspace carve_workspace_mx(void* base, int M, int K, int N, int r) {
  const WorkspaceLayout l = workspace_layout_mx(M, K, N, r);
  uint8_t* p = static_cast<uint8_t*>(base);
  MxWorkspace w;
  w.sx_rows = l.sx_rows;
  w.qx = p + l.qx;
  w.sx = p + l.sx;
  w.T = r > 0 ? reinterpret_cast<float*>(p + l.T) : nullptr;
  w.t_slices = l.t_slices;
  w.part = l.part ? reinterpret_cast<float*>(p + l.part) : nullptr;
  w.bytes = l.bytes;
  return w;
}

}  // namespace svdq

using namespace svdq;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The largest K a one-slice quantize launch stages in LDS (a multiple of 128,
// so it holds for MXFP4 too); include/svdq.h states the same bound.
constexpr int kMaxCanonicalK = 12544;

svdq_status check_shapes(int M, int K, int N, int r, bool need_n) {
  if (M < 1) return fail(SVDQ_ERR_INVALID_ARG, "M must be >= 1 (got %d)", M);
  if (K < kGroup || K % kGroup != 0)
    return fail(SVDQ_ERR_INVALID_ARG, "K must be a positive multiple of 64 (got %d)", K);
  if (need_n && (N < 16 || N % 16 != 0))
    return fail(SVDQ_ERR_INVALID_ARG, "N must be a positive multiple of 16 (got %d)", N);
  if (r < 0 || r > kMaxRank || r % 16 != 0)
    return fail(SVDQ_ERR_INVALID_ARG, "rank must be a multiple of 16 in [0, 128] (got %d)", r);
  return SVDQ_OK;
}

// MXFP4: the block-scaled MFMA takes 128 channels per step
svdq_status check_shapes_mx(int M, int K, int N, int r) {
  if (K < 128 || K % 128 != 0)
    return fail(SVDQ_ERR_INVALID_ARG, "K must be a positive multiple of 128 for MXFP4 (got %d)", K);
  return check_shapes(M, K, N, r, true);
}

svdq_status check_ptr(const void* p, const char* name, bool may_be_null) {
  if (!p) {
    if (may_be_null) return SVDQ_OK;
    return fail(SVDQ_ERR_INVALID_ARG, "%s must not be NULL", name);
  }
  if (!aligned16(p)) return fail(SVDQ_ERR_ALIGNMENT, "%s is not 16-byte aligned", name);
  return SVDQ_OK;
}

#define SVDQ_TRY(expr)                   \
  do {                                   \
    const svdq_status st_ = (expr);      \
    if (st_ != SVDQ_OK) return st_;      \
  } while (0)

svdq_status stage1_checks(const uint16_t* X, int M, int K, int r, const float* smooth,
                          const uint16_t* L1) {
  SVDQ_TRY(check_ptr(X, "X", false));
  SVDQ_TRY(check_ptr(smooth, "smooth", false));
  SVDQ_TRY(check_ptr(L1, "L1", r == 0));
  (void)M;
  (void)K;
  return SVDQ_OK;
}

svdq_status stage2_checks(int r, const uint16_t* L2, const uint8_t* Wq, const float* w_scales,
                          const uint16_t* bias, const uint16_t* Y) {
  SVDQ_TRY(check_ptr(L2, "L2", r == 0));
  SVDQ_TRY(check_ptr(Wq, "Wq", false));
  SVDQ_TRY(check_ptr(w_scales, "w_scales", false));
  SVDQ_TRY(check_ptr(bias, "bias", true));
  SVDQ_TRY(check_ptr(Y, "Y", false));
  return SVDQ_OK;
}

template <class F>
svdq_status guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return fail(SVDQ_ERR_INVALID_ARG, "unexpected C++ exception");
  }
}

svdq_status check_act(int act) {
  if (act != kActNone && act != kActGeluTanh)
    return fail(SVDQ_ERR_INVALID_ARG, "activation %d is not one of svdq_activation", act);
  return SVDQ_OK;
}

svdq_status forward_gemm(int M, int K, int N, int r, const uint16_t* L2, const uint8_t* Wq,
                         const float* w_scales, const uint16_t* bias, int act, uint16_t* Y,
                         const void* workspace, size_t workspace_bytes, void* stream) {
  SVDQ_TRY(check_shapes(M, K, N, r, true));
  SVDQ_TRY(stage2_checks(r, L2, Wq, w_scales, bias, Y));
  SVDQ_TRY(check_act(act));
  SVDQ_TRY(check_ptr(workspace, "workspace", false));
  const Workspace w = carve_workspace(const_cast<void*>(workspace), M, K, N, r);
  if (workspace_bytes < w.bytes)
    return fail(SVDQ_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", w.bytes, workspace_bytes);
  return hip_check(launch_w4a4_gemm(w.qx, w.sx, w.T, w.t_slices, M, K, N, r, L2, Wq, w_scales,
                                    bias, Y, w.part, act, static_cast<hipStream_t>(stream)),
                   "w4a4_gemm launch");
}

svdq_status linear_forward(const uint16_t* X, int M, int K, int N, int r, const float* smooth,
                           const uint16_t* L1, const uint16_t* L2, const uint8_t* Wq,
                           const float* w_scales, const uint16_t* bias, int act, uint16_t* Y,
                           void* workspace, size_t workspace_bytes, void* stream) {
  // validate everything before launching anything
  SVDQ_TRY(check_shapes(M, K, N, r, true));
  SVDQ_TRY(stage1_checks(X, M, K, r, smooth, L1));
  SVDQ_TRY(stage2_checks(r, L2, Wq, w_scales, bias, Y));
  SVDQ_TRY(check_act(act));
  SVDQ_TRY(check_ptr(workspace, "workspace", false));
  const Workspace w = carve_workspace(workspace, M, K, N, r);
  if (workspace_bytes < w.bytes)
    return fail(SVDQ_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", w.bytes, workspace_bytes);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const FusedPlan fp = fused_plan(M, K, N, r);
  if (fp.use)
    return hip_check(launch_fused_smallk(fp, X, M, K, N, r, smooth, L1, L2, Wq, w_scales, bias, Y,
                                         act, nullptr, nullptr, s),
                     "fused small-K forward launch");
  SVDQ_TRY(hip_check(launch_smooth_quant_lora_down(X, M, K, r, smooth, L1, w.qx, w.sx, w.T, false, s),
                     "smooth_quant_lora_down launch"));
  return hip_check(launch_w4a4_gemm(w.qx, w.sx, w.T, w.t_slices, M, K, N, r, L2, Wq, w_scales,
                                    bias, Y, w.part, act, s),
                   "w4a4_gemm launch");
}

svdq_status forward_gemm_mx(int M, int K, int N, int r, const uint16_t* L2, const uint8_t* Wq,
                            const uint8_t* w_e8m0, const uint16_t* bias, int act, uint16_t* Y,
                            const void* workspace, size_t workspace_bytes, void* stream) {
  SVDQ_TRY(check_shapes_mx(M, K, N, r));
  SVDQ_TRY(stage2_checks(r, L2, Wq, reinterpret_cast<const float*>(w_e8m0), bias, Y));
  SVDQ_TRY(check_act(act));
  SVDQ_TRY(check_ptr(workspace, "workspace", false));
  const MxWorkspace w = carve_workspace_mx(const_cast<void*>(workspace), M, K, N, r);
  if (workspace_bytes < w.bytes)
    return fail(SVDQ_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", w.bytes, workspace_bytes);
  return hip_check(launch_mxfp4_gemm(w.qx, w.sx, w.sx_rows, w.T, w.t_slices, M, K, N, r, L2, Wq,
                                     w_e8m0, bias, Y, w.part, act, static_cast<hipStream_t>(stream)),
                   "mxfp4_gemm launch");
}

svdq_status linear_forward_mx(const uint16_t* X, int M, int K, int N, int r, const float* smooth,
                              const uint16_t* L1, const uint16_t* L2, const uint8_t* Wq,
                              const uint8_t* w_e8m0, const uint16_t* bias, int act, uint16_t* Y,
                              void* workspace, size_t workspace_bytes, void* stream) {
  SVDQ_TRY(check_shapes_mx(M, K, N, r));
  SVDQ_TRY(stage1_checks(X, M, K, r, smooth, L1));
  SVDQ_TRY(stage2_checks(r, L2, Wq, reinterpret_cast<const float*>(w_e8m0), bias, Y));
  SVDQ_TRY(check_act(act));
  SVDQ_TRY(check_ptr(workspace, "workspace", false));
  const MxWorkspace w = carve_workspace_mx(workspace, M, K, N, r);
  if (workspace_bytes < w.bytes)
    return fail(SVDQ_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", w.bytes, workspace_bytes);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const FusedPlan fp = fused_plan_mx(M, K, N, r);
  if (fp.use)
    return hip_check(launch_fused_smallk_mx(fp, X, M, K, N, r, smooth, L1, L2, Wq, w_e8m0, bias, Y,
                                            act, nullptr, nullptr, s),
                     "fused small-K forward (MXFP4) launch");
  SVDQ_TRY(hip_check(launch_smooth_quant_lora_down_mx(X, M, K, r, smooth, L1, w.qx, w.sx, w.T,
                                                      false, w.sx_rows, s),
                     "smooth_quant_lora_down (MXFP4) launch"));
  return hip_check(launch_mxfp4_gemm(w.qx, w.sx, w.sx_rows, w.T, w.t_slices, M, K, N, r, L2, Wq,
                                     w_e8m0, bias, Y, w.part, act, s),
                   "mxfp4_gemm launch");
}

// ---- attention
// Most workgroups of a launch: the runtime takes fewer than 2^32 work-items,
// and no kernel here has more than 512 per workgroup.
constexpr int64_t kMaxBlocks = (int64_t(1) << 23) - 1;
// Heads that svdq_qk_norm_rope_forward counts in 32 bits, with their steps.
constexpr int kMaxHeads = 1 << 20;
// Sequences whose offsets a kernel looks up 64 at a time, in 32 bits.
constexpr int kMaxBatch = INT32_MAX - 512;

svdq_status check_batch(int batch) {
  if (batch < 1 || batch > kMaxBatch)
    return fail(SVDQ_ERR_INVALID_ARG, "batch must be 1 to %d (got %d)", kMaxBatch, batch);
  return SVDQ_OK;
}

svdq_status check_attention_shape(int batch, int64_t total_q, int64_t total_k, int heads_q, int heads_kv,
                                  int head_dim, bool count_blocks = true) {
  SVDQ_TRY(check_batch(batch));
  if (total_q < 0 || total_k < 0)
    return fail(SVDQ_ERR_INVALID_ARG, "negative total_q=%lld or total_k=%lld", (long long)total_q,
                (long long)total_k);
  if (heads_kv < 1 || heads_q < heads_kv || heads_q % heads_kv)
    return fail(SVDQ_ERR_INVALID_ARG, "heads_q=%d must be a positive multiple of heads_kv=%d", heads_q, heads_kv);
  if (head_dim < 8 || head_dim % 8)
    return fail(SVDQ_ERR_INVALID_ARG, "head_dim must be a positive multiple of 8 (got %d)", head_dim);
  if (head_dim > 128) return fail(SVDQ_ERR_UNSUPPORTED, "head_dim %d is above 128", head_dim);
  // the kernels count rows and keys in 32 bits: up to the end of a tile that the last one
  // begins (rows), and of the four tiles that are copied or looked at ahead (keys)
  if (total_q > INT32_MAX || total_k > INT32_MAX - 512 || total_q * (heads_q / heads_kv) > INT32_MAX - 512)
    return fail(SVDQ_ERR_INVALID_ARG, "total_q=%lld (times %d heads a group) or total_k=%lld is beyond 31 bits less 512",
                (long long)total_q, heads_q / heads_kv, (long long)total_k);
  if (count_blocks && total_q > 0 && attention_blocks((int)total_q, (int)total_k, batch, heads_q, heads_kv, head_dim) > kMaxBlocks)
    return fail(SVDQ_ERR_INVALID_ARG, "too many rows for one launch: total_q=%lld, heads_q=%d, batch=%d",
                (long long)total_q, heads_q, batch);
  return SVDQ_OK;
}

svdq_status check_ld(int64_t ld, int64_t width, const char* name) {
  if (ld < width || ld % 8)
    return fail(SVDQ_ERR_INVALID_ARG, "%s=%lld must be a multiple of 8 and at least %lld", name, (long long)ld,
                (long long)width);
  return SVDQ_OK;
}

svdq_status check_align4(const void* p, const char* name) {
  if (reinterpret_cast<uintptr_t>(p) & 3) return fail(SVDQ_ERR_ALIGNMENT, "%s is not 4-byte aligned", name);
  return SVDQ_OK;
}

// What every attention call has besides its shape.
svdq_status check_attention_call(const AttentionArgs& a) {
  if (!(a.scale > 0.f) || a.scale > 0x1p126f)      // the kernels take scale log2(e)
    return fail(SVDQ_ERR_INVALID_ARG, "scale must be positive and at most 2^126 (got %g)", (double)a.scale);
  if (a.causal != 0 && a.causal != 1) return fail(SVDQ_ERR_INVALID_ARG, "causal must be 0 or 1 (got %d)", a.causal);
  if (a.batch > 1 && (!a.cu_q || !a.cu_k))
    return fail(SVDQ_ERR_INVALID_ARG, "cu_q and cu_k must not be NULL for batch=%d", a.batch);
  const int64_t wq = (int64_t)a.heads_q * a.head_dim, wk = (int64_t)a.heads_kv * a.head_dim;
  SVDQ_TRY(check_ld(a.ldq, wq, "ldq"));
  SVDQ_TRY(check_ld(a.ldk, wk, "ldk"));
  SVDQ_TRY(check_ld(a.ldv, wk, "ldv"));
  SVDQ_TRY(check_ld(a.ldo, wq, "ldo"));
  if (a.ldk > kAttentionMaxLd || a.ldv > kAttentionMaxLd)
    return fail(SVDQ_ERR_UNSUPPORTED, "ldk=%lld or ldv=%lld is above 2^24", (long long)a.ldk, (long long)a.ldv);
  SVDQ_TRY(check_ptr(a.Q, "Q", a.total_q == 0));
  SVDQ_TRY(check_ptr(a.K, "K", a.total_k == 0 || a.total_q == 0));
  SVDQ_TRY(check_ptr(a.V, "V", a.total_k == 0 || a.total_q == 0));
  SVDQ_TRY(check_ptr(a.O, "O", a.total_q == 0));
  SVDQ_TRY(check_align4(a.cu_q, "cu_q"));
  SVDQ_TRY(check_align4(a.cu_k, "cu_k"));
  return check_align4(a.lse, "lse");
}

svdq_status check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (need == 0) return SVDQ_OK;
  SVDQ_TRY(check_ptr(workspace, "workspace", false));
  if (bytes < need) return fail(SVDQ_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, bytes);
  return SVDQ_OK;
}

// The shape of an attention call whose keys lie in two pieces, and its plan.
svdq_status check_spans_shape(const SpanArgs& a, int64_t total_q, int64_t total_k, int64_t prefix, SpanPlan& plan) {
  if (prefix < 0 || prefix > INT32_MAX - 512)
    return fail(SVDQ_ERR_INVALID_ARG, "the prefix' %lld keys are negative or beyond 31 bits less 512", (long long)prefix);
  SVDQ_TRY(check_attention_shape(a.batch, total_q, total_k, a.heads_q, a.heads_kv, a.head_dim, false));
  if (total_k + prefix > INT32_MAX - 512)
    return fail(SVDQ_ERR_INVALID_ARG, "total_k=%lld and the prefix' %lld keys are beyond 31 bits less 512",
                (long long)total_k, (long long)prefix);
  if (a.left < -1 || a.right < -1)
    return fail(SVDQ_ERR_INVALID_ARG, "window_left=%d and window_right=%d must be -1 or more", a.left, a.right);
  if (a.sinks < 0) return fail(SVDQ_ERR_INVALID_ARG, "sinks must not be negative (got %d)", a.sinks);
  if (total_q == 0) return SVDQ_OK;
  plan = plan_attention_spans(a);
  if (plan.most_blocks > kMaxBlocks)
    return fail(SVDQ_ERR_INVALID_ARG, "too many rows for one launch: total_q=%lld, heads_q=%d, batch=%d",
                (long long)total_q, a.heads_q, a.batch);
  return SVDQ_OK;
}

SpanArgs spans_of(int batch, int64_t total_q, int64_t total_k, int heads_q, int heads_kv, int head_dim, int causal,
                  int left, int right, int sinks, int64_t prefix) {
  SpanArgs a = {};
  a.batch = batch; a.total_q = (int)total_q; a.total_k = (int)total_k;
  a.heads_q = heads_q; a.heads_kv = heads_kv; a.head_dim = head_dim;
  a.causal = causal;
  a.left = left; a.right = right; a.sinks = sinks;
  a.prefix = (int)prefix;
  return a;
}

// ---- block norms and the 16-bit linear
svdq_status check_dtype(int dtype, const char* name) {
  if (dtype != SVDQ_BF16 && dtype != SVDQ_F32)
    return fail(SVDQ_ERR_INVALID_ARG, "%s %d is not one of svdq_dtype", name, dtype);
  return SVDQ_OK;
}

svdq_status check_norm(int kind, const char* name) {
  if (kind != kNormNone && kind != kNormRms && kind != kNormLayer)
    return fail(SVDQ_ERR_INVALID_ARG, "%s %d is not one of svdq_norm", name, kind);
  return SVDQ_OK;
}

svdq_status check_linear_shape(int64_t M, int K, int N) {
  if (M < 0 || M > INT32_MAX - 512)
    return fail(SVDQ_ERR_INVALID_ARG, "M=%lld is negative or beyond 31 bits", (long long)M);
  if (K < 8 || K % 8 || K > INT32_MAX - 512)
    return fail(SVDQ_ERR_INVALID_ARG, "K must be a positive multiple of 8 (got %d)", K);
  if (N < 1 || N > INT32_MAX - 512) return fail(SVDQ_ERR_INVALID_ARG, "N must be positive (got %d)", N);
  if (M > 0 && linear_blocks((int)M, K, N) > kMaxBlocks)
    return fail(SVDQ_ERR_INVALID_ARG, "M=%lld x N=%d is too much for one launch", (long long)M, N);
  return SVDQ_OK;
}

// ---- the allocation-free forward's workspace
// A file-scope device array serves as the forward's workspace for callers
// that cannot allocate.  Host code never uses the array's name as an address
// (on the host it only names the symbol); the device address comes from
// hipGetSymbolAddress, once per device, with that device current.
constexpr size_t kScratchBytes = size_t(64) << 20;
__device__ __align__(256) uint8_t scratch[kScratchBytes];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mutex;
void* g_scratch_ptr[kMaxDevices] = {};

svdq_status scratch_for_current_device(void** out) {
  int dev = 0;
  SVDQ_TRY(hip_check(hipGetDevice(&dev), "hipGetDevice"));
  if (dev < 0 || dev >= kMaxDevices)
    return fail(SVDQ_ERR_UNSUPPORTED, "device %d is beyond the %d the library tracks", dev, kMaxDevices);
  std::lock_guard<std::mutex> lock(g_scratch_mutex);
  if (!g_scratch_ptr[dev]) {
    void* ptr = nullptr;
    SVDQ_TRY(hip_check(hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch)), "hipGetSymbolAddress(scratch)"));
    if (!ptr) return fail(SVDQ_ERR_HIP, "hipGetSymbolAddress(scratch) returned NULL");
    g_scratch_ptr[dev] = ptr;
  }
  *out = g_scratch_ptr[dev];
  return SVDQ_OK;
}

}  // namespace

extern "C" {

size_t svdq_static_workspace_bytes(void) { return kScratchBytes; }

svdq_status svdq_linear_forward_noalloc(const uint16_t* X, int M, int K, int N, int r,
                                        const float* smooth, const uint16_t* L1,
                                        const uint16_t* L2, const uint8_t* Wq,
                                        const float* w_scales, const uint16_t* bias,
                                        int activation, uint16_t* Y, void* stream) {
  return guarded([&]() -> svdq_status {
    // the same checks as the workspace entry point, then the size bound
    SVDQ_TRY(check_shapes(M, K, N, r, true));
    const size_t need = workspace_layout(M, K, N, r).bytes;
    if (need > kScratchBytes)
      return fail(SVDQ_ERR_WORKSPACE,
                  "M=%d K=%d N=%d r=%d needs %zu workspace bytes; the static workspace holds %zu",
                  M, K, N, r, need, kScratchBytes);
    void* ws = nullptr;
    SVDQ_TRY(scratch_for_current_device(&ws));
    return linear_forward(X, M, K, N, r, smooth, L1, L2, Wq, w_scales, bias, activation, Y, ws,
                          kScratchBytes, stream);
  });
}

size_t svdq_forward_workspace_bytes(int M, int K, int N, int r) {
  if (M < 1 || K < kGroup || K % kGroup || N < 16 || N % 16 || r < 0 || r > kMaxRank || r % 16)
    return 0;
  return workspace_layout(M, K, N, r).bytes;
}

svdq_status svdq_forward_workspace_layout(int M, int K, int N, int r, size_t* qx_offset,
                                          size_t* sx_offset, size_t* t_offset, int* t_slices) {
  return guarded([&]() -> svdq_status {
    SVDQ_TRY(check_shapes(M, K, N, r, true));
    if (!qx_offset || !sx_offset || !t_offset || !t_slices)
      return fail(SVDQ_ERR_INVALID_ARG, "NULL output pointer");
    const WorkspaceLayout l = workspace_layout(M, K, N, r);
    *qx_offset = l.qx;
    *sx_offset = l.sx;
    *t_offset = r > 0 ? l.T : 0;
    *t_slices = r > 0 ? l.t_slices : 0;
    return SVDQ_OK;
  });
}

svdq_status svdq_forward_workspace_layout_mxfp4(int M, int K, int N, int r, size_t* qx_offset,
                                                size_t* sx_offset, size_t* t_offset, int* t_slices,
                                                int* sx_rows) {
  return guarded([&]() -> svdq_status {
    SVDQ_TRY(check_shapes_mx(M, K, N, r));
    if (!qx_offset || !sx_offset || !t_offset || !t_slices || !sx_rows)
      return fail(SVDQ_ERR_INVALID_ARG, "NULL output pointer");
    const WorkspaceLayout l = workspace_layout_mx(M, K, N, r);
    *qx_offset = l.qx;
    *sx_offset = l.sx;
    *t_offset = r > 0 ? l.T : 0;
    *t_slices = r > 0 ? l.t_slices : 0;
    *sx_rows = l.sx_rows;
    return SVDQ_OK;
  });
}

svdq_status svdq_forward_quantize(const uint16_t* X, int M, int K, int r, const float* smooth,
                                  const uint16_t* L1, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  return guarded([&]() -> svdq_status {
    SVDQ_TRY(check_shapes(M, K, 16, r, false));
    SVDQ_TRY(stage1_checks(X, M, K, r, smooth, L1));
    SVDQ_TRY(check_ptr(workspace, "workspace", false));
    const Workspace w = carve_workspace(workspace, M, K, 0, r);   // stage 1 needs no partials
    if (workspace_bytes < w.bytes)
      return fail(SVDQ_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", w.bytes, workspace_bytes);
    return hip_check(launch_smooth_quant_lora_down(X, M, K, r, smooth, L1, w.qx, w.sx, w.T, false,
                                                   static_cast<hipStream_t>(stream)),
                     "smooth_quant_lora_down launch");
  });
}

svdq_status svdq_forward_gemm(int M, int K, int N, int r, const uint16_t* L2, const uint8_t* Wq,
                              const float* w_scales, const uint16_t* bias, uint16_t* Y,
                              const void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> svdq_status {
    return forward_gemm(M, K, N, r, L2, Wq, w_scales, bias, kActNone, Y, workspace,
                        workspace_bytes, stream);
  });
}

svdq_status svdq_forward_gemm_act(int M, int K, int N, int r, const uint16_t* L2,
                                  const uint8_t* Wq, const float* w_scales, const uint16_t* bias,
                                  int activation, uint16_t* Y, const void* workspace,
                                  size_t workspace_bytes, void* stream) {
  return guarded([&]() -> svdq_status {
    return forward_gemm(M, K, N, r, L2, Wq, w_scales, bias, activation, Y, workspace,
                        workspace_bytes, stream);
  });
}

svdq_status svdq_linear_forward(const uint16_t* X, int M, int K, int N, int r,
                                const float* smooth, const uint16_t* L1, const uint16_t* L2,
                                const uint8_t* Wq, const float* w_scales, const uint16_t* bias,
                                uint16_t* Y, void* workspace, size_t workspace_bytes,
                                void* stream) {
  return guarded([&]() -> svdq_status {
    return linear_forward(X, M, K, N, r, smooth, L1, L2, Wq, w_scales, bias, kActNone, Y,
                          workspace, workspace_bytes, stream);
  });
}

svdq_status svdq_linear_forward_act(const uint16_t* X, int M, int K, int N, int r,
                                    const float* smooth, const uint16_t* L1, const uint16_t* L2,
                                    const uint8_t* Wq, const float* w_scales,
                                    const uint16_t* bias, int activation, uint16_t* Y,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> svdq_status {
    return linear_forward(X, M, K, N, r, smooth, L1, L2, Wq, w_scales, bias, activation, Y,
                          workspace, workspace_bytes, stream);
  });
}

svdq_status svdq_quantize_activations(const uint16_t* X, int M, int K, const float* smooth,
                                      const uint16_t* L1, int r, uint8_t* qx, float* sx,
                                      float* T, void* stream) {
  return guarded([&]() -> svdq_status {
    SVDQ_TRY(check_shapes(M, K, 16, r, false));
    SVDQ_TRY(stage1_checks(X, M, K, r, smooth, L1));
    SVDQ_TRY(check_ptr(qx, "qx", false));
    SVDQ_TRY(check_ptr(sx, "sx", false));
    SVDQ_TRY(check_ptr(T, "T", r == 0));
    if (!k1_one_slice_fits(K, r))
      return fail(SVDQ_ERR_INVALID_ARG,
                  "K=%d: the canonical-layout quantize stages a whole row in LDS and takes K <= %d",
                  K, kMaxCanonicalK);
    return hip_check(launch_smooth_quant_lora_down(X, M, K, r, smooth, L1, qx, sx, T, true,
                                                   static_cast<hipStream_t>(stream)),
                     "smooth_quant_lora_down launch");
  });
}

svdq_status svdq_act_absmax_update_device(const uint16_t* X, int64_t M, int K, float* amax,
                                          void* stream) {
  return guarded([&]() -> svdq_status {
    if (M < 0 || K < 1)
      return fail(SVDQ_ERR_INVALID_ARG, "bad shape M=%lld K=%d", (long long)M, K);
    if (!amax || (M > 0 && !X)) return fail(SVDQ_ERR_INVALID_ARG, "NULL buffer");
    if ((reinterpret_cast<uintptr_t>(X) & 1) || (reinterpret_cast<uintptr_t>(amax) & 3))
      return fail(SVDQ_ERR_ALIGNMENT, "X must be 2-byte and amax 4-byte aligned");
    return hip_check(launch_act_absmax(X, M, K, amax, static_cast<hipStream_t>(stream)),
                     "act_absmax launch");
  });
}

svdq_status svdq_debug_group_partials(const uint8_t* qx, const uint8_t* Wq, int M, int N, int K,
                                      int m0, int m1, int n0, int n1, int32_t* P, void* stream) {
  return guarded([&]() -> svdq_status {
    SVDQ_TRY(check_shapes(M, K, N, 0, true));
    if (m0 < 0 || m1 > M || m0 >= m1 || n0 < 0 || n1 > N || n0 >= n1)
      return fail(SVDQ_ERR_INVALID_ARG, "block [%d,%d)x[%d,%d) outside [0,%d)x[0,%d)", m0, m1, n0,
                  n1, M, N);
    SVDQ_TRY(check_ptr(qx, "qx", false));
    SVDQ_TRY(check_ptr(Wq, "Wq", false));
    SVDQ_TRY(check_ptr(P, "P", false));
    return hip_check(
        launch_group_partials(qx, Wq, M, N, K, m0, m1, n0, n1, P, static_cast<hipStream_t>(stream)),
        "group_partials launch");
  });
}

size_t svdq_attention_workspace_bytes(int64_t total_q, int64_t total_k, int batch, int heads_q, int heads_kv,
                                      int head_dim) {
  if (check_attention_shape(batch, total_q, total_k, heads_q, heads_kv, head_dim) != SVDQ_OK) return 0;
  return attention_workspace((int)total_q, (int)total_k, batch, heads_q, heads_kv, head_dim);
}

svdq_status svdq_attention_forward(const uint16_t* Q, int64_t ldq, const uint16_t* K, int64_t ldk,
                                   const uint16_t* V, int64_t ldv, const int32_t* cu_q, const int32_t* cu_k,
                                   int batch, int64_t total_q, int64_t total_k, int heads_q, int heads_kv,
                                   int head_dim, float scale, int causal, uint16_t* O, int64_t ldo, float* lse,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> svdq_status {
    SVDQ_TRY(check_attention_shape(batch, total_q, total_k, heads_q, heads_kv, head_dim));
    const AttentionArgs a = {Q, K, V, ldq, ldk, ldv, ldo, cu_q, cu_k, batch, (int)total_q, (int)total_k, heads_q,
                             heads_kv, head_dim, scale, causal, O, lse, workspace};
    SVDQ_TRY(check_attention_call(a));
    if (total_q == 0) return SVDQ_OK;
    SVDQ_TRY(check_workspace(workspace, workspace_bytes,
                             attention_workspace(a.total_q, a.total_k, batch, heads_q, heads_kv, head_dim)));
    return hip_check(launch_attention(a, static_cast<hipStream_t>(stream)), "attention launch");
  });
}

size_t svdq_attention_window_workspace_bytes(int64_t total_q, int64_t total_k, int batch, int heads_q, int heads_kv,
                                             int head_dim, int causal, int window_left, int window_right, int sinks) {
  const SpanArgs a = spans_of(batch, total_q, total_k, heads_q, heads_kv, head_dim, causal, window_left, window_right,
                              sinks, 0);
  SpanPlan plan;
  return check_spans_shape(a, total_q, total_k, 0, plan) == SVDQ_OK ? plan.bytes : 0;
}

svdq_status svdq_attention_window_forward(const uint16_t* Q, int64_t ldq, const uint16_t* K, int64_t ldk,
                                          const uint16_t* V, int64_t ldv, const int32_t* cu_q, const int32_t* cu_k,
                                          int batch, int64_t total_q, int64_t total_k, int heads_q, int heads_kv,
                                          int head_dim, float scale, int causal, int window_left, int window_right,
                                          int sinks, uint16_t* O, int64_t ldo, float* lse, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  return guarded([&]() -> svdq_status {
    SpanArgs a = spans_of(batch, total_q, total_k, heads_q, heads_kv, head_dim, causal, window_left, window_right,
                          sinks, 0);
    SpanPlan plan;
    SVDQ_TRY(check_spans_shape(a, total_q, total_k, 0, plan));
    static_cast<AttentionArgs&>(a) = {Q, K, V, ldq, ldk, ldv, ldo, cu_q, cu_k, batch, a.total_q, a.total_k, heads_q,
                                      heads_kv, head_dim, scale, causal, O, lse, workspace};
    SVDQ_TRY(check_attention_call(a));
    if (total_q == 0) return SVDQ_OK;
    SVDQ_TRY(check_workspace(workspace, workspace_bytes, plan.bytes));
    return hip_check(launch_attention_spans(a, plan, static_cast<hipStream_t>(stream)), "attention_window launch");
  });
}

size_t svdq_attention_prefix_workspace_bytes(int64_t total_q, int64_t prefix_len, int64_t total_k, int batch,
                                             int heads_q, int heads_kv, int head_dim, int causal) {
  const SpanArgs a = spans_of(batch, total_q, total_k, heads_q, heads_kv, head_dim, causal, -1, -1, 0, prefix_len);
  SpanPlan plan;
  return check_spans_shape(a, total_q, total_k, prefix_len, plan) == SVDQ_OK ? plan.bytes : 0;
}

svdq_status svdq_attention_prefix_forward(const uint16_t* Q, int64_t ldq, const uint16_t* prefix_K, int64_t ldpk,
                                          const uint16_t* prefix_V, int64_t ldpv, int64_t prefix_len,
                                          const uint16_t* K, int64_t ldk, const uint16_t* V, int64_t ldv,
                                          const int32_t* cu_q, const int32_t* cu_k, int batch, int64_t total_q,
                                          int64_t total_k, int heads_q, int heads_kv, int head_dim, float scale,
                                          int causal, uint16_t* O, int64_t ldo, float* lse, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  return guarded([&]() -> svdq_status {
    SpanArgs a = spans_of(batch, total_q, total_k, heads_q, heads_kv, head_dim, causal, -1, -1, 0, prefix_len);
    SpanPlan plan;
    SVDQ_TRY(check_spans_shape(a, total_q, total_k, prefix_len, plan));
    static_cast<AttentionArgs&>(a) = {Q, K, V, ldq, ldk, ldv, ldo, cu_q, cu_k, batch, a.total_q, a.total_k, heads_q,
                                      heads_kv, head_dim, scale, causal, O, lse, workspace};
    SVDQ_TRY(check_attention_call(a));
    const int64_t wk = (int64_t)heads_kv * head_dim;
    SVDQ_TRY(check_ld(ldpk, wk, "ldpk"));
    SVDQ_TRY(check_ld(ldpv, wk, "ldpv"));
    if (ldpk > kAttentionMaxLd || ldpv > kAttentionMaxLd)
      return fail(SVDQ_ERR_UNSUPPORTED, "ldpk=%lld or ldpv=%lld is above 2^24", (long long)ldpk, (long long)ldpv);
    SVDQ_TRY(check_ptr(prefix_K, "prefix_K", prefix_len == 0 || total_q == 0));
    SVDQ_TRY(check_ptr(prefix_V, "prefix_V", prefix_len == 0 || total_q == 0));
    if (total_q == 0) return SVDQ_OK;
    a.PK = prefix_K;
    a.PV = prefix_V;
    a.ldpk = ldpk;
    a.ldpv = ldpv;
    SVDQ_TRY(check_workspace(workspace, workspace_bytes, plan.bytes));
    return hip_check(launch_attention_spans(a, plan, static_cast<hipStream_t>(stream)), "attention_prefix launch");
  });
}

svdq_status svdq_block_norm_forward(const void* x, int stream_dtype, const uint16_t* y, int64_t rows, int width,
                                    const int32_t* cu, int batch, int post, const uint16_t* post_weight,
                                    const uint16_t* gate, int64_t ld_gate, float residual_scale,
                                    float branch_scale, int pre, const uint16_t* pre_weight,
                                    const uint16_t* pre_bias, const uint16_t* scale, int64_t ld_scale,
                                    const uint16_t* shift, int64_t ld_shift, float eps, void* x_out, uint16_t* h,
                                    void* stream) {
  return guarded([&]() -> svdq_status {
    if (rows < 0 || rows > kMaxBlocks)
      return fail(SVDQ_ERR_INVALID_ARG, "rows=%lld is negative or above %lld", (long long)rows,
                  (long long)kMaxBlocks);
    if (width < 8 || width % 8 || width > kMaxNormWidth)
      return fail(SVDQ_ERR_INVALID_ARG, "width must be a multiple of 8 in [8, %d] (got %d)", kMaxNormWidth, width);
    if (batch < 1) return fail(SVDQ_ERR_INVALID_ARG, "batch must be >= 1 (got %d)", batch);
    if (batch > 1 && !cu) return fail(SVDQ_ERR_INVALID_ARG, "cu must not be NULL for batch=%d", batch);
    SVDQ_TRY(check_dtype(stream_dtype, "stream_dtype"));
    SVDQ_TRY(check_norm(post, "post"));
    SVDQ_TRY(check_norm(pre, "pre"));
    if (!y && (post != kNormNone || post_weight || gate))
      return fail(SVDQ_ERR_INVALID_ARG, "post norm, its weight or a gate without y");
    if (!h && (pre != kNormNone || pre_weight || pre_bias || scale || shift))
      return fail(SVDQ_ERR_INVALID_ARG, "pre norm, its weights or a modulation without h");
    if (!x_out && !h) return fail(SVDQ_ERR_INVALID_ARG, "x_out and h are both NULL");
    if (!(eps >= 0.f) || !isfinite(eps))
      return fail(SVDQ_ERR_INVALID_ARG, "eps must be finite and not negative (got %g)", (double)eps);
    if (!isfinite(residual_scale) || !isfinite(branch_scale))
      return fail(SVDQ_ERR_INVALID_ARG, "residual_scale and branch_scale must be finite");
    if (gate) SVDQ_TRY(check_ld(ld_gate, width, "ld_gate"));
    if (scale) SVDQ_TRY(check_ld(ld_scale, width, "ld_scale"));
    if (shift) SVDQ_TRY(check_ld(ld_shift, width, "ld_shift"));
    SVDQ_TRY(check_ptr(x, "x", rows == 0));
    SVDQ_TRY(check_ptr(y, "y", true));
    SVDQ_TRY(check_ptr(post_weight, "post_weight", true));
    SVDQ_TRY(check_ptr(gate, "gate", true));
    SVDQ_TRY(check_ptr(pre_weight, "pre_weight", true));
    SVDQ_TRY(check_ptr(pre_bias, "pre_bias", true));
    SVDQ_TRY(check_ptr(scale, "scale", true));
    SVDQ_TRY(check_ptr(shift, "shift", true));
    SVDQ_TRY(check_ptr(x_out, "x_out", true));
    SVDQ_TRY(check_ptr(h, "h", true));
    SVDQ_TRY(check_align4(cu, "cu"));
    if (rows == 0) return SVDQ_OK;
    const BlockNormArgs a = {x, y, rows, width, cu, batch, post, post_weight, gate, ld_gate, residual_scale,
                             branch_scale, pre, pre_weight, pre_bias, scale, ld_scale, shift, ld_shift, eps, x_out,
                             h};
    return hip_check(launch_block_norm(a, stream_dtype == SVDQ_F32, static_cast<hipStream_t>(stream)),
                     "block_norm launch");
  });
}

svdq_status svdq_qk_norm_rope_forward(const uint16_t* Q, int64_t ldq, const uint16_t* K, int64_t ldk, int64_t rows,
                                      int heads_q, int heads_k, int head_dim, const int32_t* cu, int batch,
                                      const int32_t* positions, int norm, const uint16_t* q_weight,
                                      const uint16_t* q_bias, const uint16_t* k_weight, const uint16_t* k_bias,
                                      float eps, const float* cos, const float* sin, int64_t ld_table,
                                      int64_t table_rows, int rotary_dim, int pairs, uint16_t* Q_out, int64_t ldqo,
                                      uint16_t* K_out, int64_t ldko, void* stream) {
  return guarded([&]() -> svdq_status {
    if (rows < 0 || rows > INT32_MAX)      // positions and offsets are 32-bit numbers
      return fail(SVDQ_ERR_INVALID_ARG, "rows=%lld is negative or beyond 31 bits", (long long)rows);
    if (heads_q < 0 || heads_k < 0 || (heads_q == 0 && heads_k == 0) || heads_q > kMaxHeads || heads_k > kMaxHeads)
      return fail(SVDQ_ERR_INVALID_ARG, "heads_q=%d and heads_k=%d must be 0 to %d, one of them at least 1", heads_q,
                  heads_k, kMaxHeads);
    if (head_dim < 8 || head_dim % 8)
      return fail(SVDQ_ERR_INVALID_ARG, "head_dim must be a positive multiple of 8 (got %d)", head_dim);
    if (head_dim > kMaxRopeHead) return fail(SVDQ_ERR_UNSUPPORTED, "head_dim %d is above %d", head_dim, kMaxRopeHead);
    SVDQ_TRY(check_batch(batch));
    if (batch > 1 && !cu) return fail(SVDQ_ERR_INVALID_ARG, "cu must not be NULL for batch=%d", batch);
    SVDQ_TRY(check_norm(norm, "norm"));
    if (!(eps >= 0.f) || !isfinite(eps))
      return fail(SVDQ_ERR_INVALID_ARG, "eps must be finite and not negative (got %g)", (double)eps);
    if (rotary_dim < 0 || rotary_dim % 8 || rotary_dim > head_dim)
      return fail(SVDQ_ERR_INVALID_ARG, "rotary_dim must be a multiple of 8 in [0, head_dim] (got %d)", rotary_dim);
    if (pairs != SVDQ_ROPE_NEIGHBOURS && pairs != SVDQ_ROPE_HALVES)
      return fail(SVDQ_ERR_INVALID_ARG, "pairs %d is not one of svdq_rope_pairs", pairs);
    if (rotary_dim > 0) {
      if (table_rows < 0 || ld_table < rotary_dim / 2 || ld_table % 4)
        return fail(SVDQ_ERR_INVALID_ARG,
                    "table_rows=%lld must not be negative, and ld_table=%lld a multiple of 4 and at least %d",
                    (long long)table_rows, (long long)ld_table, rotary_dim / 2);
      SVDQ_TRY(check_ptr(cos, "cos", rows == 0 || table_rows == 0));
      SVDQ_TRY(check_ptr(sin, "sin", rows == 0 || table_rows == 0));
    } else if (cos || sin) {
      return fail(SVDQ_ERR_INVALID_ARG, "cos and sin must be NULL without a rotary_dim");
    }
    const int64_t wq = (int64_t)heads_q * head_dim, wk = (int64_t)heads_k * head_dim;
    if (heads_q > 0) {
      SVDQ_TRY(check_ld(ldq, wq, "ldq"));
      SVDQ_TRY(check_ld(ldqo, wq, "ldqo"));
      if (Q == Q_out && ldq != ldqo) return fail(SVDQ_ERR_INVALID_ARG, "Q_out is Q with another row stride");
      SVDQ_TRY(check_ptr(Q, "Q", rows == 0));
      SVDQ_TRY(check_ptr(Q_out, "Q_out", rows == 0));
    } else if (Q || Q_out || q_weight || q_bias) {
      return fail(SVDQ_ERR_INVALID_ARG, "heads_q=0 with a Q operand");
    }
    if (heads_k > 0) {
      SVDQ_TRY(check_ld(ldk, wk, "ldk"));
      SVDQ_TRY(check_ld(ldko, wk, "ldko"));
      if (K == K_out && ldk != ldko) return fail(SVDQ_ERR_INVALID_ARG, "K_out is K with another row stride");
      SVDQ_TRY(check_ptr(K, "K", rows == 0));
      SVDQ_TRY(check_ptr(K_out, "K_out", rows == 0));
    } else if (K || K_out || k_weight || k_bias) {
      return fail(SVDQ_ERR_INVALID_ARG, "heads_k=0 with a K operand");
    }
    SVDQ_TRY(check_ptr(q_weight, "q_weight", true));
    SVDQ_TRY(check_ptr(q_bias, "q_bias", true));
    SVDQ_TRY(check_ptr(k_weight, "k_weight", true));
    SVDQ_TRY(check_ptr(k_bias, "k_bias", true));
    SVDQ_TRY(check_align4(cu, "cu"));
    SVDQ_TRY(check_align4(positions, "positions"));
    if (rows == 0) return SVDQ_OK;
    const QkNormRopeArgs a = {Q, K, ldq, ldk, rows, heads_q, heads_k, head_dim, cu, batch, positions, norm, q_weight,
                              q_bias, k_weight, k_bias, eps, cos, sin, ld_table, table_rows, rotary_dim,
                              pairs == SVDQ_ROPE_HALVES, Q_out, ldqo, K_out, ldko};
    if (qk_norm_rope_blocks(a) > kMaxBlocks)
      return fail(SVDQ_ERR_INVALID_ARG, "too many rows for one launch: rows=%lld, heads_q=%d, heads_k=%d",
                  (long long)rows, heads_q, heads_k);
    return hip_check(launch_qk_norm_rope(a, static_cast<hipStream_t>(stream)), "qk_norm_rope launch");
  });
}

size_t svdq_linear_bf16_workspace_bytes(int64_t M, int K, int N) {
  if (check_linear_shape(M, K, N) != SVDQ_OK || M == 0) return 0;
  return linear_workspace((int)M, K, N);
}

svdq_status svdq_linear_bf16_forward(const uint16_t* X, int64_t M, int K, int N, const uint16_t* W,
                                     const uint16_t* bias, int activation, const void* residual, void* Y,
                                     int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> svdq_status {
    SVDQ_TRY(check_linear_shape(M, K, N));
    SVDQ_TRY(check_dtype(out_dtype, "out_dtype"));
    if (activation != kActNone && activation != kActGeluTanh && activation != kActSilu)
      return fail(SVDQ_ERR_INVALID_ARG, "activation %d is not one of svdq_activation", activation);
    SVDQ_TRY(check_ptr(X, "X", M == 0));
    SVDQ_TRY(check_ptr(W, "W", M == 0));
    SVDQ_TRY(check_ptr(bias, "bias", true));
    SVDQ_TRY(check_ptr(residual, "residual", true));
    SVDQ_TRY(check_ptr(Y, "Y", M == 0));
    if (M == 0) return SVDQ_OK;
    const size_t need = linear_workspace((int)M, K, N);
    if (need > 0) {
      SVDQ_TRY(check_ptr(workspace, "workspace", false));
      if (workspace_bytes < need)
        return fail(SVDQ_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, workspace_bytes);
    }
    LinearArgs a = {X, W, bias, residual, Y, (int)M, K, N, static_cast<float*>(workspace), 1, 0};
    return hip_check(launch_linear_bf16(a, activation, out_dtype == SVDQ_F32, static_cast<hipStream_t>(stream)),
                     "linear_bf16 launch");
  });
}

int svdq_forward_fused(int M, int K, int N, int r) {
  if (M < 1 || K < kGroup || K % kGroup || N < 16 || N % 16 || r < 0 || r > kMaxRank || r % 16)
    return 0;
  return fused_plan(M, K, N, r).use ? 1 : 0;
}

svdq_status svdq_debug_fused_forward(const uint16_t* X, int M, int K, int N, int r,
                                     const float* smooth, const uint16_t* L1, const uint16_t* L2,
                                     const uint8_t* Wq, const float* w_scales,
                                     const uint16_t* bias, int activation, uint16_t* Y,
                                     uint8_t* qx, float* sx, void* stream) {
  return guarded([&]() -> svdq_status {
    SVDQ_TRY(check_shapes(M, K, N, r, true));
    SVDQ_TRY(stage1_checks(X, M, K, r, smooth, L1));
    SVDQ_TRY(stage2_checks(r, L2, Wq, w_scales, bias, Y));
    SVDQ_TRY(check_act(activation));
    SVDQ_TRY(check_ptr(qx, "qx", false));
    SVDQ_TRY(check_ptr(sx, "sx", false));
    const FusedPlan fp = fused_plan(M, K, N, r);
    if (!fp.use)
      return fail(SVDQ_ERR_INVALID_ARG, "M=%d K=%d N=%d r=%d does not take the fused small-K path", M, K,
                  N, r);
    return hip_check(launch_fused_smallk(fp, X, M, K, N, r, smooth, L1, L2, Wq, w_scales, bias, Y,
                                         activation, qx, sx, static_cast<hipStream_t>(stream)),
                     "fused small-K forward launch");
  });
}

int svdq_forward_fused_mxfp4(int M, int K, int N, int r) {
  if (M < 1 || K < 128 || K % 128 || N < 16 || N % 16 || r < 0 || r > kMaxRank || r % 16) return 0;
  return fused_plan_mx(M, K, N, r).use ? 1 : 0;
}

svdq_status svdq_debug_fused_forward_mxfp4(const uint16_t* X, int M, int K, int N, int r,
                                           const float* smooth, const uint16_t* L1,
                                           const uint16_t* L2, const uint8_t* Wq,
                                           const uint8_t* w_e8m0, const uint16_t* bias,
                                           int activation, uint16_t* Y, uint8_t* qx,
                                           uint8_t* sx_e8m0, void* stream) {
  return guarded([&]() -> svdq_status {
    SVDQ_TRY(check_shapes_mx(M, K, N, r));
    SVDQ_TRY(stage1_checks(X, M, K, r, smooth, L1));
    SVDQ_TRY(stage2_checks(r, L2, Wq, reinterpret_cast<const float*>(w_e8m0), bias, Y));
    SVDQ_TRY(check_act(activation));
    SVDQ_TRY(check_ptr(qx, "qx", false));
    SVDQ_TRY(check_ptr(sx_e8m0, "sx_e8m0", false));
    const FusedPlan fp = fused_plan_mx(M, K, N, r);
    if (!fp.use)
      return fail(SVDQ_ERR_INVALID_ARG, "M=%d K=%d N=%d r=%d does not take the fused small-K path", M, K,
                  N, r);
    return hip_check(launch_fused_smallk_mx(fp, X, M, K, N, r, smooth, L1, L2, Wq, w_e8m0, bias, Y,
                                            activation, qx, sx_e8m0, static_cast<hipStream_t>(stream)),
                     "fused small-K forward (MXFP4) launch");
  });
}

size_t svdq_forward_workspace_bytes_mxfp4(int M, int K, int N, int r) {
  if (M < 1 || K < 128 || K % 128 || N < 16 || N % 16 || r < 0 || r > kMaxRank || r % 16) return 0;
  return workspace_layout_mx(M, K, N, r).bytes;
}

svdq_status svdq_forward_quantize_mxfp4(const uint16_t* X, int M, int K, int r,
                                        const float* smooth, const uint16_t* L1, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  return guarded([&]() -> svdq_status {
    SVDQ_TRY(check_shapes_mx(M, K, 16, r));
    SVDQ_TRY(stage1_checks(X, M, K, r, smooth, L1));
    SVDQ_TRY(check_ptr(workspace, "workspace", false));
    const MxWorkspace w = carve_workspace_mx(workspace, M, K, 0, r);   // stage 1 needs no partials
    if (workspace_bytes < w.bytes)
      return fail(SVDQ_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", w.bytes, workspace_bytes);
    return hip_check(launch_smooth_quant_lora_down_mx(X, M, K, r, smooth, L1, w.qx, w.sx, w.T,
                                                      false, w.sx_rows,
                                                      static_cast<hipStream_t>(stream)),
                     "smooth_quant_lora_down (MXFP4) launch");
  });
}

svdq_status svdq_forward_gemm_mxfp4(int M, int K, int N, int r, const uint16_t* L2,
                                    const uint8_t* Wq, const uint8_t* w_e8m0,
                                    const uint16_t* bias, uint16_t* Y, const void* workspace,
                                    size_t workspace_bytes, void* stream) {
  return guarded([&]() -> svdq_status {
    return forward_gemm_mx(M, K, N, r, L2, Wq, w_e8m0, bias, kActNone, Y, workspace,
                           workspace_bytes, stream);
  });
}

svdq_status svdq_forward_gemm_act_mxfp4(int M, int K, int N, int r, const uint16_t* L2,
                                        const uint8_t* Wq, const uint8_t* w_e8m0,
                                        const uint16_t* bias, int activation, uint16_t* Y,
                                        const void* workspace, size_t workspace_bytes,
                                        void* stream) {
  return guarded([&]() -> svdq_status {
    return forward_gemm_mx(M, K, N, r, L2, Wq, w_e8m0, bias, activation, Y, workspace,
                           workspace_bytes, stream);
  });
}

svdq_status svdq_linear_forward_mxfp4(const uint16_t* X, int M, int K, int N, int r,
                                      const float* smooth, const uint16_t* L1,
                                      const uint16_t* L2, const uint8_t* Wq,
                                      const uint8_t* w_e8m0, const uint16_t* bias, uint16_t* Y,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> svdq_status {
    return linear_forward_mx(X, M, K, N, r, smooth, L1, L2, Wq, w_e8m0, bias, kActNone, Y,
                             workspace, workspace_bytes, stream);
  });
}

svdq_status svdq_linear_forward_act_mxfp4(const uint16_t* X, int M, int K, int N, int r,
                                          const float* smooth, const uint16_t* L1,
                                          const uint16_t* L2, const uint8_t* Wq,
                                          const uint8_t* w_e8m0, const uint16_t* bias,
                                          int activation, uint16_t* Y, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  return guarded([&]() -> svdq_status {
    return linear_forward_mx(X, M, K, N, r, smooth, L1, L2, Wq, w_e8m0, bias, activation, Y,
                             workspace, workspace_bytes, stream);
  });
}

svdq_status svdq_quantize_activations_mxfp4(const uint16_t* X, int M, int K, const float* smooth,
                                            const uint16_t* L1, int r, uint8_t* qx,
                                            uint8_t* sx_e8m0, float* T, void* stream) {
  return guarded([&]() -> svdq_status {
    SVDQ_TRY(check_shapes_mx(M, K, 16, r));
    SVDQ_TRY(stage1_checks(X, M, K, r, smooth, L1));
    SVDQ_TRY(check_ptr(qx, "qx", false));
    SVDQ_TRY(check_ptr(sx_e8m0, "sx_e8m0", false));
    SVDQ_TRY(check_ptr(T, "T", r == 0));
    if (!k1_one_slice_fits(K, r))
      return fail(SVDQ_ERR_INVALID_ARG,
                  "K=%d: the canonical-layout quantize stages a whole row in LDS and takes K <= %d",
                  K, kMaxCanonicalK);
    return hip_check(launch_smooth_quant_lora_down_mx(X, M, K, r, smooth, L1, qx, sx_e8m0, T, true,
                                                      0, static_cast<hipStream_t>(stream)),
                     "smooth_quant_lora_down (MXFP4) launch");
  });
}

const char* svdq_status_string(svdq_status status) {
  // callers may pass any int (the ABI carries the enum as one): read its bytes
  // as an int, since loading an out-of-range value as the enum type is undefined
  int s;
  memcpy(&s, &status, sizeof(s));
  switch (s) {
    case SVDQ_OK: return "ok";
    case SVDQ_ERR_INVALID_ARG: return "invalid argument";
    case SVDQ_ERR_UNSUPPORTED: return "unsupported parameter";
    case SVDQ_ERR_ALIGNMENT: return "misaligned pointer";
    case SVDQ_ERR_WORKSPACE: return "workspace too small";
    case SVDQ_ERR_NO_CONVERGENCE: return "eigensolver did not converge";
    case SVDQ_ERR_HIP: return "HIP runtime error";
  }
  return "unknown status";
}

const char* svdq_last_error(void) { return g_err; }

}  // extern "C"
