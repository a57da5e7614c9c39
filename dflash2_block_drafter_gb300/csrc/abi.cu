// C ABI entry points: host-side validation, workspace carving and dispatch to the kernels.
// Nothing here allocates device memory; every failure returns a status before any launch.
#include <atomic>
#include <chrono>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "internal.h"

namespace dfl {

namespace {
__device__ int g_error_word = 0;  // first device-side error of the current device, 0 if none

thread_local char g_msg[512] = "";

constexpr int kMaxDevices = 64;
int g_err_ptr_ready[kMaxDevices];
int* g_err_ptr[kMaxDevices];
int g_sms[kMaxDevices];
std::mutex g_mu;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// each to its element's type (a kernel's access to one that is not would fault); NULL is
template <typename... T>
bool aligned(const T*... p) {
  return ((reinterpret_cast<uintptr_t>(p) % alignof(T) == 0) && ...);
}
}  // namespace

int fail(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return status;
}

int* device_error_word() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(g_mu);
  if (!g_err_ptr_ready[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_error_word) != cudaSuccess) return nullptr;
    g_err_ptr[dev] = static_cast<int*>(p);
    g_err_ptr_ready[dev] = 1;
  }
  return g_err_ptr[dev];
}

unsigned long long next_call_number() {
  static const unsigned long long seed =
      static_cast<unsigned long long>(std::chrono::high_resolution_clock::now().time_since_epoch().count()) *
      0x9E3779B97F4A7C15ull;
  static std::atomic<unsigned long long> count{0};
  const unsigned long long n = seed + count.fetch_add(1, std::memory_order_relaxed) + 1;
  return n != 0 ? n : 1;
}

int sm_count() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
  std::lock_guard<std::mutex> lock(g_mu);
  if (g_sms[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    g_sms[dev] = n;
  }
  return g_sms[dev];
}

}  // namespace dfl

using namespace dfl;

#define REQUIRE(cond, ...)                                  \
  do {                                                      \
    if (!(cond)) return fail(DFLASH2_ERR_INVALID_ARG, __VA_ARGS__); \
  } while (0)

static int check_conv_shape(int B, int G, int H, int gs, int taps, int dtype) {
  if (taps != 2) return fail(DFLASH2_ERR_UNSUPPORTED, "taps=%d: only the two-tap conv is implemented", taps);
  REQUIRE(dtype == DFLASH2_BF16 || dtype == DFLASH2_F32, "dtype=%d is not DFLASH2_BF16 or DFLASH2_F32", dtype);
  REQUIRE(B >= 1, "B=%d must be >= 1", B);
  REQUIRE(G >= 2 && G <= 64, "G=%d must be in [2, 64] (a block needs at least one draft row)", G);
  REQUIRE(H >= 64 && H % 64 == 0, "H=%d must be a positive multiple of 64", H);
  REQUIRE(gs >= 8 && gs % 8 == 0 && H % gs == 0, "group_size=%d must be a multiple of 8 dividing H=%d", gs, H);
  return DFLASH2_OK;
}

extern "C" {

int dflash2_version(void) { return 100; }

const char* dflash2_status_string(int status) {
  switch (status) {
    case DFLASH2_OK: return "DFLASH2_OK";
    case DFLASH2_ERR_INVALID_ARG: return "DFLASH2_ERR_INVALID_ARG";
    case DFLASH2_ERR_UNSUPPORTED: return "DFLASH2_ERR_UNSUPPORTED";
    case DFLASH2_ERR_CUDA: return "DFLASH2_ERR_CUDA";
    case DFLASH2_ERR_WORKSPACE: return "DFLASH2_ERR_WORKSPACE";
    case DFLASH2_ERR_TIMEOUT: return "DFLASH2_ERR_TIMEOUT";
    case DFLASH2_ERR_BAD_INDEX: return "DFLASH2_ERR_BAD_INDEX";
    default: return "DFLASH2_ERR_UNKNOWN";
  }
}

const char* dflash2_last_error_message(void) { return g_msg; }

int dflash2_poll_error(void* stream) {
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(DFLASH2_ERR_CUDA, "stream synchronize failed: %s", cudaGetErrorString(e));
  int* p = device_error_word();
  if (p == nullptr) return fail(DFLASH2_ERR_CUDA, "no device error word");
  int v = 0;
  e = cudaMemcpy(&v, p, sizeof(int), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return fail(DFLASH2_ERR_CUDA, "reading the error word failed: %s", cudaGetErrorString(e));
  if (v != 0) {
    const int zero = 0;
    e = cudaMemcpy(p, &zero, sizeof(int), cudaMemcpyHostToDevice);
    if (e != cudaSuccess) return fail(DFLASH2_ERR_CUDA, "clearing the error word failed: %s", cudaGetErrorString(e));
    fail(v, "a kernel recorded %s", dflash2_status_string(v));
  }
  return v;
}

size_t dflash2_conv_prepare_workspace_bytes(int B, int G, int H, int group_size, int dtype) {
  if (check_conv_shape(B, G, H, group_size, 2, dtype) != DFLASH2_OK) return 0;
  const ConvShape s{B, G, H, group_size, H / group_size, dtype};
  return conv_prepare_workspace(s, sm_count());
}

int dflash2_conv_prepare_launches(int B, int G, int H, int group_size, int dtype, int with_norm) {
  if (check_conv_shape(B, G, H, group_size, 2, dtype) != DFLASH2_OK) return -1;
  return conv_prepare_kernels(ConvShape{B, G, H, group_size, H / group_size, dtype}, with_norm != 0);
}

int dflash2_conv_finish_launches(int B, int G, int H, int group_size, int dtype, int with_next_norm) {
  if (check_conv_shape(B, G, H, group_size, 2, dtype) != DFLASH2_OK) return -1;
  return conv_finish_kernels(ConvShape{B, G, H, group_size, H / group_size, dtype}, with_next_norm != 0);
}

int dflash2_conv_prepare(const void* x, const void* norm_w, float eps, const void* w_kp, const float* base, int B,
                         int G, int H, int group_size, int taps, int dtype, void* out, void* coef1, float* d_full,
                         void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_conv_shape(B, G, H, group_size, taps, dtype);
  if (rc != DFLASH2_OK) return rc;
  REQUIRE(x && w_kp && base && out && coef1 && workspace, "a required pointer is NULL");
  REQUIRE(aligned16(x) && aligned16(w_kp) && aligned16(base) && aligned16(out) && (!norm_w || aligned16(norm_w)),
          "x, norm_w, w_kp, base and out must be 16-byte aligned");
  REQUIRE((reinterpret_cast<uintptr_t>(workspace) & 255u) == 0, "workspace must be 256-byte aligned");
  const ConvShape s{B, G, H, group_size, H / group_size, dtype};
  const int sms = sm_count();
  const size_t need = conv_prepare_workspace(s, sms);
  if (workspace_bytes < need)
    return fail(DFLASH2_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu bytes needed", workspace_bytes,
                need);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const GemmPlan plan = kp_plan(s, sms);
  const size_t es = dtype == DFLASH2_F32 ? 4 : 2;
  size_t n_bytes = static_cast<size_t>(s.rows()) * H * es;
  n_bytes = (n_bytes + 255) & ~static_cast<size_t>(255);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const void* n = x;
  if (norm_w != nullptr) {
    rc = launch_rmsnorm(x, norm_w, eps, ws, s.rows(), H, dtype, st);
    if (rc != DFLASH2_OK) return rc;
    n = ws;
  }
  if (kp_small_eligible(s, sms)) return launch_kp_small(s, n, w_kp, base, out, coef1, d_full, st);
  float* part = reinterpret_cast<float*>(ws + n_bytes);
  const GemmProblem gp{n, w_kp, nullptr, s.rows(), H, 4 * s.groups, 0, dtype};
  rc = launch_gemm_store(gp, plan, part, st);
  if (rc != DFLASH2_OK) return rc;
  return launch_conv_side0(s, n, part, plan.k_splits, base, out, coef1, d_full, st);
}

int dflash2_conv_finish(const void* y, const void* coef1, const float* base, int B, int G, int H, int group_size,
                        int taps, int dtype, const void* residual, void* out, const void* next_norm_w, float eps,
                        void* next_n, int next_row0, void* stream) {
  int rc = check_conv_shape(B, G, H, group_size, taps, dtype);
  if (rc != DFLASH2_OK) return rc;
  REQUIRE(y && coef1 && base && out, "a required pointer is NULL");
  REQUIRE((next_norm_w == nullptr) == (next_n == nullptr), "next_norm_w and next_n must be both set or both NULL");
  REQUIRE(aligned16(y) && aligned16(base) && aligned16(out) && (!residual || aligned16(residual)) &&
              (!next_norm_w || aligned16(next_norm_w)) && (!next_n || aligned16(next_n)),
          "y, base, residual, out, next_norm_w and next_n must be 16-byte aligned");
  if (next_n != nullptr) {
    REQUIRE(next_row0 >= 0 && next_row0 < G, "next_row0=%d must be in [0, G)", next_row0);
    REQUIRE(H / 8 <= 1024, "H=%d: the fused norm needs H <= 8192", H);
  }
  const ConvShape s{B, G, H, group_size, H / group_size, dtype};
  return launch_conv_side1(s, y, coef1, base, residual, out, next_norm_w, eps, next_n, next_row0,
                           static_cast<cudaStream_t>(stream));
}

int dflash2_conv_finish_ragged(const void* y, const void* coef1, const float* base, int B, int G, int H,
                               int group_size, int taps, int dtype, const void* residual, void* out,
                               const void* next_norm_w, float eps, void* next_n, int next_row0,
                               const int32_t* row_offsets, int m_rows, void* stream) {
  REQUIRE(row_offsets != nullptr, "row_offsets is NULL (use dflash2_conv_finish for dense rows)");
  REQUIRE(next_norm_w != nullptr && next_n != nullptr, "the ragged finish needs next_norm_w and next_n");
  REQUIRE(m_rows >= 1, "m_rows=%d must be >= 1", m_rows);
  int rc = check_conv_shape(B, G, H, group_size, taps, dtype);
  if (rc != DFLASH2_OK) return rc;
  REQUIRE(y && coef1 && base && out, "a required pointer is NULL");
  REQUIRE(aligned16(y) && aligned16(base) && aligned16(out) && (!residual || aligned16(residual)) &&
              aligned16(next_norm_w) && aligned16(next_n),
          "y, base, residual, out, next_norm_w and next_n must be 16-byte aligned");
  REQUIRE(next_row0 >= 0 && next_row0 < G, "next_row0=%d must be in [0, G)", next_row0);
  REQUIRE(H / 8 <= 1024, "H=%d: the fused norm needs H <= 8192", H);
  const ConvShape s{B, G, H, group_size, H / group_size, dtype};
  return launch_conv_side1(s, y, coef1, base, residual, out, next_norm_w, eps, next_n, next_row0,
                           static_cast<cudaStream_t>(stream), row_offsets, m_rows);
}

int dflash2_conv_coefficients(const void* x, const void* norm_w, float eps, const void* w_kp, int B, int G, int H,
                              int group_size, int taps, int dtype, void* n_out, float* d0, void* coef1,
                              void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_conv_shape(B, G, H, group_size, taps, dtype);
  if (rc != DFLASH2_OK) return rc;
  REQUIRE(x && w_kp && d0 && coef1 && workspace, "a required pointer is NULL");
  REQUIRE(norm_w == nullptr || n_out != nullptr, "n_out is required when norm_w is given");
  REQUIRE(aligned16(x) && aligned16(w_kp) && (!norm_w || aligned16(norm_w)) && (!n_out || aligned16(n_out)),
          "x, norm_w, w_kp and n_out must be 16-byte aligned");
  REQUIRE((reinterpret_cast<uintptr_t>(workspace) & 255u) == 0, "workspace must be 256-byte aligned");
  const ConvShape s{B, G, H, group_size, H / group_size, dtype};
  const int sms = sm_count();
  const size_t need = conv_prepare_workspace(s, sms);
  if (workspace_bytes < need)
    return fail(DFLASH2_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu bytes needed", workspace_bytes,
                need);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const GemmPlan plan = kp_plan(s, sms);
  const size_t es = dtype == DFLASH2_F32 ? 4 : 2;
  size_t n_bytes = static_cast<size_t>(s.rows()) * H * es;
  n_bytes = (n_bytes + 255) & ~static_cast<size_t>(255);
  const void* n = x;
  if (norm_w != nullptr) {
    rc = launch_rmsnorm(x, norm_w, eps, n_out, s.rows(), H, dtype, st);
    if (rc != DFLASH2_OK) return rc;
    n = n_out;
  }
  if (kp_small_eligible(s, sms)) return launch_kp_small(s, n, w_kp, nullptr, nullptr, coef1, nullptr, st, d0);
  float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + n_bytes);
  const GemmProblem gp{n, w_kp, nullptr, s.rows(), H, 4 * s.groups, 0, dtype};
  rc = launch_gemm_store(gp, plan, part, st);
  if (rc != DFLASH2_OK) return rc;
  return launch_conv_coefficients(part, plan.k_splits, s.rows(), s.groups, dtype, d0, coef1, st);
}

static int check_proj(const void* a, int M, int K, const void* w, const void* w_scales, const void* w_biases, int wbits,
                      int N, int dtype, void* out) {
  if (dtype != DFLASH2_BF16) return fail(DFLASH2_ERR_UNSUPPORTED, "the projections run in bf16 only (dtype=%d)", dtype);
  REQUIRE(a && w && out, "a required pointer is NULL");
  REQUIRE(M >= 1, "M=%d must be >= 1", M);
  REQUIRE(K >= 64 && K % 64 == 0, "K=%d must be a positive multiple of 64", K);
  REQUIRE(N >= 8 && N % 8 == 0, "N=%d must be a positive multiple of 8", N);
  REQUIRE(wbits == 16 || wbits == 4, "wbits=%d must be 16 (bf16) or 4 (affine 4-bit, groups of 64)", wbits);
  if (wbits == 4)
    REQUIRE(w_scales && w_biases && aligned16(w_scales) && aligned16(w_biases),
            "4-bit weights need 16-byte aligned w_scales and w_biases");
  REQUIRE(aligned16(a) && aligned16(w) && aligned16(out), "a, w and out must be 16-byte aligned");
  return DFLASH2_OK;
}

size_t dflash2_proj_workspace_bytes(int M, int N, int K) {
  if (M < 1 || N < 8 || K < 64) return 0;
  return proj_workspace(M, N, K, sm_count());
}

static int proj_ws(int M, int N, int K, void* workspace, size_t workspace_bytes, float** part) {
  const size_t need = proj_workspace(M, N, K, sm_count());
  *part = nullptr;
  if (need == 0) return DFLASH2_OK;
  if (workspace == nullptr || workspace_bytes < need)
    return fail(DFLASH2_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu bytes needed", workspace_bytes,
                need);
  REQUIRE((reinterpret_cast<uintptr_t>(workspace) & 255u) == 0, "workspace must be 256-byte aligned");
  *part = static_cast<float*>(workspace);
  return DFLASH2_OK;
}

int dflash2_proj(const void* a, int M, int K, const void* w, const void* w_scales, const void* w_biases, int wbits,
                 int N, int dtype, void* out, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_proj(a, M, K, w, w_scales, w_biases, wbits, N, dtype, out);
  if (rc != DFLASH2_OK) return rc;
  float* part = nullptr;
  if ((rc = proj_ws(M, N, K, workspace, workspace_bytes, &part)) != DFLASH2_OK) return rc;
  ProjSpec p{};
  p.part = part;
  p.a = a; p.w = w; p.scales = w_scales; p.qbias = w_biases; p.wbits = wbits;
  p.M = M; p.N = N; p.K = K; p.out = out;
  return launch_proj(p, static_cast<cudaStream_t>(stream));
}

int dflash2_proj_conv_in(const void* n, const float* d0, const float* base, int G, int group_size, int M, int K,
                         const void* w, const void* w_scales, const void* w_biases, int wbits, int N, int dtype,
                         void* out, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_proj(n, M, K, w, w_scales, w_biases, wbits, N, dtype, out);
  if (rc != DFLASH2_OK) return rc;
  float* part = nullptr;
  REQUIRE(d0 && base, "d0 and base are required");
  REQUIRE(G >= 2 && G <= 64 && 128 % G == 0, "G=%d must divide 128 (blocks must not straddle a 128-row tile)", G);
  REQUIRE(M % G == 0, "M=%d must be a whole number of %d-row blocks", M, G);
  REQUIRE(group_size == 16, "group_size=%d: the fused side 0 is built for groups of 16 channels", group_size);
  REQUIRE(M % 4 == 0, "M=%d must be a multiple of 4 (rows of the side-0 deltas are loaded in 16-byte units)", M);
  REQUIRE(aligned16(base) && aligned16(d0), "base and d0 must be 16-byte aligned");
  if ((rc = proj_ws(M, N, K, workspace, workspace_bytes, &part)) != DFLASH2_OK) return rc;
  ProjSpec p{};
  p.part = part;
  p.a = n; p.w = w; p.scales = w_scales; p.qbias = w_biases; p.wbits = wbits;
  p.M = M; p.N = N; p.K = K; p.out = out;
  p.d0 = d0; p.base = base; p.G = G; p.gs = group_size; p.groups = K / group_size;
  return launch_proj(p, static_cast<cudaStream_t>(stream));
}

int dflash2_proj_conv_out(const void* a, int M, int K, const void* w, const void* w_scales, const void* w_biases,
                          int wbits, int N, const void* coef1, const float* base, int G, int group_size,
                          const void* residual, int dtype, void* out, void* workspace, size_t workspace_bytes,
                          void* stream) {
  int rc = check_proj(a, M, K, w, w_scales, w_biases, wbits, N, dtype, out);
  if (rc != DFLASH2_OK) return rc;
  float* part = nullptr;
  REQUIRE(coef1 && base, "coef1 and base are required");
  REQUIRE(G >= 2 && G <= 32 && 32 % G == 0, "G=%d must divide 32 (a block's rows must share a warp)", G);
  REQUIRE(M % G == 0, "M=%d must be a whole number of %d-row blocks", M, G);
  REQUIRE(group_size == 8 || group_size == 16 || group_size == 32, "group_size=%d must be 8, 16 or 32", group_size);
  REQUIRE(N % group_size == 0 && N % 32 == 0, "N=%d must be a multiple of 32 and of group_size", N);
  REQUIRE(aligned16(base) && (!residual || aligned16(residual)), "base and residual must be 16-byte aligned");
  if ((rc = proj_ws(M, N, K, workspace, workspace_bytes, &part)) != DFLASH2_OK) return rc;
  ProjSpec p{};
  p.part = part;
  p.a = a; p.w = w; p.scales = w_scales; p.qbias = w_biases; p.wbits = wbits;
  p.M = M; p.N = N; p.K = K; p.out = out;
  p.coef1 = coef1; p.base = base; p.residual = residual; p.G = G; p.gs = group_size; p.groups = N / group_size;
  return launch_proj(p, static_cast<cudaStream_t>(stream));
}

size_t dflash2_head_topk_workspace_bytes(int M, int H, int V, int K, int R) {
  if (M < 1 || H < 64 || V < 1 || K < 1 || R < 0) return 0;
  return head_workspace(M, V, K, R, sm_count());
}

int dflash2_head_topk(const void* h, int M, int H, const void* w_head, int V, const float* bias, const void* w_proj,
                      int R, int K, int dtype, int32_t* cand, float* unary, float* z, float* logits, void* workspace,
                      size_t workspace_bytes, void* stream) {
  REQUIRE(dtype == DFLASH2_BF16 || dtype == DFLASH2_F32, "dtype=%d is not DFLASH2_BF16 or DFLASH2_F32", dtype);
  REQUIRE(M >= 1, "M=%d must be >= 1", M);
  REQUIRE(H >= 64 && H % 64 == 0, "H=%d must be a positive multiple of 64", H);
  REQUIRE(K >= 1 && K <= 16 && K <= V, "K=%d must be in [1, min(16, V)]", K);
  REQUIRE(h && w_head && cand && unary && workspace, "a required pointer is NULL");
  REQUIRE((w_proj == nullptr) == (z == nullptr), "w_proj and z must be both set or both NULL");
  if (w_proj != nullptr) REQUIRE(R >= 16 && R <= 256 && R % 16 == 0, "R=%d must be a multiple of 16 in [16, 256]", R);
  REQUIRE(aligned16(h) && aligned16(w_head) && (!w_proj || aligned16(w_proj)) && (!bias || aligned16(bias)),
          "h, w_head, w_proj and bias must be 16-byte aligned");
  REQUIRE((reinterpret_cast<uintptr_t>(workspace) & 255u) == 0, "workspace must be 256-byte aligned");
  const int r_eff = w_proj != nullptr ? R : 0;
  const int sms = sm_count();
  const size_t need = head_workspace(M, V, K, r_eff, sms);
  if (workspace_bytes < need)
    return fail(DFLASH2_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu bytes needed", workspace_bytes,
                need);
  const GemmPlan plan = head_plan(M, H, V, r_eff, sms);
  const GemmProblem gp{h, w_head, w_proj, M, H, V, r_eff, dtype};
  return launch_head_topk(gp, plan, bias, K, cand, unary, z, logits, workspace, static_cast<cudaStream_t>(stream));
}

int dflash2_head_topk_vocab(const void* h, int M, int H, const void* w_listed, int V_listed, const int32_t* vocab_ids,
                            const float* bias_listed, const void* w_proj, int R, int K, int dtype, int32_t* cand,
                            float* unary, float* z, float* logits, void* workspace, size_t workspace_bytes,
                            void* stream) {
  REQUIRE(vocab_ids != nullptr, "vocab_ids is NULL (use dflash2_head_topk for the full vocabulary)");
  REQUIRE(dtype == DFLASH2_BF16 || dtype == DFLASH2_F32, "dtype=%d is not DFLASH2_BF16 or DFLASH2_F32", dtype);
  REQUIRE(M >= 1, "M=%d must be >= 1", M);
  REQUIRE(H >= 64 && H % 64 == 0, "H=%d must be a positive multiple of 64", H);
  REQUIRE(K >= 1 && K <= 16 && K <= V_listed, "K=%d must be in [1, min(16, V_listed)]", K);
  REQUIRE(h && w_listed && cand && unary && workspace, "a required pointer is NULL");
  REQUIRE((w_proj == nullptr) == (z == nullptr), "w_proj and z must be both set or both NULL");
  if (w_proj != nullptr) REQUIRE(R >= 16 && R <= 256 && R % 16 == 0, "R=%d must be a multiple of 16 in [16, 256]", R);
  REQUIRE(aligned16(h) && aligned16(w_listed) && (!w_proj || aligned16(w_proj)) && (!bias_listed || aligned16(bias_listed)),
          "h, w_listed, w_proj and bias_listed must be 16-byte aligned");
  REQUIRE((reinterpret_cast<uintptr_t>(workspace) & 255u) == 0, "workspace must be 256-byte aligned");
  const int r_eff = w_proj != nullptr ? R : 0;
  const int sms = sm_count();
  const size_t need = head_workspace(M, V_listed, K, r_eff, sms);
  if (workspace_bytes < need)
    return fail(DFLASH2_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu bytes needed", workspace_bytes,
                need);
  const GemmPlan plan = head_plan(M, H, V_listed, r_eff, sms);
  const GemmProblem gp{h, w_listed, w_proj, M, H, V_listed, r_eff, dtype};
  return launch_head_topk(gp, plan, bias_listed, K, cand, unary, z, logits, workspace,
                          static_cast<cudaStream_t>(stream), vocab_ids);
}

int dflash2_score_edges(const int32_t* cand, const float* unary, const float* z, const int32_t* anchors,
                        const void* pred_book, const void* succ_book, int B, int steps, int K, int R, int V, int dtype,
                        float* S, int32_t* path, void* stream) {
  REQUIRE(dtype == DFLASH2_BF16 || dtype == DFLASH2_F32, "dtype=%d is not DFLASH2_BF16 or DFLASH2_F32", dtype);
  REQUIRE(B >= 1 && steps >= 1 && steps <= 63, "B=%d, steps=%d: need B >= 1 and 1 <= steps <= 63", B, steps);
  REQUIRE(K >= 1 && K <= 32, "K=%d must be in [1, 32]", K);
  REQUIRE(R >= 8 && R <= 128 && R % 8 == 0, "R=%d must be a multiple of 8 in [8, 128]", R);
  REQUIRE(V >= 1, "V=%d must be >= 1", V);
  REQUIRE(cand && unary && z && anchors && pred_book && succ_book, "a required pointer is NULL");
  REQUIRE(S != nullptr || path != nullptr, "at least one of S and path must be non-NULL");
  REQUIRE(aligned16(z) && aligned16(pred_book) && aligned16(succ_book), "z and the codebooks must be 16-byte aligned");
  return launch_score_edges(cand, unary, z, anchors, pred_book, succ_book, B, steps, K, R, V, dtype, S, path,
                            static_cast<cudaStream_t>(stream));
}

int dflash2_score_edges_depths(const int32_t* cand, const float* unary, const float* z, const int32_t* anchors,
                               const void* pred_book, const void* succ_book, const int32_t* depths, int B, int steps,
                               int K, int R, int V, int dtype, float* S, int32_t* path, void* stream) {
  REQUIRE(depths != nullptr, "depths is NULL (use dflash2_score_edges for full-depth blocks)");
  REQUIRE(dtype == DFLASH2_BF16 || dtype == DFLASH2_F32, "dtype=%d is not DFLASH2_BF16 or DFLASH2_F32", dtype);
  REQUIRE(B >= 1 && steps >= 1 && steps <= 63, "B=%d, steps=%d: need B >= 1 and 1 <= steps <= 63", B, steps);
  REQUIRE(K >= 1 && K <= 32, "K=%d must be in [1, 32]", K);
  REQUIRE(R >= 8 && R <= 128 && R % 8 == 0, "R=%d must be a multiple of 8 in [8, 128]", R);
  REQUIRE(V >= 1, "V=%d must be >= 1", V);
  REQUIRE(cand && unary && z && anchors && pred_book && succ_book && path, "a required pointer is NULL");
  REQUIRE(aligned16(z) && aligned16(pred_book) && aligned16(succ_book), "z and the codebooks must be 16-byte aligned");
  return launch_score_edges(cand, unary, z, anchors, pred_book, succ_book, B, steps, K, R, V, dtype, S, path,
                            static_cast<cudaStream_t>(stream), depths);
}

int dflash2_score_edges_ragged(const int32_t* cand, const float* unary, const float* z, const int32_t* anchors,
                               const void* pred_book, const void* succ_book, const int32_t* row_offsets, int B,
                               int steps, int K, int R, int V, int m_rows, int dtype, float* S, int32_t* path,
                               void* stream) {
  REQUIRE(row_offsets != nullptr, "row_offsets is NULL (use dflash2_score_edges for dense blocks)");
  REQUIRE(dtype == DFLASH2_BF16 || dtype == DFLASH2_F32, "dtype=%d is not DFLASH2_BF16 or DFLASH2_F32", dtype);
  REQUIRE(B >= 1 && steps >= 1 && steps <= 63, "B=%d, steps=%d: need B >= 1 and 1 <= steps <= 63", B, steps);
  REQUIRE(m_rows >= 1, "m_rows=%d must be >= 1", m_rows);
  REQUIRE(K == 16 && (R == 16 || R == 32 || (R == 64 && dtype == DFLASH2_BF16)),
          "ragged rows need K = 16 and R in {16, 32, 64} (bf16) or {16, 32} (f32); got K=%d, R=%d", K, R);
  REQUIRE(V >= 1, "V=%d must be >= 1", V);
  REQUIRE(cand && unary && z && anchors && pred_book && succ_book && path, "a required pointer is NULL");
  REQUIRE(aligned16(z) && aligned16(pred_book) && aligned16(succ_book), "z and the codebooks must be 16-byte aligned");
  return launch_score_edges(cand, unary, z, anchors, pred_book, succ_book, B, steps, K, R, V, dtype, S, path,
                            static_cast<cudaStream_t>(stream), nullptr, row_offsets, m_rows);
}

int dflash2_select_path_depths(const float* S, const int32_t* cand, const int32_t* depths, int B, int steps, int K,
                               int32_t* path, void* stream) {
  REQUIRE(depths != nullptr, "depths is NULL (use dflash2_select_path for full-depth blocks)");
  REQUIRE(B >= 1 && steps >= 1, "B=%d, steps=%d must be >= 1", B, steps);
  REQUIRE(K >= 1 && K <= 32, "K=%d must be in [1, 32]", K);
  REQUIRE(S && cand && path, "a required pointer is NULL");
  return launch_select_path(S, cand, B, steps, K, path, static_cast<cudaStream_t>(stream), depths);
}

int dflash2_select_path(const float* S, const int32_t* cand, int B, int steps, int K, int32_t* path, void* stream) {
  REQUIRE(B >= 1 && steps >= 1, "B=%d, steps=%d must be >= 1", B, steps);
  REQUIRE(K >= 1 && K <= 32, "K=%d must be in [1, 32]", K);
  REQUIRE(S && cand && path, "a required pointer is NULL");
  return launch_select_path(S, cand, B, steps, K, path, static_cast<cudaStream_t>(stream));
}

static int check_kv4(int heads, int D, int page_size, int num_pages, int dtype) {
  if (dtype != DFLASH2_BF16) return fail(DFLASH2_ERR_UNSUPPORTED, "the 4-bit cache takes bf16 rows only (dtype=%d)", dtype);
  REQUIRE(heads >= 1 && heads <= 512, "heads=%d must be in [1, 512]", heads);
  REQUIRE(D == 64 || D == 128, "head_dim=%d must be 64 or 128", D);
  REQUIRE(page_size >= 16 && page_size <= 4096 && (page_size & (page_size - 1)) == 0,
          "page_size=%d must be a power of two in [16, 4096]", page_size);
  REQUIRE(num_pages >= 1, "num_pages=%d must be >= 1", num_pages);
  return DFLASH2_OK;
}

size_t dflash2_kv4_page_bytes(int heads, int D, int page_size) {
  if (check_kv4(heads, D, page_size, 1, DFLASH2_BF16) != DFLASH2_OK) return 0;
  return static_cast<size_t>(heads) * 2 * page_size * (D / 2 + D / 64 * 4);
}

int dflash2_kv4_append(const void* k, const void* v, int64_t k_stride, int64_t v_stride, const int64_t* slots, int T,
                       int heads, int D, int page_size, int num_pages, int dtype, void* cache, void* stream) {
  int rc = check_kv4(heads, D, page_size, num_pages, dtype);
  if (rc != DFLASH2_OK) return rc;
  REQUIRE(T >= 0, "T=%d must be >= 0", T);
  if (T == 0) return DFLASH2_OK;
  REQUIRE(k && v && slots && cache, "a required pointer is NULL");
  REQUIRE(aligned16(k) && aligned16(v) && aligned16(cache) && aligned(slots),
          "k, v and cache must be 16-byte aligned, slots 8-byte aligned");
  const int64_t row = static_cast<int64_t>(heads) * D;
  REQUIRE(k_stride >= row && k_stride % 8 == 0 && v_stride >= row && v_stride % 8 == 0,
          "row strides %lld, %lld must be multiples of 8 and at least heads * head_dim = %lld",
          static_cast<long long>(k_stride), static_cast<long long>(v_stride), static_cast<long long>(row));
  const Kv4Rows r{k, v, k_stride, v_stride, slots, T, heads, D, page_size, num_pages, cache, nullptr, nullptr};
  return launch_kv4_rows(r, static_cast<cudaStream_t>(stream));
}

int dflash2_kv4_read(const void* cache, const int64_t* slots, int T, int heads, int D, int page_size, int num_pages,
                     int dtype, void* k, void* v, void* stream) {
  int rc = check_kv4(heads, D, page_size, num_pages, dtype);
  if (rc != DFLASH2_OK) return rc;
  REQUIRE(T >= 0, "T=%d must be >= 0", T);
  if (T == 0) return DFLASH2_OK;
  REQUIRE(k && v && slots && cache, "a required pointer is NULL");
  REQUIRE(aligned16(k) && aligned16(v) && aligned16(cache) && aligned(slots),
          "k, v and cache must be 16-byte aligned, slots 8-byte aligned");
  const Kv4Rows r{nullptr, nullptr, 0, 0, slots, T, heads, D, page_size, num_pages, const_cast<void*>(cache), k, v};
  return launch_kv4_rows(r, static_cast<cudaStream_t>(stream));
}

static int check_kv4_attention(int B, int G, int Hq, int Hkv, int D, int page_size, int num_pages, int max_pages,
                               int dtype) {
  int rc = check_kv4(Hkv, D, page_size, num_pages, dtype);
  if (rc != DFLASH2_OK) return rc;
  REQUIRE(B >= 1, "B=%d must be >= 1", B);
  REQUIRE(G >= 1 && G <= 64, "G=%d must be in [1, 64]", G);
  REQUIRE(Hq >= Hkv && Hq % Hkv == 0 && Hq / Hkv <= 64, "Hq=%d must be 1 to 64 times Hkv=%d", Hq, Hkv);
  REQUIRE(max_pages >= 1 && static_cast<int64_t>(max_pages) * page_size <= 0x7fffff00LL,
          "max_pages=%d must be >= 1, and a sequence's pages hold less than 2^31 tokens", max_pages);
  return DFLASH2_OK;
}

size_t dflash2_kv4_attention_workspace_bytes(int B, int G, int Hq, int Hkv, int D, int page_size, int max_pages) {
  if (check_kv4_attention(B, G, Hq, Hkv, D, page_size, 1, max_pages, DFLASH2_BF16) != DFLASH2_OK) return 0;
  return kv4_attention_workspace(B, G, Hq, Hkv, D, page_size, max_pages, sm_count());
}

static int kv4_attention_call(Kv4Attention r, int dtype, size_t workspace_bytes, void* stream) {
  int rc = check_kv4_attention(r.B, r.G, r.Hq, r.Hkv, r.D, r.page_size, r.num_pages, r.max_pages, dtype);
  if (rc != DFLASH2_OK) return rc;
  REQUIRE(r.q && r.cache && r.table && r.ctx && r.out, "a required pointer is NULL");
  REQUIRE((r.k_new == nullptr) == (r.v_new == nullptr), "k_new and v_new must be both set or both NULL");
  REQUIRE(aligned16(r.q) && aligned16(r.cache) && aligned16(r.out) && aligned16(r.k_new) && aligned16(r.v_new),
          "q, cache, k_new, v_new and out must be 16-byte aligned");
  REQUIRE(aligned(r.table, r.ctx, r.parents), "page_table, ctx_len and parents must be 4-byte aligned");
  REQUIRE(r.q_stride >= static_cast<int64_t>(r.Hq) * r.D && r.q_stride % 8 == 0,
          "q_stride=%lld must be a multiple of 8 and at least Hq * head_dim", static_cast<long long>(r.q_stride));
  if (r.k_new != nullptr)
    REQUIRE(r.new_stride >= static_cast<int64_t>(r.Hkv) * r.D && r.new_stride % 8 == 0,
            "new_stride=%lld must be a multiple of 8 and at least Hkv * head_dim", static_cast<long long>(r.new_stride));
  REQUIRE(r.window >= 0, "window=%d must be >= 0 (0: none)", r.window);
  REQUIRE(r.causal == 0 || r.causal == 1, "causal=%d must be 0 or 1", r.causal);
  REQUIRE(r.scale == r.scale && r.scale - r.scale == 0.f, "scale must be finite");
  const size_t need = kv4_attention_workspace(r.B, r.G, r.Hq, r.Hkv, r.D, r.page_size, r.max_pages, sm_count());
  if (need > 0) {
    if (r.workspace == nullptr || workspace_bytes < need)
      return fail(DFLASH2_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu bytes needed", workspace_bytes,
                  need);
    REQUIRE((reinterpret_cast<uintptr_t>(r.workspace) & 255u) == 0, "workspace must be 256-byte aligned");
  }
  // a window that reaches every key from every row is none (and the rows' positions less it stay above -2^31)
  if (static_cast<int64_t>(r.window) >= static_cast<int64_t>(r.max_pages) * r.page_size + 2 * r.G) r.window = 0;
  return launch_kv4_attention(r, static_cast<cudaStream_t>(stream));
}

int dflash2_kv4_attention(const void* q, int64_t q_stride, const void* cache, const int32_t* page_table,
                          const int32_t* ctx_len, const void* k_new, const void* v_new, int64_t new_stride, int B, int G,
                          int Hq, int Hkv, int D, int page_size, int num_pages, int max_pages, int causal, int window,
                          float scale, int dtype, void* out, void* workspace, size_t workspace_bytes, void* stream) {
  return kv4_attention_call(Kv4Attention{q, q_stride, cache, page_table, ctx_len, k_new, v_new, new_stride, B, G, Hq, Hkv,
                                         D, page_size, num_pages, max_pages, causal, window, scale, out, workspace, nullptr},
                            dtype, workspace_bytes, stream);
}

int dflash2_kv4_attention_tree(const void* q, int64_t q_stride, const void* cache, const int32_t* page_table,
                               const int32_t* ctx_len, const void* k_new, const void* v_new, int64_t new_stride,
                               const int32_t* parents, int B, int G, int Hq, int Hkv, int D, int page_size, int num_pages,
                               int max_pages, int window, float scale, int dtype, void* out, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (dtype == DFLASH2_BF16)  // (any other is refused as such)
    REQUIRE(parents && k_new && v_new, "a tree needs parents, k_new and v_new");
  return kv4_attention_call(Kv4Attention{q, q_stride, cache, page_table, ctx_len, k_new, v_new, new_stride, B, G, Hq, Hkv,
                                         D, page_size, num_pages, max_pages, 0, window, scale, out, workspace, parents},
                            dtype, workspace_bytes, stream);
}

int dflash2_kv4_plan(const int32_t* ctx_len, const int32_t* change, int32_t* page_table, int32_t* free_pages,
                     const int32_t* free_state, const int32_t* place, int B, int G, int rows, int max_pages, int page_size,
                     int num_pages, int capacity, int32_t* ctx_out, int32_t* state_out, int32_t* row_offsets,
                     int64_t* slots, int32_t* positions, void* stream) {
  REQUIRE(B >= 1 && B <= kPlanMaxSequences, "B=%d must be in [1, %d]", B, kPlanMaxSequences);
  REQUIRE(page_size >= 16 && page_size <= 4096 && (page_size & (page_size - 1)) == 0,
          "page_size=%d must be a power of two in [16, 4096]", page_size);
  // (entries, pages and rows are counted in int, by steps of all threads: 2^31 - 2^16 leaves room for the last step)
  constexpr int kMost = 0x7fff0000;
  REQUIRE(num_pages >= 1 && capacity >= 1 && capacity <= kMost,
          "num_pages=%d must be >= 1 and capacity=%d in [1, 2^31 - 2^16]", num_pages, capacity);
  REQUIRE(max_pages >= 1 && static_cast<int64_t>(max_pages) * page_size <= 0x7fffff00LL,
          "max_pages=%d must be >= 1, and a sequence's pages hold less than 2^31 tokens", max_pages);
  REQUIRE(ctx_len && change && page_table && free_pages && free_state && ctx_out && state_out && row_offsets,
          "a required pointer is NULL");
  if (place != nullptr)
    REQUIRE(G >= 1 && static_cast<int64_t>(B) * G <= kMost, "G=%d must be >= 1 and B * G at most 2^31 - 2^16", G);
  else
    REQUIRE(rows >= 0 && rows <= kMost, "rows=%d must be in [0, 2^31 - 2^16]", rows);
  REQUIRE((place == nullptr && rows == 0) || (slots && positions), "slots and positions are required");
  REQUIRE(aligned(ctx_len, change, page_table, free_pages, free_state, place, ctx_out, state_out, row_offsets, slots, positions),
          "every array must be aligned to its elements");
  const Kv4Plan r{ctx_len, change, free_state, place, page_table, free_pages, ctx_out, state_out, row_offsets, positions,
                  slots, B, max_pages, page_size, num_pages, capacity, G, place != nullptr ? 0x7fffffff : rows};
  return launch_kv4_plan(r, static_cast<cudaStream_t>(stream));
}

static int check_logits(int M, int V, int B, int max_len, int n_bias, int K) {
  REQUIRE(M >= 0 && B >= 1, "M=%d must be >= 0 and B=%d >= 1", M, B);
  REQUIRE(V >= 1 && V <= (1 << 22), "V=%d must be in [1, 2^22]", V);
  REQUIRE(K >= 0 && K <= 16 && K <= V, "K=%d must be in [0, min(16, V)]", K);
  REQUIRE(max_len >= 0 && max_len <= (1 << 20) - 128, "max_len=%d must be in [0, 2^20 - 128]", max_len);
  REQUIRE(n_bias >= 0 && n_bias <= 2047, "n_bias=%d must be in [0, 2047]", n_bias);
  // tiles of 1024 tokens a row, and windows of 2^18 a request, are counted in int
  const int64_t tiles = (V + 1024LL) / 1024 + 1, windows = (V + 0x3ffffLL) >> 18;
  REQUIRE(M * tiles <= 0x3fffffff && B * windows <= 0x3fffffff, "M=%d, V=%d, B=%d are too large", M, V, B);
  return DFLASH2_OK;
}

size_t dflash2_logits_topk_workspace_bytes(int M, int V, int B, int ragged, int max_len, int drafted, int n_bias, int K) {
  if (check_logits(M, V, B, max_len, n_bias, K) != DFLASH2_OK) return 0;
  return logits_topk_workspace(M, V, B, ragged != 0, max_len, drafted != 0, n_bias, K);
}

int dflash2_logits_topk(const void* logits, int64_t stride, int M, int V, int dtype, int B, const int32_t* row_offsets,
                        const int32_t* history, int64_t history_stride, const int32_t* prompt_len,
                        const int32_t* history_len, int max_len, const float* repetition, const float* frequency,
                        const float* presence, const int32_t* tokens, const int32_t* parents, const int32_t* bias_ids,
                        const float* bias, int n_bias, const int32_t* mask, int64_t mask_stride, int K, int32_t* cand,
                        float* unary, void* out, int64_t out_stride, void* workspace, size_t workspace_bytes,
                        void* stream) {
  REQUIRE(dtype == DFLASH2_BF16 || dtype == DFLASH2_F32, "dtype=%d is not DFLASH2_BF16 or DFLASH2_F32", dtype);
  int rc = check_logits(M, V, B, max_len, n_bias, K);
  if (rc != DFLASH2_OK) return rc;
  REQUIRE(row_offsets != nullptr || M % B == 0, "M=%d rows are no whole number for each of B=%d requests", M, B);
  if (M == 0) return DFLASH2_OK;
  REQUIRE(logits != nullptr, "a required pointer is NULL");
  REQUIRE(K == 0 || (cand && unary), "cand and unary are required");
  REQUIRE(K > 0 || out != nullptr, "nothing is wanted: K = 0 and no out");
  const uintptr_t size = dtype == DFLASH2_F32 ? 4 : 2;
  REQUIRE(reinterpret_cast<uintptr_t>(logits) % size == 0 && reinterpret_cast<uintptr_t>(out) % size == 0,
          "logits and out must be aligned to their type");
  REQUIRE(aligned(row_offsets, history, prompt_len, history_len, repetition, frequency, presence, tokens, parents, bias_ids, bias,
                  mask, cand, unary),
          "every array must be aligned to its elements");
  REQUIRE(stride >= V || M == 1, "stride=%lld must be at least V=%d", static_cast<long long>(stride), V);
  REQUIRE(out == nullptr || out_stride >= V || M == 1, "out_stride=%lld must be at least V=%d",
          static_cast<long long>(out_stride), V);
  if (history != nullptr) {
    REQUIRE(history_len != nullptr, "history needs history_len");
    REQUIRE(history_stride >= max_len || B == 1, "history_stride=%lld must be at least max_len=%d",
            static_cast<long long>(history_stride), max_len);
  }
  REQUIRE(parents == nullptr || tokens != nullptr, "parents need tokens");
  REQUIRE(tokens == nullptr || row_offsets != nullptr || M / B <= 64, "a request's drafted rows are at most 64, got %d", M / B);
  REQUIRE(n_bias == 0 || (bias_ids && bias), "bias_ids and bias are required");
  REQUIRE(mask == nullptr || mask_stride >= (V + 31) / 32 || M == 1, "mask_stride=%lld must be at least V / 32 words",
          static_cast<long long>(mask_stride));
  if (history == nullptr) max_len = 0;
  const size_t need = logits_topk_workspace(M, V, B, row_offsets != nullptr, max_len, tokens != nullptr, n_bias, K);
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need)
      return fail(DFLASH2_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu bytes needed", workspace_bytes,
                  need);
    REQUIRE((reinterpret_cast<uintptr_t>(workspace) & 255u) == 0, "workspace must be 256-byte aligned");
  }
  const LogitsTopk r{logits, stride, M, V, dtype, B, row_offsets, max_len > 0 ? history : nullptr, history_stride, prompt_len,
                     history_len, max_len, repetition, frequency, presence, tokens, parents, bias_ids, bias, n_bias, mask,
                     mask_stride, K, cand, unary, out, out_stride, workspace};
  return launch_logits_topk(r, static_cast<cudaStream_t>(stream));
}

static int check_ffn(int M, int H, int F, int act, int dtype) {
  if (dtype != DFLASH2_BF16) return fail(DFLASH2_ERR_UNSUPPORTED, "the gated feed-forward runs in bf16 only (dtype=%d)", dtype);
  REQUIRE(M >= 0, "M=%d must be >= 0", M);
  REQUIRE(H >= 8 && H % 8 == 0 && F >= 8 && F % 8 == 0, "H=%d and F=%d must be positive multiples of 8", H, F);
  REQUIRE(act == DFLASH2_ACT_SILU || act == DFLASH2_ACT_GELU_TANH, "act=%d is not a dflash2_act", act);
  // tiles of 256 rows by 128 columns (and twice 256 by 256 for the weights' gradients) are counted in int
  const int64_t m = (M + 255LL) / 256, h = (H + 127LL) / 128, f = (F + 127LL) / 128;
  // (and H and F rounded up to 64 columns are ints)
  REQUIRE(H <= 0x7fffffc0 && F <= 0x7fffffc0 && m * f <= 0x3fffffff && m * h <= 0x3fffffff && f * h <= 0x3fffffff, "M=%d, H=%d, F=%d are too large", M, H, F);
  return DFLASH2_OK;
}

static int check_ffn_workspace(int M, int H, int F, bool backward, const void* workspace, size_t workspace_bytes) {
  const size_t need = gated_ffn_workspace(M, H, F, backward, sm_count());
  if (workspace == nullptr || workspace_bytes < need)
    return fail(DFLASH2_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu bytes needed",
                workspace == nullptr ? 0 : workspace_bytes, need);
  REQUIRE((reinterpret_cast<uintptr_t>(workspace) & 255u) == 0, "workspace must be 256-byte aligned");
  return DFLASH2_OK;
}

size_t dflash2_gated_ffn_workspace_bytes(int M, int H, int F, int backward) {
  if (check_ffn(M, H, F, DFLASH2_ACT_SILU, DFLASH2_BF16) != DFLASH2_OK) return 0;
  return gated_ffn_workspace(M, H, F, backward != 0, sm_count());
}

int dflash2_gated_ffn(const void* x, int M, int H, const void* w_gate, const void* w_up, int F, int act, int dtype,
                      void* h, void* pre, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_ffn(M, H, F, act, dtype);
  if (rc != DFLASH2_OK || M == 0) return rc;
  REQUIRE(x && w_gate && w_up && h, "a required pointer is NULL");
  REQUIRE(aligned16(x) && aligned16(w_gate) && aligned16(w_up) && aligned16(h) && aligned16(pre),
          "x, w_gate, w_up, h and pre must be 16-byte aligned");
  if ((rc = check_ffn_workspace(M, H, F, false, workspace, workspace_bytes)) != DFLASH2_OK) return rc;
  GatedFfn r{};
  r.x = x; r.w_gate = w_gate; r.w_up = w_up; r.h = h; r.pre = pre;
  r.M = M; r.H = H; r.F = F; r.act = act; r.workspace = workspace;
  return launch_gated_ffn(r, static_cast<cudaStream_t>(stream));
}

int dflash2_gated_ffn_backward(const void* dh, const void* pre, const void* x, const void* w_gate, const void* w_up,
                               int M, int H, int F, int act, int dtype, void* dx, void* dw_gate, void* dw_up,
                               void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_ffn(M, H, F, act, dtype);
  if (rc != DFLASH2_OK) return rc;
  REQUIRE((dw_gate == nullptr) == (dw_up == nullptr), "dw_gate and dw_up must be both set or both NULL");
  if (M == 0) {  // no rows: the weights' gradients are zero
    const size_t n = static_cast<size_t>(F) * H * 2;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dw_gate != nullptr && (cudaMemsetAsync(dw_gate, 0, n, st) != cudaSuccess ||
                               cudaMemsetAsync(dw_up, 0, n, st) != cudaSuccess))
      return fail(DFLASH2_ERR_CUDA, "clearing the weights' gradients failed");
    return DFLASH2_OK;
  }
  REQUIRE(dx || dw_gate, "nothing to compute: dx and the weights' gradients are all NULL");
  REQUIRE(dh && pre && (!dw_gate || x) && (!dx || (w_gate && w_up)), "a required pointer is NULL");
  REQUIRE(aligned16(dh) && aligned16(pre) && aligned16(x) && aligned16(w_gate) && aligned16(w_up) && aligned16(dx) &&
              aligned16(dw_gate) && aligned16(dw_up),
          "every tensor must be 16-byte aligned");
  if ((rc = check_ffn_workspace(M, H, F, true, workspace, workspace_bytes)) != DFLASH2_OK) return rc;
  GatedFfn r{};
  r.x = x; r.w_gate = w_gate; r.w_up = w_up; r.dh = dh; r.pre = const_cast<void*>(pre);
  r.dx = dx; r.dw_gate = dw_gate; r.dw_up = dw_up;
  r.M = M; r.H = H; r.F = F; r.act = act; r.workspace = workspace;
  return launch_gated_ffn_backward(r, static_cast<cudaStream_t>(stream));
}

int dflash2_selftest_bounded_wait(int limit_us, void* stream) {
  REQUIRE(limit_us >= 1 && limit_us <= 1000000, "limit_us=%d must be in [1, 1000000]", limit_us);
  return launch_wait_selftest(limit_us, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
