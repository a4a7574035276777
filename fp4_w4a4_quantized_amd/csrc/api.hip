// api.hip -- the C ABI of libfp4q (declared in include/fp4q.h): host-side
// argument validation, workspace queries and kernel launches.  Every check
// runs before the first HIP call, so invalid calls fail without touching
// the device.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "fp4q_internal.h"

namespace {

thread_local int g_last_hip_error = 0;

// FP4Q_HOOK_FAIL_NEXT_LAUNCH: a hipError_t that the next call which would
// launch reports instead of launching (0: none).
std::atomic<int> g_fail_next{0};

// True (and the hook consumed) when a test asked the launch path to fail.
inline bool injected_failure() {
  const int e = g_fail_next.exchange(0);
  if (e == 0) return false;
  g_last_hip_error = e;
  return true;
}

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

inline int blk_of(int fmt) { return fmt == FP4Q_NVFP4 ? 16 : 32; }

inline bool fmt_ok(int fmt) { return fmt == FP4Q_NVFP4 || fmt == FP4Q_MXFP4; }

inline bool layout_ok(int layout) {
  return layout == FP4Q_LAYOUT_ROWMAJOR || layout == FP4Q_LAYOUT_TILED;
}

// Clear any stale error state before a launch, so that check_launch() sees
// only what this call's launches produced.
inline void clear_error() { (void)hipGetLastError(); }

// Report launch errors from the calls just made on this thread.
inline int check_launch() {
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) {
    g_last_hip_error = (int)e;
    return FP4Q_ERR_HIP;
  }
  return FP4Q_OK;
}

constexpr int MAX_GROUPS = 2048;  // grouped GEMM scans 8 groups per thread of 256

}  // namespace

extern "C" {

const char* fp4q_status_str(int status) {
  switch (status) {
    case FP4Q_OK: return "ok";
    case FP4Q_ERR_INVALID: return "invalid argument";
    case FP4Q_ERR_UNSUPPORTED: return "unsupported shape";
    case FP4Q_ERR_WORKSPACE: return "workspace missing or too small";
    case FP4Q_ERR_HIP: return "HIP error";
    default: return "unknown status";
  }
}

int fp4q_last_hip_error(void) { return g_last_hip_error; }

int fp4q_packed_bytes(fp4q_format_t fmt, fp4q_layout_t layout, int64_t rows, int64_t cols,
                      size_t* code_bytes, size_t* scale_bytes) {
  if (!fmt_ok(fmt) || !layout_ok(layout) || rows < 0 || cols <= 0) return FP4Q_ERR_INVALID;
  const int blk = blk_of(fmt);
  if (cols % blk != 0) return FP4Q_ERR_INVALID;
  int64_t rc = rows, rs = rows;
  if (layout == FP4Q_LAYOUT_TILED) {
    if (cols % 128 != 0) return FP4Q_ERR_INVALID;
    rc = (rows + 15) / 16 * 16;
    rs = (rows + 63) / 64 * 64;
  }
  if (code_bytes) *code_bytes = (size_t)(rc * (cols / 2));
  if (scale_bytes) *scale_bytes = (size_t)(rs * (cols / blk));
  return FP4Q_OK;
}

size_t fp4q_quantize_workspace_bytes(fp4q_format_t fmt, int64_t rows, int64_t cols,
                                     int32_t num_groups) {
  (void)rows;
  (void)cols;
  return fp4q::quantize_workspace_bytes(fmt, num_groups > 0 ? num_groups : 1);
}

}  // extern "C"

namespace fp4q {

void set_last_hip_error(int e) { g_last_hip_error = e; }

// fp4q_quantize's argument checks other than the workspace (host only).
int quantize_checks(int fmt, int layout, const uint16_t* x, int64_t rows, int64_t cols,
                    int64_t ldx, const int32_t* group_offsets, int32_t num_groups,
                    const int32_t* chan_idx, int32_t n_chan, const uint8_t* q,
                    const uint8_t* scales, const float* tensor_scale, const uint16_t* resid) {
  if (!fmt_ok(fmt) || !layout_ok(layout)) return FP4Q_ERR_INVALID;
  const int blk = blk_of(fmt);
  if (rows < 0 || cols <= 0 || cols % blk != 0 || ldx < cols || ldx % 8 != 0)
    return FP4Q_ERR_INVALID;
  if (layout == FP4Q_LAYOUT_TILED && cols % 128 != 0) return FP4Q_ERR_INVALID;
  if (num_groups < 1 || (num_groups > 1 && !group_offsets)) return FP4Q_ERR_INVALID;
  if (n_chan < 0 || n_chan > cols) return FP4Q_ERR_INVALID;
  if ((n_chan > 0) != (chan_idx != nullptr) || (n_chan > 0) != (resid != nullptr))
    return FP4Q_ERR_INVALID;
  if (fmt == FP4Q_NVFP4 && !tensor_scale) return FP4Q_ERR_INVALID;
  if (fmt == FP4Q_MXFP4 && tensor_scale) return FP4Q_ERR_INVALID;
  if (rows > 0 && (!x || !q || !scales)) return FP4Q_ERR_INVALID;
  if (rows > 0 && (!aligned(x, 16) || !aligned(q, 16) || !aligned(scales, 4)))
    return FP4Q_ERR_INVALID;
  const int64_t prow = layout == FP4Q_LAYOUT_TILED ? (rows + 15) / 16 * 16 : rows;
  if (prow * (cols / 8) >= ((int64_t)1 << 31)) return FP4Q_ERR_UNSUPPORTED;  // 32-bit chunk index
  return FP4Q_OK;
}

}  // namespace fp4q

extern "C" {

int fp4q_quantize(fp4q_format_t fmt, fp4q_layout_t layout, const uint16_t* x, int64_t rows,
                  int64_t cols, int64_t ldx, const int32_t* group_offsets, int32_t num_groups,
                  const int32_t* chan_idx, int32_t n_chan, uint8_t* q, uint8_t* scales,
                  float* tensor_scale, uint16_t* resid, void* workspace, size_t workspace_bytes,
                  void* stream) {
  const int rc = fp4q::quantize_checks(fmt, layout, x, rows, cols, ldx, group_offsets, num_groups,
                                       chan_idx, n_chan, q, scales, tensor_scale, resid);
  if (rc != FP4Q_OK) return rc;
  const size_t need = fp4q_quantize_workspace_bytes(fmt, rows, cols, num_groups);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 8)))
    return FP4Q_ERR_WORKSPACE;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  fp4q::launch_quantize(fmt, layout == FP4Q_LAYOUT_TILED, x, rows, cols, ldx, group_offsets,
                        num_groups, chan_idx, n_chan, q, scales, tensor_scale, resid, workspace,
                        static_cast<hipStream_t>(stream));
  return check_launch();
}

size_t fp4q_qdq_fallback_workspace_bytes(fp4q_format_t fmt, int64_t rows, int64_t cols) {
  (void)rows;
  (void)cols;
  return fp4q::quantize_workspace_bytes(fmt, 1);
}

int fp4q_qdq_fallback(fp4q_format_t fmt, const uint16_t* x, int64_t rows, int64_t cols,
                      int64_t ldx, float* y, int64_t ldy, int64_t* n_fallback, void* workspace,
                      size_t workspace_bytes, void* stream) {
  if (!fmt_ok(fmt)) return FP4Q_ERR_INVALID;
  if (rows < 0 || cols <= 0 || cols % blk_of(fmt) != 0 || ldx < cols || ldx % 8 != 0)
    return FP4Q_ERR_INVALID;
  if (ldy < cols || ldy % 4 != 0) return FP4Q_ERR_INVALID;
  if (rows > 0 && (!x || !y || !aligned(x, 16) || !aligned(y, 16))) return FP4Q_ERR_INVALID;
  if (n_fallback && !aligned(n_fallback, 8)) return FP4Q_ERR_INVALID;
  if (rows * (cols / 8) >= ((int64_t)1 << 31)) return FP4Q_ERR_UNSUPPORTED;
  const size_t need = fp4q_qdq_fallback_workspace_bytes(fmt, rows, cols);
  if (need > 0 && rows > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 8)))
    return FP4Q_ERR_WORKSPACE;
  if (rows == 0 && !n_fallback) return FP4Q_OK;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  fp4q::launch_qdq_fallback(fmt, x, rows, cols, ldx, y, ldy, n_fallback, workspace,
                            static_cast<hipStream_t>(stream));
  return check_launch();
}

int fp4q_quantize_status(const void* workspace, size_t workspace_bytes, int32_t* status,
                         void* stream) {
  if (!status) return FP4Q_ERR_INVALID;
  if (!workspace || !aligned(workspace, 8) ||
      workspace_bytes < fp4q_quantize_workspace_bytes(FP4Q_NVFP4, 0, 16, 1))
    return FP4Q_ERR_WORKSPACE;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  uint32_t v = 0;
  if (fp4q::quantize_status(workspace, static_cast<hipStream_t>(stream), &v) != 0) {
    const hipError_t e = hipGetLastError();
    g_last_hip_error = e != hipSuccess ? (int)e : (int)hipErrorUnknown;
    return FP4Q_ERR_HIP;
  }
  *status = (int32_t)v;
  return FP4Q_OK;
}

int fp4q_test_hook(int32_t hook, int64_t value) {
  switch (hook) {
    case FP4Q_HOOK_RESET:
      g_fail_next.store(0);
      fp4q::set_grid_hooks(0, -1);
      return FP4Q_OK;
    case FP4Q_HOOK_FAIL_NEXT_LAUNCH:
      if (value <= 0 || value > INT32_MAX) return FP4Q_ERR_INVALID;
      g_fail_next.store((int)value);
      return FP4Q_OK;
    case FP4Q_HOOK_GRID_SPIN_LIMIT:
      if (value < 0 || value > UINT32_MAX) return FP4Q_ERR_INVALID;
      fp4q::set_grid_hooks((uint32_t)value, fp4q::grid_hook_skip());
      return FP4Q_OK;
    case FP4Q_HOOK_GRID_SKIP_SLOT:
      if (value < -1 || value > 1 << 20) return FP4Q_ERR_INVALID;
      fp4q::set_grid_hooks(fp4q::grid_hook_spin(), (int)value);
      return FP4Q_OK;
    default:
      return FP4Q_ERR_INVALID;
  }
}

static int validate_gemm_common(int fmt, int64_t N, int64_t K, const uint8_t* a_q,
                                const uint8_t* a_s, const float* a_ts, const uint8_t* b_q,
                                const uint8_t* b_s, const float* b_ts, const int32_t* chan_idx,
                                int32_t n_chan, const uint16_t* resid, const void* y,
                                int y_dtype, int64_t rows) {
  if (!fmt_ok(fmt)) return FP4Q_ERR_INVALID;
  if (y_dtype != FP4Q_OUT_F32 && y_dtype != FP4Q_OUT_BF16) return FP4Q_ERR_INVALID;
  if (rows < 0 || N < 0 || K <= 0 || K % blk_of(fmt) != 0) return FP4Q_ERR_INVALID;
  if (n_chan < 0 || n_chan > K) return FP4Q_ERR_INVALID;
  if ((n_chan > 0) != (chan_idx != nullptr) || (n_chan > 0) != (resid != nullptr))
    return FP4Q_ERR_INVALID;
  if (n_chan > 0 && !aligned(resid, 16)) return FP4Q_ERR_INVALID;
  if (fmt == FP4Q_NVFP4 && (!a_ts || !b_ts)) return FP4Q_ERR_INVALID;
  if (fmt == FP4Q_MXFP4 && (a_ts || b_ts)) return FP4Q_ERR_INVALID;
  if (rows > 0 && N > 0) {
    if (!a_q || !a_s || !b_q || !b_s || !y) return FP4Q_ERR_INVALID;
    if (!aligned(a_q, 16) || !aligned(b_q, 16) || !aligned(a_s, 8) || !aligned(b_s, 8))
      return FP4Q_ERR_INVALID;
  }
  if (K % 128 != 0) return FP4Q_ERR_UNSUPPORTED;
  return FP4Q_OK;
}

// The experts' weight layout of a grouped GEMM: row-major everywhere; tiled
// where the 128 x 512 NVFP4 grouped kernel serves the shape (its tokens'
// codes below 4 GiB when gathered).
static int validate_w_layout(int fmt, int w_layout, int64_t N, int64_t K, int32_t n_chan,
                             int64_t gather_bytes = 0) {
  if (!layout_ok(w_layout)) return FP4Q_ERR_INVALID;
  if (w_layout != FP4Q_LAYOUT_TILED) return FP4Q_OK;
  if (K % 128 != 0) return FP4Q_ERR_INVALID;
  if (!fp4q::grouped_tiled_ok(fmt, N, K, n_chan) || gather_bytes > (int64_t)UINT32_MAX)
    return FP4Q_ERR_UNSUPPORTED;
  return FP4Q_OK;
}

size_t fp4q_gemm_workspace_bytes(fp4q_format_t fmt, fp4q_layout_t layout, int64_t M, int64_t N,
                                 int64_t K, int32_t n_chan) {
  (void)fmt;
  (void)layout;
  if (M <= 0 || N <= 0 || K <= 0 || n_chan <= 0) return 0;
  return fp4q::gemm_workspace_bytes(M, N, K, n_chan);
}

int fp4q_gemm(fp4q_format_t fmt, fp4q_layout_t layout, int64_t M, int64_t N, int64_t K,
              const uint8_t* a_q, const uint8_t* a_s, const float* a_ts, const uint8_t* b_q,
              const uint8_t* b_s, const float* b_ts, const int32_t* chan_idx, int32_t n_chan,
              const uint16_t* resid, void* y, fp4q_dtype_t y_dtype, int64_t ldy, void* workspace,
              size_t workspace_bytes, void* stream) {
  if (!layout_ok(layout)) return FP4Q_ERR_INVALID;
  int rc = validate_gemm_common(fmt, N, K, a_q, a_s, a_ts, b_q, b_s, b_ts, chan_idx, n_chan,
                                resid, y, y_dtype, M);
  if (rc != FP4Q_OK) return rc;
  if (ldy < N) return FP4Q_ERR_INVALID;
  if ((M + 127) / 128 > (int64_t)UINT32_MAX || (N + 31) / 32 > 65535) return FP4Q_ERR_UNSUPPORTED;
  const size_t need = fp4q_gemm_workspace_bytes(fmt, layout, M, N, K, n_chan);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
    return FP4Q_ERR_WORKSPACE;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  fp4q::launch_gemm(fmt, layout == FP4Q_LAYOUT_TILED, M, N, K, nullptr, 1, a_q, a_s, a_ts, b_q,
                    b_s, b_ts, chan_idx, n_chan, resid, nullptr, y, y_dtype == FP4Q_OUT_BF16, ldy,
                    workspace, static_cast<hipStream_t>(stream));
  return check_launch();
}

size_t fp4q_comp_weights_bytes(fp4q_format_t fmt, fp4q_layout_t layout, int64_t N, int64_t K,
                               int32_t n_chan) {
  (void)fmt;
  (void)layout;
  (void)K;
  return fp4q::comp_weights_bytes(N, n_chan);
}

int fp4q_comp_weights(fp4q_format_t fmt, fp4q_layout_t layout, int64_t N, int64_t K,
                      const uint8_t* b_q, const uint8_t* b_s, const int32_t* chan_idx,
                      int32_t n_chan, uint8_t* out, size_t out_bytes, void* stream) {
  if (!layout_ok(layout) || !fmt_ok(fmt)) return FP4Q_ERR_INVALID;
  if (N < 0 || K < 0 || n_chan < 0) return FP4Q_ERR_INVALID;
  if ((n_chan > 0) != (chan_idx != nullptr)) return FP4Q_ERR_INVALID;
  if (N == 0 || n_chan == 0) return FP4Q_OK;
  if (!b_q || !b_s || !out || !aligned(out, 16)) return FP4Q_ERR_INVALID;
  if (K % 128 != 0) return FP4Q_ERR_UNSUPPORTED;
  if (out_bytes < fp4q_comp_weights_bytes(fmt, layout, N, K, n_chan)) return FP4Q_ERR_WORKSPACE;
  if (((N + 15) / 16) * ((n_chan + 31) / 32) / 4 >= (int64_t)UINT32_MAX)
    return FP4Q_ERR_UNSUPPORTED;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  fp4q::launch_comp_weights(fmt, layout == FP4Q_LAYOUT_TILED, b_q, b_s, N, K, chan_idx, n_chan, 1,
                            out, static_cast<hipStream_t>(stream));
  return check_launch();
}

int fp4q_gemm_prepared(fp4q_format_t fmt, fp4q_layout_t layout, int64_t M, int64_t N, int64_t K,
                       const uint8_t* a_q, const uint8_t* a_s, const float* a_ts,
                       const uint8_t* b_q, const uint8_t* b_s, const float* b_ts,
                       const int32_t* chan_idx, int32_t n_chan, const uint16_t* resid,
                       const uint8_t* comp_w, size_t comp_w_bytes, void* y,
                       fp4q_dtype_t y_dtype, int64_t ldy, void* stream) {
  if (!layout_ok(layout)) return FP4Q_ERR_INVALID;
  int rc = validate_gemm_common(fmt, N, K, a_q, a_s, a_ts, b_q, b_s, b_ts, chan_idx, n_chan,
                                resid, y, y_dtype, M);
  if (rc != FP4Q_OK) return rc;
  if (ldy < N) return FP4Q_ERR_INVALID;
  if ((M + 127) / 128 > (int64_t)UINT32_MAX || (N + 31) / 32 > 65535) return FP4Q_ERR_UNSUPPORTED;
  const bool work = M > 0 && N > 0 && n_chan > 0;
  if (work && (!comp_w || !aligned(comp_w, 16) ||
               comp_w_bytes < fp4q_comp_weights_bytes(fmt, layout, N, K, n_chan)))
    return FP4Q_ERR_WORKSPACE;
  // shapes whose kernels stream no compensation weights take the term from
  // chan_idx as fp4q_gemm does (they need no workspace)
  if (fp4q::gemm_path(M, N, K, n_chan) == fp4q::PATH_GENERIC) comp_w = nullptr;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  fp4q::launch_gemm(fmt, layout == FP4Q_LAYOUT_TILED, M, N, K, nullptr, 1, a_q, a_s, a_ts, b_q,
                    b_s, b_ts, chan_idx, n_chan, resid, nullptr, y, y_dtype == FP4Q_OUT_BF16, ldy,
                    nullptr, static_cast<hipStream_t>(stream), work ? comp_w : nullptr);
  return check_launch();
}

int fp4q_gemm_decode_fused(fp4q_format_t fmt, fp4q_layout_t layout, int64_t M, int64_t N,
                           int64_t K, const uint16_t* x, int64_t ldx, const uint8_t* b_q,
                           const uint8_t* b_s, const float* b_ts, const int32_t* chan_idx,
                           int32_t n_chan, const uint8_t* comp_w, size_t comp_w_bytes, void* y,
                           fp4q_dtype_t y_dtype, int64_t ldy, uint8_t* a_q_out,
                           uint8_t* a_s_out, float* a_ts_out, uint16_t* resid_out,
                           void* stream) {
  if (!fmt_ok(fmt) || !layout_ok(layout)) return FP4Q_ERR_INVALID;
  if (y_dtype != FP4Q_OUT_F32 && y_dtype != FP4Q_OUT_BF16) return FP4Q_ERR_INVALID;
  if (M < 0 || N < 0 || K <= 0 || K % 16 != 0 || ldx < K || ldx % 8 != 0 || ldy < N)
    return FP4Q_ERR_INVALID;
  if (n_chan < 0 || n_chan > K || (n_chan > 0) != (chan_idx != nullptr)) return FP4Q_ERR_INVALID;
  if (!b_ts) return FP4Q_ERR_INVALID;
  const bool outs = a_q_out != nullptr;
  if (outs != (a_s_out != nullptr) || outs != (a_ts_out != nullptr) ||
      (outs && n_chan > 0) != (resid_out != nullptr))
    return FP4Q_ERR_INVALID;
  if (M > 0 && N > 0) {
    if (!x || !b_q || !b_s || !y) return FP4Q_ERR_INVALID;
    if (!aligned(x, 16) || !aligned(b_q, 16) || !aligned(b_s, 8)) return FP4Q_ERR_INVALID;
    if (outs && (!aligned(a_q_out, 16) || !aligned(a_s_out, 2))) return FP4Q_ERR_INVALID;
  }
  if (fmt != FP4Q_NVFP4 || K % 128 != 0 || !fp4q::decode_fused_eligible(M > 0 ? M : 1, K, n_chan))
    return FP4Q_ERR_UNSUPPORTED;
  if ((N + 47) / 48 > (int64_t)INT32_MAX) return FP4Q_ERR_UNSUPPORTED;
  const bool work = M > 0 && N > 0;
  if (work && n_chan > 0 &&
      (!comp_w || !aligned(comp_w, 16) ||
       comp_w_bytes < fp4q_comp_weights_bytes(fmt, layout, N, K, n_chan)))
    return FP4Q_ERR_WORKSPACE;
  if (!work) return FP4Q_OK;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  fp4q::launch_gemm_decode_fused(layout == FP4Q_LAYOUT_TILED, M, N, K, x, ldx, b_q, b_s, b_ts,
                                 chan_idx, n_chan, n_chan > 0 ? comp_w : nullptr, y,
                                 y_dtype == FP4Q_OUT_BF16, ldy, a_q_out, a_s_out, a_ts_out,
                                 resid_out, static_cast<hipStream_t>(stream));
  return check_launch();
}

static size_t deq_resid_bytes(int64_t M, int32_t n_chan) {
  return (size_t)((M * n_chan * 2 + 255) / 256 * 256);
}

size_t fp4q_gemm_residual_fp4_workspace_bytes(fp4q_format_t fmt, fp4q_layout_t layout, int64_t M,
                                              int64_t N, int64_t K, int32_t n_chan) {
  if (M <= 0 || N <= 0 || K <= 0 || n_chan <= 0) return 0;
  return deq_resid_bytes(M, n_chan) + fp4q_gemm_workspace_bytes(fmt, layout, M, N, K, n_chan);
}

int fp4q_gemm_residual_fp4(fp4q_format_t fmt, fp4q_layout_t layout, int64_t M, int64_t N,
                           int64_t K, const uint8_t* a_q, const uint8_t* a_s, const float* a_ts,
                           const uint8_t* b_q, const uint8_t* b_s, const float* b_ts,
                           const int32_t* chan_idx, int32_t n_chan, const uint8_t* r_q,
                           const uint8_t* r_s, const float* r_ts, void* y, fp4q_dtype_t y_dtype,
                           int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  if (!layout_ok(layout) || !fmt_ok(fmt)) return FP4Q_ERR_INVALID;
  if (n_chan < 0 || (n_chan > 0) != (r_q != nullptr) || (n_chan > 0) != (r_s != nullptr))
    return FP4Q_ERR_INVALID;
  if (n_chan % blk_of(fmt) != 0) return FP4Q_ERR_INVALID;
  if (fmt == FP4Q_NVFP4 && (n_chan > 0) != (r_ts != nullptr)) return FP4Q_ERR_INVALID;
  if (fmt == FP4Q_MXFP4 && r_ts) return FP4Q_ERR_INVALID;
  const bool work = M > 0 && N > 0 && n_chan > 0;
  const size_t need = work ? fp4q_gemm_residual_fp4_workspace_bytes(fmt, layout, M, N, K, n_chan)
                           : 0;
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
    return FP4Q_ERR_WORKSPACE;
  // the decoded residual goes to the front of the workspace; it stands in
  // for fp4q_gemm's resid in the shared validation (an empty product only
  // needs a non-null stand-in, never read)
  alignas(16) static const uint16_t kNoRows[8] = {};
  uint16_t* rdeq = work ? static_cast<uint16_t*>(workspace) : nullptr;
  const uint16_t* rval = work ? rdeq : (n_chan > 0 ? kNoRows : nullptr);
  int rc = validate_gemm_common(fmt, N, K, a_q, a_s, a_ts, b_q, b_s, b_ts, chan_idx, n_chan,
                                rval, y, y_dtype, M);
  if (rc != FP4Q_OK) return rc;
  if (ldy < N) return FP4Q_ERR_INVALID;
  if ((M + 127) / 128 > (int64_t)UINT32_MAX || (N + 31) / 32 > 65535) return FP4Q_ERR_UNSUPPORTED;
  if (M * (int64_t)n_chan / 8 >= ((int64_t)1 << 31)) return FP4Q_ERR_UNSUPPORTED;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  void* gws = work ? static_cast<uint8_t*>(workspace) + deq_resid_bytes(M, n_chan) : nullptr;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (work) fp4q::launch_deq_resid(fmt, M, n_chan, r_q, r_s, rdeq, st);
  fp4q::launch_gemm(fmt, layout == FP4Q_LAYOUT_TILED, M, N, K, nullptr, 1, a_q, a_s, a_ts, b_q,
                    b_s, b_ts, chan_idx, n_chan, rval, r_ts, y, y_dtype == FP4Q_OUT_BF16, ldy, gws,
                    st);
  return check_launch();
}

size_t fp4q_grouped_gemm_workspace_bytes(fp4q_format_t fmt, fp4q_layout_t w_layout,
                                         int64_t total_rows, int64_t N, int64_t K,
                                         int32_t num_groups, int32_t n_chan) {
  (void)fmt;
  (void)w_layout;
  if (total_rows <= 0 || N <= 0 || K <= 0 || n_chan <= 0 || num_groups < 1) return 0;
  return fp4q::grouped_workspace_bytes(N, K, num_groups, n_chan);
}

int fp4q_grouped_gemm(fp4q_format_t fmt, fp4q_layout_t w_layout, int64_t total_rows, int64_t N,
                      int64_t K, const int32_t* group_offsets, int32_t num_groups,
                      const uint8_t* a_q,
                      const uint8_t* a_s, const float* a_ts, const uint8_t* b_q,
                      const uint8_t* b_s, const float* b_ts, const int32_t* chan_idx,
                      int32_t n_chan, const uint16_t* resid, void* y, fp4q_dtype_t y_dtype,
                      void* workspace, size_t workspace_bytes, void* stream) {
  int rc = validate_gemm_common(fmt, N, K, a_q, a_s, a_ts, b_q, b_s, b_ts, chan_idx, n_chan,
                                resid, y, y_dtype, total_rows);
  if (rc != FP4Q_OK) return rc;
  if ((rc = validate_w_layout(fmt, w_layout, N, K, n_chan)) != FP4Q_OK) return rc;
  if (num_groups < 1 || !group_offsets) return FP4Q_ERR_INVALID;
  if (num_groups > MAX_GROUPS) return FP4Q_ERR_UNSUPPORTED;
  if ((N + 127) / 128 > 65535) return FP4Q_ERR_UNSUPPORTED;
  const size_t need =
      fp4q_grouped_gemm_workspace_bytes(fmt, w_layout, total_rows, N, K, num_groups, n_chan);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
    return FP4Q_ERR_WORKSPACE;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  fp4q::launch_gemm(fmt, w_layout == FP4Q_LAYOUT_TILED, total_rows, N, K, group_offsets,
                    num_groups, a_q, a_s, a_ts, b_q,
                    b_s, b_ts, chan_idx, n_chan, resid, nullptr, y, y_dtype == FP4Q_OUT_BF16, N,
                    workspace, static_cast<hipStream_t>(stream));
  return check_launch();
}

size_t fp4q_grouped_gemm_residual_fp4_workspace_bytes(fp4q_format_t fmt,
                                                      fp4q_layout_t w_layout,
                                                      int64_t total_rows, int64_t N, int64_t K,
                                                      int32_t num_groups, int32_t n_chan) {
  if (total_rows <= 0 || N <= 0 || K <= 0 || n_chan <= 0 || num_groups < 1) return 0;
  return deq_resid_bytes(total_rows, n_chan) +
         fp4q_grouped_gemm_workspace_bytes(fmt, w_layout, total_rows, N, K, num_groups, n_chan);
}

int fp4q_grouped_gemm_residual_fp4(fp4q_format_t fmt, fp4q_layout_t w_layout,
                                   int64_t total_rows, int64_t N, int64_t K,
                                   const int32_t* group_offsets, int32_t num_groups,
                                   const uint8_t* a_q, const uint8_t* a_s, const float* a_ts,
                                   const uint8_t* b_q, const uint8_t* b_s, const float* b_ts,
                                   const int32_t* chan_idx, int32_t n_chan, const uint8_t* r_q,
                                   const uint8_t* r_s, const float* r_ts, void* y,
                                   fp4q_dtype_t y_dtype, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  if (!fmt_ok(fmt)) return FP4Q_ERR_INVALID;
  if (n_chan < 0 || (n_chan > 0) != (r_q != nullptr) || (n_chan > 0) != (r_s != nullptr))
    return FP4Q_ERR_INVALID;
  if (n_chan % blk_of(fmt) != 0) return FP4Q_ERR_INVALID;
  if (fmt == FP4Q_NVFP4 && (n_chan > 0) != (r_ts != nullptr)) return FP4Q_ERR_INVALID;
  if (fmt == FP4Q_MXFP4 && r_ts) return FP4Q_ERR_INVALID;
  if (num_groups < 1 || !group_offsets) return FP4Q_ERR_INVALID;
  if (num_groups > MAX_GROUPS) return FP4Q_ERR_UNSUPPORTED;
  const bool work = total_rows > 0 && N > 0 && n_chan > 0;
  const size_t need = work ? fp4q_grouped_gemm_residual_fp4_workspace_bytes(
                                 fmt, w_layout, total_rows, N, K, num_groups, n_chan)
                           : 0;
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
    return FP4Q_ERR_WORKSPACE;
  // the decoded residual goes to the front of the workspace and stands in
  // for fp4q_grouped_gemm's resid (an empty product only needs a non-null
  // stand-in, never read)
  alignas(16) static const uint16_t kNoRows[8] = {};
  uint16_t* rdeq = work ? static_cast<uint16_t*>(workspace) : nullptr;
  const uint16_t* rval = work ? rdeq : (n_chan > 0 ? kNoRows : nullptr);
  int rc = validate_gemm_common(fmt, N, K, a_q, a_s, a_ts, b_q, b_s, b_ts, chan_idx, n_chan,
                                rval, y, y_dtype, total_rows);
  if (rc != FP4Q_OK) return rc;
  if ((rc = validate_w_layout(fmt, w_layout, N, K, n_chan)) != FP4Q_OK) return rc;
  if ((N + 127) / 128 > 65535) return FP4Q_ERR_UNSUPPORTED;
  if (total_rows * (int64_t)n_chan / 8 >= ((int64_t)1 << 31)) return FP4Q_ERR_UNSUPPORTED;
  if (total_rows == 0 || N == 0) return FP4Q_OK;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  void* gws = work ? static_cast<uint8_t*>(workspace) + deq_resid_bytes(total_rows, n_chan)
                   : nullptr;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (work) fp4q::launch_deq_resid(fmt, total_rows, n_chan, r_q, r_s, rdeq, st);
  fp4q::launch_gemm(fmt, w_layout == FP4Q_LAYOUT_TILED, total_rows, N, K, group_offsets,
                    num_groups, a_q, a_s, a_ts, b_q,
                    b_s, b_ts, chan_idx, n_chan, rval, r_ts, y, y_dtype == FP4Q_OUT_BF16, N, gws,
                    st);
  return check_launch();
}

size_t fp4q_grouped_comp_weights_bytes(fp4q_format_t fmt, int64_t N, int64_t K,
                                       int32_t num_groups, int32_t n_chan) {
  (void)fmt;
  (void)K;
  if (num_groups < 1) return 0;
  return (size_t)num_groups * fp4q::comp_weights_bytes(N, n_chan);
}

int fp4q_grouped_comp_weights(fp4q_format_t fmt, fp4q_layout_t w_layout, int64_t N, int64_t K,
                              int32_t num_groups, const uint8_t* b_q, const uint8_t* b_s,
                              const int32_t* chan_idx, int32_t n_chan, uint8_t* out,
                              size_t out_bytes, void* stream) {
  if (!fmt_ok(fmt) || !layout_ok(w_layout)) return FP4Q_ERR_INVALID;
  if (N < 0 || K < 0 || n_chan < 0 || num_groups < 1) return FP4Q_ERR_INVALID;
  if (num_groups > MAX_GROUPS) return FP4Q_ERR_UNSUPPORTED;
  if ((n_chan > 0) != (chan_idx != nullptr)) return FP4Q_ERR_INVALID;
  if (N == 0 || n_chan == 0) return FP4Q_OK;
  if (!b_q || !b_s || !out || !aligned(out, 16)) return FP4Q_ERR_INVALID;
  if (K % 128 != 0) return FP4Q_ERR_UNSUPPORTED;
  if (out_bytes < fp4q_grouped_comp_weights_bytes(fmt, N, K, num_groups, n_chan))
    return FP4Q_ERR_WORKSPACE;
  if ((int64_t)num_groups * ((N + 15) / 16) * ((n_chan + 31) / 32) / 4 >= (int64_t)UINT32_MAX)
    return FP4Q_ERR_UNSUPPORTED;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  fp4q::launch_comp_weights(fmt, w_layout == FP4Q_LAYOUT_TILED, b_q, b_s, N, K, chan_idx,
                            n_chan, num_groups, out, static_cast<hipStream_t>(stream));
  return check_launch();
}

int fp4q_grouped_gemm_prepared(fp4q_format_t fmt, fp4q_layout_t w_layout, int64_t total_rows,
                               int64_t N, int64_t K, const int32_t* group_offsets,
                               int32_t num_groups,
                               const uint8_t* a_q, const uint8_t* a_s, const float* a_ts,
                               const uint8_t* b_q, const uint8_t* b_s, const float* b_ts,
                               const int32_t* chan_idx, int32_t n_chan, const uint16_t* resid,
                               const uint8_t* comp_w, size_t comp_w_bytes, void* y,
                               fp4q_dtype_t y_dtype, void* stream) {
  int rc = validate_gemm_common(fmt, N, K, a_q, a_s, a_ts, b_q, b_s, b_ts, chan_idx, n_chan,
                                resid, y, y_dtype, total_rows);
  if (rc != FP4Q_OK) return rc;
  if ((rc = validate_w_layout(fmt, w_layout, N, K, n_chan)) != FP4Q_OK) return rc;
  if (num_groups < 1 || !group_offsets) return FP4Q_ERR_INVALID;
  if (num_groups > MAX_GROUPS) return FP4Q_ERR_UNSUPPORTED;
  if ((N + 127) / 128 > 65535) return FP4Q_ERR_UNSUPPORTED;
  const bool work = total_rows > 0 && N > 0 && n_chan > 0;
  if (work && (!comp_w || !aligned(comp_w, 16) ||
               comp_w_bytes < fp4q_grouped_comp_weights_bytes(fmt, N, K, num_groups, n_chan)))
    return FP4Q_ERR_WORKSPACE;
  // shapes served by the general grouped kernel take the term from chan_idx
  if (!fp4q::big_grouped_eligible(N, K, n_chan)) comp_w = nullptr;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  fp4q::launch_gemm(fmt, w_layout == FP4Q_LAYOUT_TILED, total_rows, N, K, group_offsets,
                    num_groups, a_q, a_s, a_ts, b_q, b_s, b_ts, chan_idx, n_chan, resid, nullptr,
                    y, y_dtype == FP4Q_OUT_BF16, N, nullptr, static_cast<hipStream_t>(stream),
                    work ? comp_w : nullptr);
  return check_launch();
}

int fp4q_grouped_gemm_gather(fp4q_format_t fmt, fp4q_layout_t w_layout, int64_t total_rows,
                             int64_t N, int64_t K, const int32_t* group_offsets,
                             int32_t num_groups,
                             const int32_t* row_src, int64_t tokens, const uint8_t* a_q,
                             const uint8_t* a_s, const float* a_ts, const uint8_t* b_q,
                             const uint8_t* b_s, const float* b_ts, const int32_t* chan_idx,
                             int32_t n_chan, const uint16_t* resid, const uint8_t* comp_w,
                             size_t comp_w_bytes, void* y, fp4q_dtype_t y_dtype, void* stream) {
  int rc = validate_gemm_common(fmt, N, K, a_q, a_s, a_ts, b_q, b_s, b_ts, chan_idx, n_chan,
                                resid, y, y_dtype, total_rows);
  if (rc != FP4Q_OK) return rc;
  if (num_groups < 1 || !group_offsets) return FP4Q_ERR_INVALID;
  if (tokens < 0 || (total_rows > 0 && (tokens == 0 || !row_src))) return FP4Q_ERR_INVALID;
  if ((rc = validate_w_layout(fmt, w_layout, N, K, n_chan, tokens * (K / 2))) != FP4Q_OK)
    return rc;
  if (num_groups > MAX_GROUPS) return FP4Q_ERR_UNSUPPORTED;
  if ((N + 127) / 128 > 65535 || !fp4q::big_grouped_eligible(N, K, n_chan))
    return FP4Q_ERR_UNSUPPORTED;
  const bool work = total_rows > 0 && N > 0;
  if (work && n_chan > 0 &&
      (!comp_w || !aligned(comp_w, 16) ||
       comp_w_bytes < fp4q_grouped_comp_weights_bytes(fmt, N, K, num_groups, n_chan)))
    return FP4Q_ERR_WORKSPACE;
  if (!work) return FP4Q_OK;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  fp4q::launch_gemm_big_grouped(fmt, total_rows, N, K, group_offsets, num_groups, a_q, a_s, a_ts,
                                b_q, b_s, b_ts, chan_idx, n_chan, resid, nullptr,
                                n_chan > 0 ? comp_w : nullptr, y, y_dtype == FP4Q_OUT_BF16, nullptr,
                                static_cast<hipStream_t>(stream), w_layout == FP4Q_LAYOUT_TILED,
                                row_src, tokens);
  return check_launch();
}

size_t fp4q_select_channels_workspace_bytes(int64_t rows, int64_t cols) {
  return fp4q::select_workspace_bytes(rows, cols);
}

int fp4q_select_channels(fp4q_format_t fmt, fp4q_layout_t layout, const uint16_t* x,
                         int64_t rows, int64_t cols, int64_t ldx, const uint8_t* q,
                         const uint8_t* scales, const float* tensor_scale, int32_t k,
                         int32_t* chan_out, uint16_t* resid_out, void* workspace,
                         size_t workspace_bytes, void* stream) {
  if (!fmt_ok(fmt) || !layout_ok(layout)) return FP4Q_ERR_INVALID;
  if (rows < 0 || cols <= 0 || cols % blk_of(fmt) != 0 || ldx < cols || ldx % 8 != 0)
    return FP4Q_ERR_INVALID;
  if (layout == FP4Q_LAYOUT_TILED && cols % 128 != 0) return FP4Q_ERR_INVALID;
  if (k < 0 || k > cols) return FP4Q_ERR_INVALID;
  if (fmt == FP4Q_NVFP4 && !tensor_scale) return FP4Q_ERR_INVALID;
  if (fmt == FP4Q_MXFP4 && tensor_scale) return FP4Q_ERR_INVALID;
  if (k > 0 && (!chan_out || !aligned(chan_out, 4))) return FP4Q_ERR_INVALID;
  if (rows > 0 && k > 0 && (!resid_out || !aligned(resid_out, 2))) return FP4Q_ERR_INVALID;
  if (rows > 0 && (!x || !q || !scales)) return FP4Q_ERR_INVALID;
  if (rows > 0 && (!aligned(x, 16) || !aligned(q, 4))) return FP4Q_ERR_INVALID;
  if (cols > INT32_MAX || rows * (int64_t)k >= ((int64_t)1 << 31)) return FP4Q_ERR_UNSUPPORTED;
  if (k == 0) return FP4Q_OK;
  const size_t need = fp4q::select_workspace_bytes(rows, cols);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return FP4Q_ERR_WORKSPACE;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  fp4q::launch_select(fmt, layout == FP4Q_LAYOUT_TILED, x, rows, cols, ldx, q, scales,
                      tensor_scale, k, chan_out, resid_out, workspace,
                      static_cast<hipStream_t>(stream));
  return check_launch();
}

static size_t round256_sz(size_t b) { return (b + 255) / 256 * 256; }

size_t fp4q_quantize_select_workspace_bytes(fp4q_format_t fmt, fp4q_layout_t layout,
                                            int64_t rows, int64_t cols) {
  if (!fmt_ok(fmt) || !layout_ok(layout) || rows < 0 || cols <= 0) return 0;
  const size_t qb = round256_sz(fp4q_quantize_workspace_bytes(fmt, rows, cols, 1));
  size_t sb = fp4q::select_workspace_bytes(rows, cols);
  if (rows > 0 && cols % 32 == 0) {
    const int64_t bands = fp4q::quantize_score_bands(layout == FP4Q_LAYOUT_TILED, rows, cols);
    sb = std::max(sb, fp4q::select_scored_workspace_bytes(bands, cols));
  }
  return qb + sb;
}

int fp4q_quantize_select(fp4q_format_t fmt, fp4q_layout_t layout, const uint16_t* x,
                         int64_t rows, int64_t cols, int64_t ldx, int32_t k, uint8_t* q,
                         uint8_t* scales, float* tensor_scale, int32_t* chan_out,
                         uint16_t* resid_out, void* workspace, size_t workspace_bytes,
                         void* stream) {
  const int rc = fp4q::quantize_checks(fmt, layout, x, rows, cols, ldx, nullptr, 1, nullptr, 0, q,
                                       scales, tensor_scale, nullptr);
  if (rc != FP4Q_OK) return rc;
  if (k < 0 || k > cols || ldx % 8 != 0) return FP4Q_ERR_INVALID;
  if (k > 0 && (!chan_out || !aligned(chan_out, 4))) return FP4Q_ERR_INVALID;
  if (rows > 0 && k > 0 && (!resid_out || !aligned(resid_out, 2))) return FP4Q_ERR_INVALID;
  if (rows > 0 && (!aligned(x, 16) || !aligned(q, 4))) return FP4Q_ERR_INVALID;
  if (cols > INT32_MAX || rows * (int64_t)k >= ((int64_t)1 << 31)) return FP4Q_ERR_UNSUPPORTED;
  const size_t need = fp4q_quantize_select_workspace_bytes(fmt, layout, rows, cols);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return FP4Q_ERR_WORKSPACE;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  const bool tiled = layout == FP4Q_LAYOUT_TILED;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  void* wsq = workspace;
  void* wss = static_cast<char*>(workspace) +
              round256_sz(fp4q_quantize_workspace_bytes(fmt, rows, cols, 1));
  if (k > 0 && rows > 0 && cols % 32 == 0) {
    const int64_t bands = fp4q::launch_quantize_scored(fmt, tiled, x, rows, cols, ldx, q, scales,
                                                       tensor_scale, wsq,
                                                       static_cast<uint16_t*>(wss), st);
    fp4q::launch_select_scored(fmt, tiled, x, rows, cols, ldx, q, scales, tensor_scale, k,
                               chan_out, resid_out, static_cast<const uint16_t*>(wss), bands, wss,
                               st);
  } else {
    fp4q::launch_quantize(fmt, tiled, x, rows, cols, ldx, nullptr, 1, nullptr, 0, q, scales,
                          tensor_scale, nullptr, wsq, st);
    if (k > 0)
      fp4q::launch_select(fmt, tiled, x, rows, cols, ldx, q, scales, tensor_scale, k, chan_out,
                          resid_out, wss, st);
  }
  return check_launch();
}

size_t fp4q_select_channels_grouped_workspace_bytes(int64_t rows, int64_t cols,
                                                    int32_t num_groups) {
  return fp4q::select_grouped_workspace_bytes(rows, cols, num_groups);
}

int fp4q_select_channels_grouped(fp4q_format_t fmt, const uint16_t* x, int64_t rows, int64_t cols,
                                 int64_t ldx, const int32_t* group_offsets, int32_t num_groups,
                                 const uint8_t* q, const uint8_t* scales,
                                 const float* tensor_scale, int32_t k, int32_t* chan_out,
                                 uint16_t* resid_out, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  if (!fmt_ok(fmt)) return FP4Q_ERR_INVALID;
  if (rows < 0 || cols <= 0 || cols % blk_of(fmt) != 0 || ldx < cols || ldx % 8 != 0)
    return FP4Q_ERR_INVALID;
  if (k < 0 || k > cols) return FP4Q_ERR_INVALID;
  if (num_groups < 1 || !group_offsets) return FP4Q_ERR_INVALID;
  if (num_groups > MAX_GROUPS) return FP4Q_ERR_UNSUPPORTED;
  if (fmt == FP4Q_NVFP4 && !tensor_scale) return FP4Q_ERR_INVALID;
  if (fmt == FP4Q_MXFP4 && tensor_scale) return FP4Q_ERR_INVALID;
  if (k > 0 && (!chan_out || !aligned(chan_out, 4))) return FP4Q_ERR_INVALID;
  if (rows > 0 && k > 0 && (!resid_out || !aligned(resid_out, 2))) return FP4Q_ERR_INVALID;
  if (rows > 0 && (!x || !q || !scales)) return FP4Q_ERR_INVALID;
  if (rows > 0 && (!aligned(x, 16) || !aligned(q, 4))) return FP4Q_ERR_INVALID;
  if (!fp4q::select_grouped_cols_ok(cols)) return FP4Q_ERR_UNSUPPORTED;
  if (rows * (int64_t)k >= ((int64_t)1 << 31)) return FP4Q_ERR_UNSUPPORTED;
  if (k == 0) return FP4Q_OK;
  const size_t need = fp4q::select_grouped_workspace_bytes(rows, cols, num_groups);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return FP4Q_ERR_WORKSPACE;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  fp4q::launch_select_grouped(fmt, x, rows, cols, ldx, q, scales, tensor_scale, group_offsets,
                              num_groups, k, chan_out, resid_out, workspace,
                              static_cast<hipStream_t>(stream));
  return check_launch();
}

int fp4q_permute_quantized(fp4q_format_t fmt, const uint16_t* x, int64_t tokens, int64_t cols,
                           int64_t ldx, const uint8_t* q, const uint8_t* scales,
                           const float* tensor_scale, const int32_t* row_src, int64_t rows,
                           const int32_t* group_offsets, int32_t num_groups,
                           const int32_t* chan_idx, int32_t n_chan, uint8_t* q_out,
                           uint8_t* scales_out, float* tensor_scale_out, uint16_t* resid_out,
                           void* stream) {
  if (!fmt_ok(fmt)) return FP4Q_ERR_INVALID;
  if (tokens < 0 || rows < 0 || cols <= 0 || cols % blk_of(fmt) != 0) return FP4Q_ERR_INVALID;
  if (rows > 0 && tokens == 0) return FP4Q_ERR_INVALID;
  if (num_groups < 1 || !group_offsets) return FP4Q_ERR_INVALID;
  if (n_chan < 0 || n_chan > cols) return FP4Q_ERR_INVALID;
  if ((n_chan > 0) != (chan_idx != nullptr) || (n_chan > 0) != (resid_out != nullptr))
    return FP4Q_ERR_INVALID;
  if (fmt == FP4Q_NVFP4 && (!tensor_scale || !tensor_scale_out)) return FP4Q_ERR_INVALID;
  if (fmt == FP4Q_MXFP4 && (tensor_scale || tensor_scale_out)) return FP4Q_ERR_INVALID;
  // q_out and scales_out both NULL: the residual (and tensor scales) only,
  // for a grouped GEMM that gathers the codes itself
  if ((q_out == nullptr) != (scales_out == nullptr)) return FP4Q_ERR_INVALID;
  if (rows > 0 && (!row_src || !q || !scales)) return FP4Q_ERR_INVALID;
  if (rows > 0 && (!aligned(q, 8) || !aligned(q_out, 8))) return FP4Q_ERR_INVALID;
  if (rows > 0 && n_chan > 0 && (!x || !aligned(x, 2) || ldx < cols)) return FP4Q_ERR_INVALID;
  if (rows >= ((int64_t)1 << 31) || cols >= ((int64_t)1 << 30) || num_groups > MAX_GROUPS)
    return FP4Q_ERR_UNSUPPORTED;
  if (rows == 0 && fmt == FP4Q_MXFP4) return FP4Q_OK;  // no rows and no tensor scales to copy
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  fp4q::launch_permute(fmt, x, ldx, tokens, cols, q, scales, tensor_scale, row_src, rows,
                       group_offsets, num_groups, chan_idx, n_chan, q_out, scales_out,
                       tensor_scale_out, resid_out, static_cast<hipStream_t>(stream));
  return check_launch();
}

size_t fp4q_error_decompose_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols <= 0) return 0;
  return fp4q::decompose_workspace_bytes(rows, cols);
}

int fp4q_error_decompose(fp4q_format_t fmt, const uint16_t* x, int64_t rows, int64_t cols,
                         int64_t ldx, fp4q_err_stats_t* out, void* workspace,
                         size_t workspace_bytes, void* stream) {
  if (!fmt_ok(fmt)) return FP4Q_ERR_INVALID;
  if (rows < 0 || cols <= 0 || cols % blk_of(fmt) != 0 || ldx < cols || ldx % 8 != 0)
    return FP4Q_ERR_INVALID;
  if (!out || !aligned(out, 8)) return FP4Q_ERR_INVALID;
  if (rows > 0 && (!x || !aligned(x, 16))) return FP4Q_ERR_INVALID;
  const size_t need = fp4q::decompose_workspace_bytes(rows, cols);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return FP4Q_ERR_WORKSPACE;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  fp4q::launch_decompose(fmt, x, rows, cols, ldx, out, workspace,
                         static_cast<hipStream_t>(stream));
  return check_launch();
}

}  // extern "C"

// ---- the key/value cache, the router and the combination -------------------

namespace {

inline bool dtype_ok(int d) { return d == FP4Q_OUT_F32 || d == FP4Q_OUT_BF16; }

inline int page_shift_of(int32_t page) {
  for (int s = 4; s <= 10; ++s)
    if (page == (1 << s)) return s;
  return -1;
}

// What the cache's calls have in common, short of the packed tensors.
int kv_checks(int fmt, const uint8_t* cache, int64_t n_pages, int32_t page, int32_t kv_heads,
              int32_t dim, const int32_t* offsets, int32_t batch, const int32_t* page_table,
              int64_t ld_table,
              int64_t table_cols, const int32_t* lens, int64_t rows, const float* k_scale,
              const float* v_scale) {
  if (!fmt_ok(fmt)) return FP4Q_ERR_INVALID;
  if (n_pages < 0 || page < 1 || kv_heads < 1 || dim < 1 || batch < 0 || table_cols < 0 || rows < 0 ||
      ld_table < (batch > 1 ? table_cols : 0))
    return FP4Q_ERR_INVALID;
  if (fmt == FP4Q_NVFP4 ? (!k_scale || !v_scale) : (k_scale || v_scale)) return FP4Q_ERR_INVALID;
  if (rows > 0 && (n_pages < 1 || batch < 1 || table_cols < 1)) return FP4Q_ERR_INVALID;
  if (rows > 0 && (!cache || !offsets || !page_table || !lens || !aligned(cache, 16)))
    return FP4Q_ERR_INVALID;
  if (page_shift_of(page) < 0 || (dim != 64 && dim != 128 && dim != 256))
    return FP4Q_ERR_UNSUPPORTED;
  if (kv_heads >= (1 << 20) || table_cols >= ((int64_t)1 << 31) / page) return FP4Q_ERR_UNSUPPORTED;
  return FP4Q_OK;
}

inline bool packed_ok(const void* p, int64_t ld, int64_t cols) {
  return p && aligned(p, 16) && ld >= cols && ld % 8 == 0;
}

int kv_copy(bool append, int fmt, uint8_t* cache, int64_t n_pages, int32_t page, int32_t kv_heads,
            int32_t dim, const int32_t* offsets, int32_t batch, const int32_t* page_table,
            int64_t ld_table,
            int64_t table_cols, const int32_t* lens, int64_t rows, uint16_t* k, int64_t ldk,
            uint16_t* v, int64_t ldv, const float* k_scale, const float* v_scale, void* stream) {
  const int rc = kv_checks(fmt, cache, n_pages, page, kv_heads, dim, offsets, batch, page_table,
                           ld_table, table_cols, lens, rows, k_scale, v_scale);
  if (rc != FP4Q_OK) return rc;
  if (rows == 0) return FP4Q_OK;
  const int64_t cols = (int64_t)kv_heads * dim;
  if (rows >= ((int64_t)1 << 31) || (rows + 3) / 4 * 4 * (cols / 32) >= ((int64_t)1 << 31))
    return FP4Q_ERR_UNSUPPORTED;  // (before k and v: a caller may not have made them)
  if (!packed_ok(k, ldk, cols) || !packed_ok(v, ldv, cols)) return FP4Q_ERR_INVALID;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  fp4q::launch_kv_copy(append, fmt, cache, n_pages, page_shift_of(page), kv_heads, dim, offsets,
                       batch, page_table, ld_table, table_cols, lens, rows, k, ldk, v, ldv, k_scale, v_scale,
                       static_cast<hipStream_t>(stream));
  return check_launch();
}

int combine_backward_checks(int dtype, const void* y, int64_t rows, int64_t cols, int64_t ldy,
                            const int32_t* row_of, const float* weights, int64_t tokens, int32_t k,
                            const void* d_out, int64_t ldo, const void* d_y, int64_t lddy,
                            const float* d_weights) {
  if (!dtype_ok(dtype) || rows < 0 || cols < 1 || ldy < cols || tokens < 0 || k < 1 ||
      ldo < cols || lddy < cols)
    return FP4Q_ERR_INVALID;
  if (tokens > 0 && (!row_of || !weights || !d_out || !d_weights || (rows > 0 && (!y || !d_y))))
    return FP4Q_ERR_INVALID;
  const int el = dtype == FP4Q_OUT_F32 ? 4 : 2;
  if (!aligned(y, el) || !aligned(d_out, el) || !aligned(d_y, el) || !aligned(row_of, 4) ||
      !aligned(weights, 4) || !aligned(d_weights, 4))
    return FP4Q_ERR_INVALID;
  if (k > 128 || tokens >= ((int64_t)1 << 31) / k || cols >= ((int64_t)1 << 31) ||
      tokens * ((cols + 7) / 8) >= ((int64_t)1 << 31))
    return FP4Q_ERR_UNSUPPORTED;
  return FP4Q_OK;
}

}  // namespace

extern "C" {

size_t fp4q_kv_page_bytes(fp4q_format_t fmt, int32_t page, int32_t dim) {
  if (!fmt_ok(fmt) || page_shift_of(page) < 0 || (dim != 64 && dim != 128 && dim != 256)) return 0;
  return (size_t)page * (size_t)(dim + 2 * (dim / blk_of(fmt)));
}

int fp4q_kv_append(fp4q_format_t fmt, uint8_t* cache, int64_t n_pages, int32_t page,
                   int32_t kv_heads, int32_t dim, const int32_t* offsets, int32_t batch,
                   const int32_t* page_table, int64_t ld_table,
                   int64_t table_cols, const int32_t* lens, int64_t rows,
                   const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                   const float* k_scale, const float* v_scale, void* stream) {
  return kv_copy(true, fmt, cache, n_pages, page, kv_heads, dim, offsets, batch, page_table,
                 ld_table, table_cols, lens, rows, const_cast<uint16_t*>(k), ldk, const_cast<uint16_t*>(v),
                 ldv, k_scale, v_scale, stream);
}

int fp4q_kv_read(fp4q_format_t fmt, const uint8_t* cache, int64_t n_pages, int32_t page,
                 int32_t kv_heads, int32_t dim, const int32_t* offsets, int32_t batch,
                 const int32_t* page_table, int64_t ld_table,
                 int64_t table_cols, const int32_t* lens, int64_t rows,
                 uint16_t* k, int64_t ldk, uint16_t* v, int64_t ldv, const float* k_scale,
                 const float* v_scale, void* stream) {
  return kv_copy(false, fmt, const_cast<uint8_t*>(cache), n_pages, page, kv_heads, dim, offsets,
                 batch, page_table, ld_table, table_cols, lens, rows, k, ldk, v, ldv, k_scale, v_scale, stream);
}

size_t fp4q_kv_attention_workspace_bytes(fp4q_format_t fmt, int64_t rows, int32_t heads,
                                         int32_t kv_heads, int32_t dim, int32_t batch,
                                         int64_t max_new, int64_t max_len, int32_t window) {
  if (!fmt_ok(fmt) || rows <= 0 || heads < 1 || kv_heads < 1 || heads % kv_heads != 0 ||
      batch < 1 || max_new < 1 || max_len < 0 || window < 0 ||
      (dim != 64 && dim != 128 && dim != 256) ||
      !fp4q::attention_shape_ok(rows, dim, batch, kv_heads, heads / kv_heads, max_new, max_len, window))
    return 0;
  return fp4q::attention_workspace_bytes(rows, dim, batch, kv_heads, heads / kv_heads, max_new,
                                         max_len, window);
}

int fp4q_kv_attention(fp4q_format_t fmt, const uint8_t* cache, int64_t n_pages, int32_t page,
                      int32_t kv_heads, int32_t dim, const int32_t* offsets, int32_t batch,
                      const int32_t* page_table, int64_t ld_table,
                      int64_t table_cols, const int32_t* lens, int64_t rows, const uint16_t* q, int64_t ldq, int32_t heads,
                      int64_t max_new, int64_t max_len, int32_t window, float scale,
                      const float* k_scale, const float* v_scale, void* y, fp4q_dtype_t y_dtype,
                      int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = kv_checks(fmt, cache, n_pages, page, kv_heads, dim, offsets, batch, page_table,
                           ld_table, table_cols, lens, rows, k_scale, v_scale);
  if (rc != FP4Q_OK && rc != FP4Q_ERR_UNSUPPORTED) return rc;
  if (!dtype_ok(y_dtype) || heads < 1 || heads % kv_heads != 0 || max_new < 0 || max_len < 0 ||
      window < 0 || !(scale > 0.0f) || !(scale <= 3.4e38f))
    return FP4Q_ERR_INVALID;
  if (rc != FP4Q_OK) return rc;
  if (rows == 0) return FP4Q_OK;
  const int64_t cols = (int64_t)heads * dim;
  if (max_new < 1 || !packed_ok(q, ldq, cols) || !packed_ok(y, ldy, cols)) return FP4Q_ERR_INVALID;
  if (!fp4q::attention_shape_ok(rows, dim, batch, kv_heads, heads / kv_heads, max_new, max_len, window))
    return FP4Q_ERR_UNSUPPORTED;
  // the kernels look up to 2^12 keys past the last in 32 bits
  const int64_t far = ((int64_t)1 << 31) - 4096;
  if (max_len > far && table_cols * page > far) return FP4Q_ERR_UNSUPPORTED;
  const size_t need = fp4q_kv_attention_workspace_bytes(fmt, rows, heads, kv_heads, dim, batch,
                                                        max_new, max_len, window);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
    return FP4Q_ERR_WORKSPACE;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  fp4q::launch_attention(fmt, cache, n_pages, page_shift_of(page), kv_heads, dim, offsets, batch,
                         page_table, ld_table, table_cols, lens, q, ldq, rows, heads / kv_heads, max_new,
                         max_len, window, scale, k_scale, v_scale, y, y_dtype == FP4Q_OUT_BF16,
                         ldy, workspace, static_cast<hipStream_t>(stream));
  return check_launch();
}

size_t fp4q_route_workspace_bytes(int64_t tokens, int32_t experts) {
  if (tokens <= 0 || experts < 1) return 0;
  return fp4q::route_workspace_bytes(tokens, experts);
}

int fp4q_route(const void* logits, fp4q_dtype_t dtype, int64_t tokens, int32_t n_experts,
               int64_t ldx, int32_t k, fp4q_score_t score, const float* bias, int32_t n_groups,
               int32_t top_groups, int32_t renorm, int32_t* experts, float* weights,
               int32_t* offsets, int32_t* row_src, int32_t* row_of, void* workspace,
               size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype) || (score != FP4Q_SCORE_SOFTMAX && score != FP4Q_SCORE_SIGMOID))
    return FP4Q_ERR_INVALID;
  if (tokens < 0 || n_experts < 1 || ldx < n_experts || k < 1 || n_groups < 1 ||
      n_experts % n_groups != 0 || top_groups < 1 || top_groups > n_groups ||
      k > n_experts / n_groups * top_groups)
    return FP4Q_ERR_INVALID;
  if (n_experts > FP4Q_ROUTE_MAX_EXPERTS || n_groups > FP4Q_ROUTE_MAX_GROUPS ||
      k > FP4Q_ROUTE_MAX_K || tokens >= ((int64_t)1 << 27) / k)
    return FP4Q_ERR_UNSUPPORTED;  // (before the results: a caller may not have made them)
  if (!offsets || !aligned(offsets, 4) || !aligned(bias, 4)) return FP4Q_ERR_INVALID;
  if (tokens > 0 && (!logits || !experts || !weights || !row_src || !row_of))
    return FP4Q_ERR_INVALID;
  if (!aligned(logits, dtype == FP4Q_OUT_F32 ? 4 : 2) || !aligned(experts, 4) ||
      !aligned(weights, 4) || !aligned(row_src, 4) || !aligned(row_of, 4))
    return FP4Q_ERR_INVALID;
  const size_t need = fp4q_route_workspace_bytes(tokens, n_experts);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 8)))
    return FP4Q_ERR_WORKSPACE;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  fp4q::launch_route(logits, dtype == FP4Q_OUT_F32, tokens, ldx, n_experts, k, score, bias,
                     n_groups, top_groups, renorm != 0, experts, weights, offsets, row_src, row_of,
                     workspace, static_cast<hipStream_t>(stream));
  return check_launch();
}

int fp4q_route_backward(const void* logits, fp4q_dtype_t dtype, int64_t tokens,
                        int32_t n_experts, int64_t ldx, int32_t k, fp4q_score_t score,
                        int32_t renorm, const int32_t* experts, const float* d_weights,
                        void* d_logits, int64_t ldd, void* stream) {
  if (!dtype_ok(dtype) || (score != FP4Q_SCORE_SOFTMAX && score != FP4Q_SCORE_SIGMOID))
    return FP4Q_ERR_INVALID;
  if (tokens < 0 || n_experts < 1 || ldx < n_experts || ldd < n_experts || k < 1 || k > n_experts)
    return FP4Q_ERR_INVALID;
  if (tokens > 0 && (!logits || !experts || !d_weights || !d_logits)) return FP4Q_ERR_INVALID;
  const int el = dtype == FP4Q_OUT_F32 ? 4 : 2;
  if (!aligned(logits, el) || !aligned(d_logits, el) || !aligned(experts, 4) ||
      !aligned(d_weights, 4))
    return FP4Q_ERR_INVALID;
  if (n_experts > FP4Q_ROUTE_MAX_EXPERTS || k > FP4Q_ROUTE_MAX_K ||
      tokens >= ((int64_t)1 << 27) / k)
    return FP4Q_ERR_UNSUPPORTED;
  if (tokens == 0) return FP4Q_OK;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  fp4q::launch_route_backward(logits, dtype == FP4Q_OUT_F32, tokens, ldx, n_experts, k, score,
                              renorm != 0, experts, d_weights, d_logits, ldd,
                              static_cast<hipStream_t>(stream));
  return check_launch();
}

int fp4q_combine(fp4q_dtype_t dtype, const void* y, int64_t rows, int64_t cols, int64_t ldy,
                 const int32_t* row_of, const float* weights, int64_t tokens, int32_t k,
                 void* out, int64_t ldo, void* stream) {
  if (!dtype_ok(dtype) || rows < 0 || cols < 1 || ldy < cols || tokens < 0 || k < 1 || ldo < cols)
    return FP4Q_ERR_INVALID;
  if (tokens > 0 && (!row_of || !weights || !out || (rows > 0 && !y))) return FP4Q_ERR_INVALID;
  const int el = dtype == FP4Q_OUT_F32 ? 4 : 2;
  if (!aligned(y, el) || !aligned(out, el) || !aligned(row_of, 4) || !aligned(weights, 4))
    return FP4Q_ERR_INVALID;
  if (k > 128 || tokens >= ((int64_t)1 << 31) / k || cols >= ((int64_t)1 << 31) ||
      tokens * ((cols + 7) / 8) >= ((int64_t)1 << 31))
    return FP4Q_ERR_UNSUPPORTED;
  if (tokens == 0) return FP4Q_OK;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  fp4q::launch_combine(dtype == FP4Q_OUT_F32, y, rows, cols, ldy, row_of, weights, tokens, k, out,
                       ldo, static_cast<hipStream_t>(stream));
  return check_launch();
}

int fp4q_combine_backward(fp4q_dtype_t dtype, const void* y, int64_t rows, int64_t cols,
                          int64_t ldy, const int32_t* row_of, const float* weights,
                          int64_t tokens, int32_t k, const void* d_out, int64_t ldo, void* d_y,
                          int64_t lddy, float* d_weights, void* stream) {
  const int rc = combine_backward_checks(dtype, y, rows, cols, ldy, row_of, weights, tokens, k, d_out,
                                         ldo, d_y, lddy, d_weights);
  if (rc != FP4Q_OK) return rc;
  if (tokens == 0) return FP4Q_OK;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  fp4q::launch_combine_backward(dtype == FP4Q_OUT_F32, y, rows, cols, ldy, row_of, weights, tokens,
                                k, d_out, ldo, d_y, lddy, d_weights, nullptr,
                                static_cast<hipStream_t>(stream));
  return check_launch();
}

size_t fp4q_combine_backward_zeroed_workspace_bytes(int64_t rows) {
  return rows > 0 && rows < ((int64_t)1 << 31) ? (size_t)rows * sizeof(int32_t) : 0;
}

int fp4q_combine_backward_zeroed(fp4q_dtype_t dtype, const void* y, int64_t rows, int64_t cols,
                                 int64_t ldy, const int32_t* row_of, const float* weights,
                                 int64_t tokens, int32_t k, const void* d_out, int64_t ldo, void* d_y,
                                 int64_t lddy, float* d_weights, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  const int rc = combine_backward_checks(dtype, y, rows, cols, ldy, row_of, weights, tokens, k, d_out,
                                         ldo, d_y, lddy, d_weights);
  if (rc != FP4Q_OK) return rc;
  if (rows > 0 && !d_y) return FP4Q_ERR_INVALID;
  if (rows >= ((int64_t)1 << 31)) return FP4Q_ERR_UNSUPPORTED;
  const size_t need = fp4q_combine_backward_zeroed_workspace_bytes(rows);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 4)))
    return FP4Q_ERR_WORKSPACE;
  if (tokens == 0 && rows == 0) return FP4Q_OK;
  if (injected_failure()) return FP4Q_ERR_HIP;
  clear_error();
  fp4q::launch_combine_backward(dtype == FP4Q_OUT_F32, y, rows, cols, ldy, row_of, weights, tokens,
                                k, d_out, ldo, d_y, lddy, d_weights, static_cast<int32_t*>(workspace),
                                static_cast<hipStream_t>(stream));
  return check_launch();
}

}  // extern "C"
