// C ABI of librd.so (declared in include/rd.h): host-side validation and
// dispatch.  Everything that depends on device-resident values (group sizes,
// offset, limit) is decided inside the kernels; this file only checks what
// the host can see and sizes the persistent grids.
#include "rd.h"

#include <hip/hip_runtime_api.h>

#include "rd_launch.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_groups(int32_t num_groups, const int32_t* group_offset, int32_t num_local) {
  if (num_groups < 1 || num_local < 1) return RD_EINVAL;
  if (num_groups > RD_MAX_GROUPS || num_local > RD_MAX_GROUPS) return RD_EUNSUPPORTED;
  if (num_local > num_groups) return RD_EINVAL;
  if (group_offset == nullptr && num_local != num_groups) return RD_EINVAL;
  if (group_offset != nullptr && (reinterpret_cast<uintptr_t>(group_offset) & 3u)) return RD_EINVAL;
  return RD_OK;
}

int check_dims(int64_t m, int64_t k, int64_t n) {
  if (m < 0 || k <= 0 || n <= 0) return RD_EINVAL;
  if (m >= (int64_t(1) << 31) || k >= (int64_t(1) << 31) || n >= (int64_t(1) << 31)) return RD_EUNSUPPORTED;
  if ((k % 8) != 0 || (n % 8) != 0) return RD_EUNSUPPORTED;
  return RD_OK;
}

int forward_common(const void* x, const void* w, const int32_t* group_sizes, int32_t num_groups,
                   const int32_t* group_offset, int32_t num_local, const int32_t* limit, void* out,
                   int32_t out_dtype, int64_t m, int64_t k, int64_t n, void* workspace, size_t workspace_bytes,
                   void* stream, bool trans_rhs, bool noalloc = false) {
  int st = check_dims(m, k, n);
  if (st != RD_OK) return st;
  st = check_groups(num_groups, group_offset, num_local);
  if (st != RD_OK) return st;
  if (out_dtype != RD_BF16 && out_dtype != RD_F32) return RD_EINVAL;
  if (!w || !group_sizes) return RD_EINVAL;
  if (m == 0) return RD_OK;  // no rows: x and out may be empty (null)
  if (!x || !out) return RD_EINVAL;
  if (!aligned16(x) || !aligned16(w) || !aligned16(out) || !aligned16(workspace)) return RD_EINVAL;
  if ((reinterpret_cast<uintptr_t>(group_sizes) & 3u) || (reinterpret_cast<uintptr_t>(limit) & 3u))
    return RD_EINVAL;
  rd::GemmProblem p{};
  p.a = x;
  p.b = w;
  p.group_sizes = group_sizes;
  p.num_groups = num_groups;
  p.group_offset = group_offset;
  p.num_local = num_local;
  p.limit = limit;
  p.out = out;
  p.out_f32 = out_dtype == RD_F32;
  p.m = static_cast<int>(m);
  p.k = static_cast<int>(k);
  p.n = static_cast<int>(n);
  if (noalloc) return rd::launch_forward_noalloc(p, static_cast<hipStream_t>(stream));
  return rd::launch_forward(p, trans_rhs, workspace, workspace_bytes, static_cast<hipStream_t>(stream));
}

// The GemmProblem of a forward call of these sizes (pointers unset).
rd::GemmProblem shape_only(int64_t m, int64_t k, int64_t n, int32_t num_local) {
  rd::GemmProblem p{};
  p.num_groups = num_local;
  p.num_local = num_local;
  p.m = static_cast<int>(m);
  p.k = static_cast<int>(k);
  p.n = static_cast<int>(n);
  return p;
}

}  // namespace

extern "C" {

int rd_abi_version(void) { return RD_ABI_VERSION; }

const char* rd_status_string(int status) {
  switch (status) {
    case RD_OK: return "ok";
    case RD_EINVAL: return "invalid argument (null or misaligned pointer, bad size or dtype)";
    case RD_EUNSUPPORTED: return "unsupported size (k, n, h, hidden must be multiples of 8, MX blocks whole; dims < 2^31; groups <= RD_MAX_GROUPS)";
    case RD_EHIP: return "HIP runtime error while launching";
    case RD_ESCRATCH: return "the call needs more device scratch than rd_forward_noalloc holds (RD_NOALLOC_SCRATCH_BYTES)";
    default: return "unknown status";
  }
}

size_t rd_forward_workspace_size(int64_t m, int64_t k, int64_t n, int32_t num_local, int32_t trans_rhs) {
  if (check_dims(m, k, n) != RD_OK || num_local < 1 || num_local > RD_MAX_GROUPS) return 0;
  const rd::DecodePlan d = rd::plan_decode(shape_only(m, k, n, num_local), trans_rhs != 0);
  return d.use ? d.ws_bytes : 0;
}

int rd_forward(const void* x, const void* w, const int32_t* group_sizes, int32_t num_groups,
               const int32_t* group_offset, int32_t num_local, const int32_t* limit, void* out,
               int32_t out_dtype, int64_t m, int64_t k, int64_t n, void* workspace, size_t workspace_bytes,
               void* stream) {
  return forward_common(x, w, group_sizes, num_groups, group_offset, num_local, limit, out, out_dtype, m,
                        k, n, workspace, workspace_bytes, stream, false);
}

int rd_forward_noalloc(const void* x, const void* w, const int32_t* group_sizes, int32_t num_groups,
                       const int32_t* group_offset, int32_t num_local, const int32_t* limit, void* out,
                       int32_t out_dtype, int64_t m, int64_t k, int64_t n, void* stream) {
  return forward_common(x, w, group_sizes, num_groups, group_offset, num_local, limit, out, out_dtype, m, k, n,
                        nullptr, 0, stream, false, true);
}

int rd_forward_trans_rhs(const void* x, const void* w, const int32_t* group_sizes,
                         int32_t num_groups, const int32_t* group_offset, int32_t num_local,
                         const int32_t* limit, void* out, int32_t out_dtype, int64_t m, int64_t k,
                         int64_t n, void* workspace, size_t workspace_bytes, void* stream) {
  return forward_common(x, w, group_sizes, num_groups, group_offset, num_local, limit, out, out_dtype, m,
                        k, n, workspace, workspace_bytes, stream, true);
}

int rd_forward_glu(const void* x, const void* wi, const int32_t* group_sizes, int32_t num_groups,
                   const int32_t* group_offset, int32_t num_local, const int32_t* limit, void* act,
                   void* fused, int64_t m, int64_t k, int64_t h, void* stream) {
  if (h <= 0) return RD_EINVAL;
  if (h >= (int64_t(1) << 30)) return RD_EUNSUPPORTED;  // the weight's width 2h stays below 2^31
  int st = check_dims(m, k, 2 * h);
  if (st != RD_OK) return st;
  st = check_groups(num_groups, group_offset, num_local);
  if (st != RD_OK) return st;
  if (!wi || !group_sizes) return RD_EINVAL;
  if (m == 0) return RD_OK;  // no rows: x, act and fused may be empty (null)
  if (!x || !act) return RD_EINVAL;
  if (!aligned16(x) || !aligned16(wi) || !aligned16(act) || (fused && !aligned16(fused))) return RD_EINVAL;
  if ((reinterpret_cast<uintptr_t>(group_sizes) & 3u) || (reinterpret_cast<uintptr_t>(limit) & 3u) ||
      (reinterpret_cast<uintptr_t>(group_offset) & 3u))
    return RD_EINVAL;
  rd::GemmProblem p{};
  p.a = x;
  p.b = wi;
  p.group_sizes = group_sizes;
  p.num_groups = num_groups;
  p.group_offset = group_offset;
  p.num_local = num_local;
  p.limit = limit;
  p.out = act;
  p.out2 = fused;
  p.out_f32 = false;
  p.m = static_cast<int>(m);
  p.k = static_cast<int>(k);
  p.n = static_cast<int>(h);
  if (!rd::fused_glu_supported(p)) return RD_EUNSUPPORTED;
  return rd::launch_forward_glu(p, static_cast<hipStream_t>(stream));
}

namespace {
int forward_fp8(const void* x, const void* w, const int32_t* group_sizes, int32_t num_groups,
                const int32_t* group_offset, int32_t num_local, const int32_t* limit, void* out, int32_t out_dtype,
                int64_t m, int64_t k, int64_t n, void* stream, bool trans_rhs) {
  int st = check_dims(m, k, n);
  if (st != RD_OK) return st;
  if ((k % 128) != 0 || (!trans_rhs && (n % 16) != 0)) return RD_EUNSUPPORTED;
  if (k * (m > n ? m : n) >= (int64_t(1) << 32)) return RD_EUNSUPPORTED;
  st = check_groups(num_groups, group_offset, num_local);
  if (st != RD_OK) return st;
  if (out_dtype != RD_BF16 && out_dtype != RD_F32) return RD_EINVAL;
  if (!w || !group_sizes) return RD_EINVAL;
  if (m == 0) return RD_OK;  // no rows: x and out may be empty (null)
  if (!x || !out) return RD_EINVAL;
  if (!aligned16(x) || !aligned16(w) || !aligned16(out)) return RD_EINVAL;
  if ((reinterpret_cast<uintptr_t>(group_sizes) & 3u) || (reinterpret_cast<uintptr_t>(limit) & 3u) ||
      (reinterpret_cast<uintptr_t>(group_offset) & 3u))
    return RD_EINVAL;
  rd::GemmProblem p{};
  p.a = x;
  p.b = w;
  p.group_sizes = group_sizes;
  p.num_groups = num_groups;
  p.group_offset = group_offset;
  p.num_local = num_local;
  p.limit = limit;
  p.out = out;
  p.out_f32 = out_dtype == RD_F32;
  p.m = static_cast<int>(m);
  p.k = static_cast<int>(k);
  p.n = static_cast<int>(n);
  return rd::launch_forward_fp8(p, trans_rhs, static_cast<hipStream_t>(stream));
}
}  // namespace

int rd_forward_fp8(const void* x, const void* w, const int32_t* group_sizes, int32_t num_groups,
                   const int32_t* group_offset, int32_t num_local, const int32_t* limit, void* out,
                   int32_t out_dtype, int64_t m, int64_t k, int64_t n, void* stream) {
  return forward_fp8(x, w, group_sizes, num_groups, group_offset, num_local, limit, out, out_dtype, m, k, n, stream,
                     false);
}

int rd_forward_trans_rhs_fp8(const void* x, const void* w, const int32_t* group_sizes, int32_t num_groups,
                             const int32_t* group_offset, int32_t num_local, const int32_t* limit, void* out,
                             int32_t out_dtype, int64_t m, int64_t k, int64_t n, void* stream) {
  return forward_fp8(x, w, group_sizes, num_groups, group_offset, num_local, limit, out, out_dtype, m, k, n, stream,
                     true);
}

size_t rd_trans_workspace_size(int64_t m, int64_t k, int64_t n, int32_t num_local) {
  if (check_dims(m, k, n) != RD_OK || num_local <= 0 || num_local > RD_MAX_GROUPS || m == 0) return 0;
  rd::GemmProblem p{};
  p.num_local = num_local;
  p.m = static_cast<int>(m);
  p.k = static_cast<int>(k);
  p.n = static_cast<int>(n);
  return rd::trans_workspace_size(p);
}

int rd_trans_fp8(const void* x, const void* dy, const int32_t* group_sizes, int32_t num_groups,
                 const int32_t* group_offset, int32_t num_local, const int32_t* limit, void* dw,
                 int32_t dw_dtype, int64_t m, int64_t k, int64_t n, void* workspace, size_t workspace_bytes,
                 void* stream) {
  int st = check_dims(m, k, n);
  if (st != RD_OK) return st;
  if ((k % 16) != 0 || (n % 16) != 0) return RD_EUNSUPPORTED;
  if (m * (k > n ? k : n) >= (int64_t(1) << 32)) return RD_EUNSUPPORTED;
  st = check_groups(num_groups, group_offset, num_local);
  if (st != RD_OK) return st;
  if (dw_dtype != RD_BF16 && dw_dtype != RD_F32) return RD_EINVAL;
  if (!group_sizes || !dw) return RD_EINVAL;
  if (m > 0 && (!x || !dy)) return RD_EINVAL;  // no rows: x and dy may be empty (null)
  if ((m > 0 && (!aligned16(x) || !aligned16(dy))) || !aligned16(dw)) return RD_EINVAL;
  if ((reinterpret_cast<uintptr_t>(group_sizes) & 3u) || (reinterpret_cast<uintptr_t>(limit) & 3u) ||
      (reinterpret_cast<uintptr_t>(group_offset) & 3u))
    return RD_EINVAL;
  if (workspace_bytes > 0 && (workspace == nullptr || !aligned16(workspace))) return RD_EINVAL;
  rd::GemmProblem p{};
  p.a = x;
  p.b = dy;
  p.group_sizes = group_sizes;
  p.num_groups = num_groups;
  p.group_offset = group_offset;
  p.num_local = num_local;
  p.limit = limit;
  p.out = dw;
  p.out_f32 = dw_dtype == RD_F32;
  p.m = static_cast<int>(m);
  p.k = static_cast<int>(k);
  p.n = static_cast<int>(n);
  return rd::launch_trans_fp8(p, workspace_bytes > 0 ? workspace : nullptr, workspace_bytes,
                              static_cast<hipStream_t>(stream));
}

int rd_trans(const void* x, const void* dy, const int32_t* group_sizes, int32_t num_groups,
             const int32_t* group_offset, int32_t num_local, const int32_t* limit, void* dw,
             int32_t dw_dtype, int64_t m, int64_t k, int64_t n, void* workspace,
             size_t workspace_bytes, void* stream) {
  int st = check_dims(m, k, n);
  if (st != RD_OK) return st;
  st = check_groups(num_groups, group_offset, num_local);
  if (st != RD_OK) return st;
  if (dw_dtype != RD_BF16 && dw_dtype != RD_F32) return RD_EINVAL;
  if (!group_sizes || !dw) return RD_EINVAL;
  if (m > 0 && (!x || !dy)) return RD_EINVAL;  // no rows: x and dy may be empty (null)
  if ((m > 0 && (!aligned16(x) || !aligned16(dy))) || !aligned16(dw)) return RD_EINVAL;
  if ((reinterpret_cast<uintptr_t>(group_sizes) & 3u) || (reinterpret_cast<uintptr_t>(limit) & 3u))
    return RD_EINVAL;
  if (workspace_bytes > 0 && (workspace == nullptr || !aligned16(workspace))) return RD_EINVAL;
  rd::GemmProblem p{};
  p.a = x;
  p.b = dy;
  p.group_sizes = group_sizes;
  p.num_groups = num_groups;
  p.group_offset = group_offset;
  p.num_local = num_local;
  p.limit = limit;
  p.out = dw;
  p.out_f32 = dw_dtype == RD_F32;
  p.m = static_cast<int>(m);
  p.k = static_cast<int>(k);
  p.n = static_cast<int>(n);
  return rd::launch_trans(p, workspace_bytes > 0 ? workspace : nullptr, workspace_bytes,
                          static_cast<hipStream_t>(stream));
}

int rd_glu_fwd(const void* fused, const int32_t* limit, void* out, int64_t rows, int64_t h,
               void* stream) {
  if (rows < 0 || h <= 0) return RD_EINVAL;
  if ((h % 8) != 0) return RD_EUNSUPPORTED;
  if (rows >= (int64_t(1) << 31) || h >= (int64_t(1) << 30)) return RD_EUNSUPPORTED;
  if (rows == 0) return RD_OK;  // no rows: the buffers may be empty (null)
  if (!fused || !out) return RD_EINVAL;
  if (!aligned16(fused) || !aligned16(out) || (reinterpret_cast<uintptr_t>(limit) & 3u)) return RD_EINVAL;
  return rd::launch_glu_fwd(fused, limit, out, static_cast<int>(rows), static_cast<int>(h),
                            static_cast<hipStream_t>(stream));
}

int rd_glu_bwd(const void* fused, const void* d_out, const int32_t* limit, void* d_fused,
               int64_t rows, int64_t h, void* stream) {
  if (rows < 0 || h <= 0) return RD_EINVAL;
  if ((h % 8) != 0) return RD_EUNSUPPORTED;
  if (rows >= (int64_t(1) << 31) || h >= (int64_t(1) << 30)) return RD_EUNSUPPORTED;
  if (rows == 0) return RD_OK;  // no rows: the buffers may be empty (null)
  if (!fused || !d_out || !d_fused) return RD_EINVAL;
  if (!aligned16(fused) || !aligned16(d_out) || !aligned16(d_fused) ||
      (reinterpret_cast<uintptr_t>(limit) & 3u))
    return RD_EINVAL;
  return rd::launch_glu_bwd(fused, d_out, limit, d_fused, static_cast<int>(rows), static_cast<int>(h),
                            static_cast<hipStream_t>(stream));
}

int rd_unsort_bwd_rows(const void* g, const void* y, const float* w, const int32_t* limit, void* grad, float* dot,
                       int64_t rows, int64_t hidden, void* stream) {
  if (rows < 0 || hidden <= 0) return RD_EINVAL;
  if ((hidden % 8) != 0) return RD_EUNSUPPORTED;
  if (rows >= (int64_t(1) << 31) || hidden >= (int64_t(1) << 30)) return RD_EUNSUPPORTED;
  if (rows == 0) return RD_OK;  // no rows: the buffers may be empty (null)
  if (!g || !y || !w || !grad || !dot) return RD_EINVAL;
  if (!aligned16(g) || !aligned16(y) || !aligned16(grad) || (reinterpret_cast<uintptr_t>(w) & 3u) ||
      (reinterpret_cast<uintptr_t>(dot) & 3u) || (reinterpret_cast<uintptr_t>(limit) & 3u))
    return RD_EINVAL;
  return rd::launch_unsort_bwd_rows(g, y, w, limit, grad, dot, static_cast<int>(rows), static_cast<int>(hidden),
                                    static_cast<hipStream_t>(stream));
}

int rd_zero_rows_from_limit(void* buf, const int32_t* limit, int64_t rows, int64_t row_bytes, void* stream) {
  if (rows < 0 || row_bytes <= 0) return RD_EINVAL;
  if ((row_bytes % 16) != 0) return RD_EUNSUPPORTED;
  if (rows > 0 && row_bytes > (int64_t(1) << 62) / rows) return RD_EUNSUPPORTED;
  if (rows == 0 || limit == nullptr) return RD_OK;  // no rows past the limit: nothing to write
  if (!buf) return RD_EINVAL;
  if (!aligned16(buf) || (reinterpret_cast<uintptr_t>(limit) & 3u)) return RD_EINVAL;
  return rd::launch_zero_rows(buf, limit, rows, row_bytes, static_cast<hipStream_t>(stream));
}

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned_to(const void* p, int32_t dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (dtype == RD_F32 ? 3u : 1u)) == 0;
}

int check_route(int32_t dtype, int64_t tokens, int32_t experts, int32_t top_k, int32_t score) {
  if (dtype != RD_BF16 && dtype != RD_F32) return RD_EINVAL;
  if (score != RD_SOFTMAX && score != RD_SIGMOID) return RD_EINVAL;
  if (tokens < 0 || experts < 1 || top_k < 1 || top_k > experts) return RD_EINVAL;
  if (experts > RD_MAX_GROUPS || top_k > RD_MAX_TOP_K || tokens >= (int64_t(1) << 31) - 64) return RD_EUNSUPPORTED;
  return RD_OK;
}

int check_rows(int64_t tokens, int32_t top_k, int64_t hidden, int64_t rows) {
  if (tokens < 0 || top_k < 1 || hidden <= 0 || rows < 0) return RD_EINVAL;
  if (top_k > RD_MAX_TOP_K || hidden % 8 != 0 || hidden >= (int64_t(1) << 30) || rows >= (int64_t(1) << 31))
    return RD_EUNSUPPORTED;
  if (tokens >= (int64_t(1) << 31) / ((hidden + 511) / 512)) return RD_EUNSUPPORTED;  // below 2^31 from here on
  if (tokens * top_k >= (int64_t(1) << 31)) return RD_EUNSUPPORTED;
  return RD_OK;
}

constexpr int64_t kMaxGluRows = (int64_t(1) << 31) - (1 << 20);  // a row number and the grid's stride fit 32 bits

int check_mx(int64_t rows, int64_t cols, int32_t bits) {
  if (rows < 0 || cols <= 0 || (bits != 4 && bits != 8)) return RD_EINVAL;
  if (cols % 32 != 0 || (rows > 0 && cols > (int64_t(1) << 62) / rows)) return RD_EUNSUPPORTED;
  return RD_OK;
}

}  // namespace

int rd_route(const void* logits, int32_t dtype, const float* bias, const int32_t* limit, float* weights, int32_t* ids,
             int64_t tokens, int32_t experts, int32_t top_k, int32_t score, int32_t groups, int32_t top_groups,
             int32_t renormalize, float scale, void* stream) {
  const int st = check_route(dtype, tokens, experts, top_k, score);
  if (st != RD_OK) return st;
  if (groups < 1 || top_groups < 1 || top_groups > groups || experts % groups != 0) return RD_EINVAL;
  if (groups > RD_MAX_ROUTE_GROUPS) return RD_EUNSUPPORTED;
  if (top_k > top_groups * (experts / groups)) return RD_EINVAL;
  if (tokens == 0) return RD_OK;  // no rows: the buffers may be empty (null)
  if (!logits || !weights || !ids) return RD_EINVAL;
  if (!aligned_to(logits, dtype) || !aligned4(bias) || !aligned4(limit) || !aligned4(weights) || !aligned4(ids))
    return RD_EINVAL;
  rd::RouteProblem p{logits, dtype == RD_BF16, bias, limit, weights, ids, static_cast<int>(tokens), experts, top_k,
                     groups, top_groups, score == RD_SIGMOID, renormalize != 0, scale};
  return rd::launch_route(p, static_cast<hipStream_t>(stream));
}

int rd_route_bwd(const void* logits, int32_t dtype, const int32_t* ids, const float* d_weights, void* d_logits,
                 int64_t tokens, int32_t experts, int32_t top_k, int32_t score, int32_t renormalize, float scale,
                 void* stream) {
  const int st = check_route(dtype, tokens, experts, top_k, score);
  if (st != RD_OK) return st;
  if (tokens == 0) return RD_OK;  // no rows: the buffers may be empty (null)
  if (!logits || !ids || !d_weights || !d_logits) return RD_EINVAL;
  if (!aligned_to(logits, dtype) || !aligned_to(d_logits, dtype) || !aligned4(ids) || !aligned4(d_weights))
    return RD_EINVAL;
  rd::RouteProblem p{logits, dtype == RD_BF16, nullptr, nullptr, nullptr, const_cast<int32_t*>(ids),
                     static_cast<int>(tokens), experts, top_k, 1, 1, score == RD_SIGMOID, renormalize != 0, scale};
  return rd::launch_route_bwd(p, d_weights, d_logits, static_cast<hipStream_t>(stream));
}

size_t rd_group_rows_workspace_size(int64_t n, int32_t experts) {
  if (n < 0 || n > (int64_t(1) << 30) || experts < 1 || experts > RD_MAX_GROUPS) return 0;
  return rd::group_rows_workspace_size(n, experts);
}

int rd_group_rows(const int32_t* ids, int64_t n, int32_t experts, int32_t* sizes, int32_t* rows, int32_t* slots,
                  int32_t* total, void* workspace, size_t workspace_bytes, void* stream) {
  if (n < 0 || experts < 1) return RD_EINVAL;
  if (n > (int64_t(1) << 30) || experts > RD_MAX_GROUPS) return RD_EUNSUPPORTED;
  if (!sizes || !total || (n > 0 && (!ids || !rows || !slots))) return RD_EINVAL;
  if (!aligned4(ids) || !aligned4(sizes) || !aligned4(rows) || !aligned4(slots) || !aligned4(total)) return RD_EINVAL;
  const size_t need = rd::group_rows_workspace_size(n, experts);
  if (need > 0 && (!workspace || !aligned4(workspace) || workspace_bytes < need)) return RD_EINVAL;
  return rd::launch_group_rows(ids, static_cast<int>(n), experts, sizes, rows, slots, total,
                               static_cast<int32_t*>(workspace), static_cast<hipStream_t>(stream));
}

int rd_dispatch_rows(const void* x, const int32_t* slots, void* xs, int64_t tokens, int32_t top_k, int64_t hidden,
                     int64_t rows, void* stream) {
  const int st = check_rows(tokens, top_k, hidden, rows);
  if (st != RD_OK) return st;
  if (tokens == 0 || rows == 0) return RD_OK;  // nothing to write: the buffers may be empty (null)
  if (!x || !slots || !xs || !aligned16(x) || !aligned4(slots) || !aligned16(xs)) return RD_EINVAL;
  rd::RowsProblem p{x, nullptr, slots, nullptr, xs, nullptr, static_cast<int>(tokens), top_k,
                    static_cast<int>(hidden), rows};
  return rd::launch_dispatch_rows(p, static_cast<hipStream_t>(stream));
}

int rd_combine_rows(const void* y, const int32_t* slots, const float* weights, void* out, int64_t tokens,
                    int32_t top_k, int64_t hidden, int64_t rows, void* stream) {
  const int st = check_rows(tokens, top_k, hidden, rows);
  if (st != RD_OK) return st;
  if (tokens == 0) return RD_OK;  // no rows: the buffers may be empty (null)
  if (!slots || !out || (rows > 0 && !y)) return RD_EINVAL;
  if (!aligned16(y) || !aligned4(slots) || !aligned4(weights) || !aligned16(out)) return RD_EINVAL;
  rd::RowsProblem p{y, nullptr, slots, weights, out, nullptr, static_cast<int>(tokens), top_k,
                    static_cast<int>(hidden), rows};
  return rd::launch_combine_rows(p, static_cast<hipStream_t>(stream));
}

int rd_combine_rows_bwd(const void* g, const void* y, const int32_t* slots, const float* weights, void* dy, float* dw,
                        int64_t tokens, int32_t top_k, int64_t hidden, int64_t rows, void* stream) {
  const int st = check_rows(tokens, top_k, hidden, rows);
  if (st != RD_OK) return st;
  if (tokens == 0) return RD_OK;  // no rows: the buffers may be empty (null)
  if (!g || !slots || !weights || !dw || (rows > 0 && (!y || !dy))) return RD_EINVAL;
  if (!aligned16(g) || !aligned16(y) || !aligned4(slots) || !aligned4(weights) || !aligned16(dy) || !aligned4(dw))
    return RD_EINVAL;
  rd::RowsProblem p{g, y, slots, weights, dy, dw, static_cast<int>(tokens), top_k, static_cast<int>(hidden), rows};
  return rd::launch_combine_rows_bwd(p, static_cast<hipStream_t>(stream));
}

int rd_quantize_mx(const void* x, int32_t dtype, const int32_t* limit, void* codes, void* scales, int64_t rows,
                   int64_t cols, int32_t bits, void* stream) {
  const int st = check_mx(rows, cols, bits);
  if (st != RD_OK) return st;
  if (dtype != RD_BF16 && dtype != RD_F32) return RD_EINVAL;
  if (rows == 0) return RD_OK;  // no rows: the buffers may be empty (null)
  if (!x || !codes || !scales || !aligned16(x) || !aligned16(codes) || !aligned4(limit)) return RD_EINVAL;
  return rd::launch_quantize_mx(x, dtype == RD_F32, limit, codes, static_cast<uint8_t*>(scales), rows, cols, bits,
                                static_cast<hipStream_t>(stream));
}

int rd_dequantize_mx(const void* codes, const void* scales, const int32_t* limit, void* out, int32_t dtype,
                     int64_t rows, int64_t cols, int32_t bits, void* stream) {
  const int st = check_mx(rows, cols, bits);
  if (st != RD_OK) return st;
  if (dtype != RD_BF16 && dtype != RD_F32) return RD_EINVAL;
  if (rows == 0) return RD_OK;  // no rows: the buffers may be empty (null)
  if (!codes || !scales || !out || !aligned16(codes) || !aligned16(out) || !aligned4(limit)) return RD_EINVAL;
  return rd::launch_dequantize_mx(codes, static_cast<const uint8_t*>(scales), limit, out, dtype == RD_F32, rows, cols,
                                  bits, static_cast<hipStream_t>(stream));
}

int rd_forward_mx(const void* x_codes, const void* x_scales, int32_t x_bits, const void* w_codes, const void* w_scales,
                  const int32_t* group_sizes, int32_t num_groups, const int32_t* group_offset, int32_t num_local,
                  const int32_t* limit, void* out, int32_t out_dtype, int64_t m, int64_t k, int64_t n, void* stream) {
  int st = check_dims(m, k, n);
  if (st != RD_OK) return st;
  if (x_bits != 4 && x_bits != 8) return RD_EINVAL;
  if (k % 128 != 0 || k >= (int64_t(1) << 24) || n * k >= (int64_t(1) << 32)) return RD_EUNSUPPORTED;
  st = check_groups(num_groups, group_offset, num_local);
  if (st != RD_OK) return st;
  if (out_dtype != RD_BF16 && out_dtype != RD_F32) return RD_EINVAL;
  if (!w_codes || !w_scales || !group_sizes) return RD_EINVAL;
  if (m == 0) return RD_OK;  // no rows: x and out may be empty (null)
  if (!x_codes || !x_scales || !out) return RD_EINVAL;
  if (!aligned16(x_codes) || !aligned16(w_codes) || !aligned16(out) || !aligned4(x_scales) || !aligned4(w_scales) ||
      !aligned4(group_sizes) || !aligned4(limit))
    return RD_EINVAL;
  rd::GemmProblem p{};
  p.a = x_codes;
  p.b = w_codes;
  p.group_sizes = group_sizes;
  p.num_groups = num_groups;
  p.group_offset = group_offset;
  p.num_local = num_local;
  p.limit = limit;
  p.out = out;
  p.out_f32 = out_dtype == RD_F32;
  p.m = static_cast<int>(m);
  p.k = static_cast<int>(k);
  p.n = static_cast<int>(n);
  return rd::launch_forward_mx(p, static_cast<const uint8_t*>(x_scales), static_cast<const uint8_t*>(w_scales), x_bits,
                               static_cast<hipStream_t>(stream));
}

int rd_glu_fwd_mx8(const void* fused, const int32_t* limit, void* act, void* codes, void* scales, int64_t rows,
                   int64_t h, void* stream) {
  if (rows < 0 || h <= 0) return RD_EINVAL;
  if (h % 32 != 0 || rows > kMaxGluRows || h >= (int64_t(1) << 30)) return RD_EUNSUPPORTED;
  if (rows == 0) return RD_OK;  // no rows: the buffers may be empty (null)
  if (!fused || !act || !codes || !scales) return RD_EINVAL;
  if (!aligned16(fused) || !aligned16(act) || !aligned16(codes) || !aligned4(limit)) return RD_EINVAL;
  return rd::launch_glu_fwd_mx8(fused, limit, act, codes, static_cast<uint8_t*>(scales), static_cast<int>(rows),
                                static_cast<int>(h), static_cast<hipStream_t>(stream));
}

int rd_glu_bwd_mx8(const void* codes, const void* scales, const void* d_act, const int32_t* limit, const float* weights,
                   const int32_t* row_slots, void* d_fused, void* act, float* dot, int64_t rows, int64_t h,
                   int64_t slots, void* stream) {
  if (rows < 0 || h <= 0 || slots < 0 || (row_slots == nullptr && slots < rows)) return RD_EINVAL;
  if (h % 32 != 0 || rows > kMaxGluRows || h >= (int64_t(1) << 30)) return RD_EUNSUPPORTED;
  if (rows == 0) return RD_OK;  // no rows: the buffers may be empty (null)
  if (!codes || !scales || !d_act || !d_fused || !act || (slots > 0 && !dot)) return RD_EINVAL;
  if (!aligned16(codes) || !aligned16(d_act) || !aligned16(d_fused) || !aligned16(act) || !aligned4(limit) ||
      !aligned4(weights) || !aligned4(row_slots) || !aligned4(dot))
    return RD_EINVAL;
  rd::GluMxProblem p{codes, static_cast<const uint8_t*>(scales), d_act, limit, weights, row_slots, d_fused, act, dot,
                     static_cast<int>(rows), static_cast<int>(h), slots};
  return rd::launch_glu_bwd_mx8(p, static_cast<hipStream_t>(stream));
}

int rd_tune_set(int32_t which, int32_t value) { return rd::tune_set(which, value); }

int rd_tune_tile_count(void) { return rd::tile_count(); }

}  // extern "C"
