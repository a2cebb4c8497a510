// MX quantisation for gfx950: rows of bf16 or float32 to 4- or 8-bit elements
// with a scale for every 32, back again, and the GLU whose [gate | up] input
// is kept in 8 bits for the backward pass.
//
// All are streams: a lane owns eight consecutive elements (16 bytes of bf16)
// and a quad of lanes one block, whose largest magnitude is found with two
// lane swaps.  Only rows below the limit are read or written.
#include "rd_glu_math.h"
#include "rd_launch.h"
#include "rd_mx_math.h"

#pragma clang fp contract(off)

namespace rd {
namespace {

__device__ __forceinline__ long long clamp_limit(const int32_t* limp, long long rows) {
  if (limp == nullptr) return rows;
  const long long v = *limp;
  return v < 0 ? 0 : (v > rows ? rows : v);
}

// Non-temporal accesses, for rows read once and outputs that are read much later, so that they do not displace
// what the next kernel reads.  65536 x 4096 bf16 to 4 bits and back, one after the other: 275 us without, 225 with
// (loads of the one, stores of the other).  The GLU forward of 32768 x 2048 (loads and codes) and its backward: 111
// without, 108 with; the backward itself gains nothing and keeps ordinary accesses.
typedef uint32_t nt_u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t nt_u32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint4 nt_load(const void* x, long long i) {
  const nt_u32x4 a = __builtin_nontemporal_load(static_cast<const nt_u32x4*>(x) + i);
  return make_uint4(a.x, a.y, a.z, a.w);
}
__device__ __forceinline__ void nt_store(void* x, long long i, uint4 v) {
  const nt_u32x4 a = {v.x, v.y, v.z, v.w};
  __builtin_nontemporal_store(a, static_cast<nt_u32x4*>(x) + i);
}
__device__ __forceinline__ void nt_store(void* x, long long i, uint2 v) {
  const nt_u32x2 a = {v.x, v.y};
  __builtin_nontemporal_store(a, static_cast<nt_u32x2*>(x) + i);
}

__device__ __forceinline__ void load8_once(const uint16_t* x, long long i, float (&v)[8]) { unpack8(nt_load(x, i), v); }
__device__ __forceinline__ void load8_once(const float* x, long long i, float (&v)[8]) {
  const uint4 a = nt_load(x, 2 * i), b = nt_load(x, 2 * i + 1);
  const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(u[k]);
}
__device__ __forceinline__ void store8_away(uint16_t* x, long long i, const float (&v)[8]) { nt_store(x, i, pack8(v)); }
__device__ __forceinline__ void store8_away(float* x, long long i, const float (&v)[8]) {
  uint32_t u[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) u[k] = __float_as_uint(v[k]);
  nt_store(x, 2 * i, make_uint4(u[0], u[1], u[2], u[3]));
  nt_store(x, 2 * i + 1, make_uint4(u[4], u[5], u[6], u[7]));
}
__device__ __forceinline__ void load8(const uint16_t* x, long long i, float (&v)[8]) {
  unpack8(reinterpret_cast<const uint4*>(x)[i], v);
}
__device__ __forceinline__ void store8(uint16_t* x, long long i, const float (&v)[8]) {
  reinterpret_cast<uint4*>(x)[i] = pack8(v);
}

// Codes of a lane's eight elements; returns the block's scale byte (the same in the quad).
template <int BITS>
__device__ __forceinline__ uint32_t encode8(const float (&x)[8], uint2& codes) {
  const uint32_t b = mx_scale<BITS>(quad_max(amax8(x)));
  const float inv = mx_inverse(b);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = b == kMxNan ? 0.f : x[i] * inv;
  if constexpr (BITS == 4)
    codes = make_uint2(to_e2m1x8(q), 0);
  else
    codes = to_e4m3x8(q);
  return b;
}
template <int BITS>
__device__ __forceinline__ void decode8(const uint8_t* codes, uint32_t scale, long long i, float (&v)[8]) {
  if constexpr (BITS == 4)
    from_e2m1x8(reinterpret_cast<const uint32_t*>(codes)[i], v);
  else
    from_e4m3x8(reinterpret_cast<const uint2*>(codes)[i], v);
  const float f = mx_factor(scale);
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] *= f;
}

// cols is a multiple of 32, so the valid rows are one run of blocks.  A wave takes U x 64 chunks of eight
// elements.  With U = 4 these are 64 blocks, whose scales it stores as one run of bytes (lane 4 q + u that of block
// q of its u-th 16).  Bandwidth-bound: at 65536 x 4096 bf16 to 4 bits the 0.68 GB take 110 us (6.2 TB/s).
constexpr long long kOneChunk = 1ll << 27;  // elements up to which U = 1 is faster, see below
template <int BITS, int U, class T>
__global__ __launch_bounds__(kThreads) void quantize_mx_kernel(const T* __restrict__ x, const int32_t* __restrict__ limp,
                                                               uint8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ scales, long long rows,
                                                               long long cols) {
  static_assert(U == 1 || U == 4, "the lanes' scales");
  const long long n = clamp_limit(limp, rows) * (cols / 8);
  const int lane = threadIdx.x & 63;
  const long long step = static_cast<long long>(gridDim.x) * (kThreads * U);
  for (long long i0 = static_cast<long long>(blockIdx.x) * (kThreads * U) + (threadIdx.x >> 6) * (64 * U); i0 < n;
       i0 += step) {
    float v[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long i = i0 + 64 * u + lane;
      if (i < n) {
        load8_once(x, i, v[u]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[u][k] = 0.f;
      }
    }
    uint32_t mine = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long i = i0 + 64 * u + lane;
      uint2 c;
      const uint32_t b = encode8<BITS>(v[u], c);
      if (U == 1 || (lane & 3) == u) mine = b;
      if (i < n) {
        if constexpr (BITS == 4)
          reinterpret_cast<uint32_t*>(codes)[i] = c.x;
        else
          reinterpret_cast<uint2*>(codes)[i] = c;
      }
    }
    const long long at = (i0 >> 2) + 16 * (lane & 3) + (lane >> 2);
    if ((U == 4 || (lane & 3) == 0) && at < (n >> 2)) scales[at] = static_cast<uint8_t>(mine);
  }
}

// The values: 65536 x 4096 of 4 bits to bf16, 0.69 GB, 115 us (6.0 TB/s).
template <int BITS, class T>
__global__ __launch_bounds__(kThreads) void dequantize_mx_kernel(const uint8_t* __restrict__ codes,
                                                                 const uint8_t* __restrict__ scales,
                                                                 const int32_t* __restrict__ limp, T* __restrict__ out,
                                                                 long long rows, long long cols) {
  const long long n = clamp_limit(limp, rows) * (cols / 8);
  for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < n;
       i += static_cast<long long>(gridDim.x) * kThreads) {
    float v[8];
    decode8<BITS>(codes, scales[i >> 2], i, v);
    store8_away(out, i, v);
  }
}

// act = silu(gate) * up of the bf16 input, and that input in MX 8-bit elements; one wave per row, so that a limit
// cuts whole waves and the 8-bit copy costs no second reading.  Bandwidth-bound: 32768 rows of h 1024, 0.27 GB, 43
// us (6.3 TB/s), and so down to h 512, where every lane has a chunk; h 256 reaches 4.7 TB/s, 128 2.6, 64 1.4.
__global__ __launch_bounds__(kThreads) void glu_fwd_mx8_kernel(const uint16_t* __restrict__ fused,
                                                               const int32_t* __restrict__ limp,
                                                               uint16_t* __restrict__ act, uint8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ scales, int rows, int h) {
  const int L = static_cast<int>(clamp_limit(limp, rows));
  const int hc = h >> 3, lane = threadIdx.x & 63;
  const int waves = gridDim.x * (kThreads / 64);
  for (int r = blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6); r < L; r += waves) {
    const long long fi = static_cast<long long>(r) * 2 * hc;  // the row's first 8-element chunk
    for (int c = lane; c < hc; c += 64) {
      float g[8], u[8], a[8];
      load8_once(fused, fi + c, g);
      load8_once(fused, fi + hc + c, u);
#pragma unroll
      for (int q = 0; q < 8; ++q) a[q] = glu_f32(g[q], u[q]);
      store8(act, static_cast<long long>(r) * hc + c, a);
      uint2 cg, cu;
      const uint32_t bg = encode8<8>(g, cg), bu = encode8<8>(u, cu);
      nt_store(codes, fi + c, cg);
      nt_store(codes, fi + hc + c, cu);
      if ((c & 3) == 0) {
        scales[(fi + c) >> 2] = static_cast<uint8_t>(bg);
        scales[(fi + hc + c) >> 2] = static_cast<uint8_t>(bu);
      }
    }
  }
}

struct GluBwdArgs {
  const uint8_t *codes, *scales;
  const uint16_t* d_act;
  const int32_t* limp;
  const float* weights;   // [slots] or null (all 1)
  const int32_t* row_at;  // row -> its slot, or null (slot r)
  uint16_t *d_fused, *act;
  float* dot;  // [slots]
  int rows, h;
  long long slots;
};

// One wave per row r with slot s and weight w: act = w silu(g) u, d_fused = w d times the GLU's partial
// derivatives, dot[s] = <d, silu(g) u>, which one wave sums: no partial sums, and the same result every time.
// Bandwidth-bound: 32768 rows of h 1024, 0.34 GB, 60 us (5.7 TB/s), h 512 5.6 TB/s; narrower rows leave lanes without
// a chunk: h 256 3.4 TB/s, 128 1.9, 64 1.1.
__global__ __launch_bounds__(kThreads) void glu_bwd_mx8_kernel(GluBwdArgs p) {
  const int L = static_cast<int>(clamp_limit(p.limp, p.rows));
  const int hc = p.h >> 3, lane = threadIdx.x & 63;
  const int waves = gridDim.x * (kThreads / 64);
  for (int r = blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6); r < L; r += waves) {
    const long long fi = static_cast<long long>(r) * 2 * hc;
    const long long at = p.row_at != nullptr ? p.row_at[r] : r;
    const bool ok = at >= 0 && at < p.slots;
    const float w = p.weights == nullptr ? 1.f : (ok ? p.weights[at] : 0.f);
    double acc = 0.0;
    for (int c = lane; c < hc; c += 64) {
      float g[8], u[8], d[8], a[8], dg[8], du[8];
      decode8<8>(p.codes, p.scales[(fi + c) >> 2], fi + c, g);
      decode8<8>(p.codes, p.scales[(fi + hc + c) >> 2], fi + hc + c, u);
      load8(p.d_act, static_cast<long long>(r) * hc + c, d);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float s = glu_f32(g[q], u[q]);
        acc += static_cast<double>(s * d[q]);
        a[q] = s * w;
        glu_grad_f32(g[q], u[q], d[q] * w, dg[q], du[q]);
      }
      store8(p.act, static_cast<long long>(r) * hc + c, a);
      store8(p.d_fused, fi + c, dg);
      store8(p.d_fused, fi + hc + c, du);
    }
#pragma unroll
    for (int k = 32; k >= 1; k >>= 1) acc += __shfl_xor(acc, k, 64);
    if (lane == 0 && ok) p.dot[at] = static_cast<float>(acc);
  }
}

int stream_grid(long long threads, int per_cu) {
  const long long blocks = (threads + kThreads - 1) / kThreads;
  const long long cap = static_cast<long long>(device_cu_count()) * per_cu;
  return static_cast<int>(blocks < cap ? (blocks < 1 ? 1 : blocks) : cap);
}

template <int BITS, class T>
void quantize_as(const T* x, const int32_t* limit, uint8_t* codes, uint8_t* scales, long long rows, long long cols,
                 hipStream_t stream) {
  // one chunk a lane, four times the waves: 512 x 4096 to 8 bits 3.1 us against 4.6, 8192 x 4096 19.4 against 21.2,
  // 32768 x 2048 34.6 against 38.0; 65536 x 4096 to 4 bits and back 234 against 225.  Float32, to 4 bits and back:
  // 2^24 elements 38.6 against 39.4, 2^25 81 against 80, 2^27 355 against 349, 2^28 766 against 745
  if (rows * cols <= kOneChunk)
    quantize_mx_kernel<BITS, 1>
        <<<stream_grid(rows * (cols / 8), 32), kThreads, 0, stream>>>(x, limit, codes, scales, rows, cols);
  else
    quantize_mx_kernel<BITS, 4>
        <<<stream_grid(rows * (cols / 8) / 4 + 1, 32), kThreads, 0, stream>>>(x, limit, codes, scales, rows, cols);
}
template <int BITS>
void quantize_as(const void* x, bool f32, const int32_t* limit, uint8_t* codes, uint8_t* scales, long long rows,
                 long long cols, hipStream_t stream) {
  if (f32)
    quantize_as<BITS>(static_cast<const float*>(x), limit, codes, scales, rows, cols, stream);
  else
    quantize_as<BITS>(static_cast<const uint16_t*>(x), limit, codes, scales, rows, cols, stream);
}
template <int BITS>
void dequantize_as(const uint8_t* codes, const uint8_t* scales, const int32_t* limit, void* out, bool f32,
                   long long rows, long long cols, hipStream_t stream) {
  const int grid = stream_grid(rows * (cols / 8), 32);
  if (f32)
    dequantize_mx_kernel<BITS><<<grid, kThreads, 0, stream>>>(codes, scales, limit, static_cast<float*>(out), rows,
                                                              cols);
  else
    dequantize_mx_kernel<BITS><<<grid, kThreads, 0, stream>>>(codes, scales, limit, static_cast<uint16_t*>(out), rows,
                                                              cols);
}

}  // namespace

int launch_quantize_mx(const void* x, bool f32, const int32_t* limit, void* codes, uint8_t* scales, long long rows,
                       long long cols, int bits, hipStream_t stream) {
  if (bits == 4)
    quantize_as<4>(x, f32, limit, static_cast<uint8_t*>(codes), scales, rows, cols, stream);
  else
    quantize_as<8>(x, f32, limit, static_cast<uint8_t*>(codes), scales, rows, cols, stream);
  return hipGetLastError() == hipSuccess ? RD_OK : RD_EHIP;
}

int launch_dequantize_mx(const void* codes, const uint8_t* scales, const int32_t* limit, void* out, bool f32,
                         long long rows, long long cols, int bits, hipStream_t stream) {
  if (bits == 4)
    dequantize_as<4>(static_cast<const uint8_t*>(codes), scales, limit, out, f32, rows, cols, stream);
  else
    dequantize_as<8>(static_cast<const uint8_t*>(codes), scales, limit, out, f32, rows, cols, stream);
  return hipGetLastError() == hipSuccess ? RD_OK : RD_EHIP;
}

int launch_glu_fwd_mx8(const void* fused, const int32_t* limit, void* act, void* codes, uint8_t* scales, int rows,
                       int h, hipStream_t stream) {
  glu_fwd_mx8_kernel<<<stream_grid(static_cast<long long>(rows) * 64, 32), kThreads, 0, stream>>>(
      static_cast<const uint16_t*>(fused), limit, static_cast<uint16_t*>(act), static_cast<uint8_t*>(codes), scales,
      rows, h);
  return hipGetLastError() == hipSuccess ? RD_OK : RD_EHIP;
}

int launch_glu_bwd_mx8(const GluMxProblem& q, hipStream_t stream) {
  GluBwdArgs a{static_cast<const uint8_t*>(q.codes), q.scales, static_cast<const uint16_t*>(q.d_act), q.limit,
               q.weights, q.row_at, static_cast<uint16_t*>(q.d_fused), static_cast<uint16_t*>(q.act), q.dot, q.rows,
               q.h, q.slots};
  glu_bwd_mx8_kernel<<<stream_grid(static_cast<long long>(a.rows) * 64, 32), kThreads, 0, stream>>>(a);
  return hipGetLastError() == hipSuccess ? RD_OK : RD_EHIP;
}

}  // namespace rd
