// The rows' way to the experts and back for gfx950: token rows copied to
// their slots of the expert-sorted buffer, expert outputs added up for each
// token, and the gradients of that sum.
//
// slots[t, i] is the row that token t's i-th choice has in the sorted buffer,
// -1 (or anything outside [0, rows)) where it has none: such a choice is
// neither read nor written and adds nothing.
#include "rd_device.h"
#include "rd_launch.h"

namespace rd {
namespace {

typedef unsigned int nt_u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint4 nt_load(const uint4* p) {
  const nt_u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const nt_u32x4*>(p));
  return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ void nt_store(uint4* p, uint4 v) {
  const nt_u32x4 x = {v.x, v.y, v.z, v.w};
  __builtin_nontemporal_store(x, reinterpret_cast<nt_u32x4*>(p));
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

struct RowsArgs {
  const uint4* in;       // dispatch: x; combine: y; combine_bwd: g
  const uint4* y;        // combine_bwd only
  const int32_t* slots;  // [T, K]
  const float* weights;  // [T, K] or null (all 1)
  uint4* out;            // dispatch: xs; combine: out; combine_bwd: dy
  float* dw;             // combine_bwd only
  int T, K;
  int chunks;            // 16-byte chunks per row
  long long rows;        // rows of the sorted buffer
  int parts;             // parts a row is cut into (one wave each)
  int first;             // the launch's first wave
};

// The wave's number in the call, known to be the same in its lanes (slots and weights then come through
// the scalar cache, and their addresses stay out of the vector registers).
__device__ __forceinline__ long long wave_index(const RowsArgs& p) {
  return __builtin_amdgcn_readfirstlane(p.first + static_cast<int>(blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6)));
}
__device__ __forceinline__ long long slot_of(const RowsArgs& p, long long t, int i) {
  const long long s = p.slots[t * p.K + i];
  return s >= 0 && s < p.rows ? s : -1;
}

constexpr int kChunks = 8;  // 16-byte chunks of a row that a lane of dispatch carries at once

// One wave per (choice, part of its row).  The waves of a token follow each other and find its row in the caches;
// what bounds the copy is the writing, which goes on in whole rows: the packed buffer's 126152 rows of 8 KB take
// 221 us (5.3 TB/s with x's bytes), where one wave that wrote the row to all of its slots in turn took 235, sorted
// rows that were gathered 289, and 4 KB a wave 227.  (1 KB a wave gains 0.2 us below 128 choices and loses from 512.)
// Rows of 1024 and more reach 6.3 TB/s where they fit the caches, 512 4.4, 256 2.4, 128 1.2: a wave a row, and most of
// its loads empty.
__global__ __launch_bounds__(kThreads) void dispatch_rows_kernel(RowsArgs p) {
  const int lane = threadIdx.x & 63;
  const long long unit = wave_index(p);
  const long long choice = unit / p.parts;
  if (choice >= static_cast<long long>(p.T) * p.K) return;
  const int part = static_cast<int>(unit - choice * p.parts);
  const long long s = p.slots[choice];
  if (s < 0 || s >= p.rows) return;
  const uint4* from = p.in + choice / p.K * p.chunks;
  for (int c0 = part * 64 + lane; c0 < p.chunks; c0 += p.parts * 64 * kChunks) {
    uint4 v[kChunks];
#pragma unroll
    for (int q = 0; q < kChunks; ++q)
      if (c0 + p.parts * 64 * q < p.chunks) v[q] = from[c0 + p.parts * 64 * q];
#pragma unroll
    for (int q = 0; q < kChunks; ++q)
      if (c0 + p.parts * 64 * q < p.chunks) nt_store(p.out + s * p.chunks + c0 + p.parts * 64 * q, v[q]);
  }
}

// One wave per (token, part of its row): the K rows' parts are read four at a time and added in the order
// of the choices.  Bandwidth-bound: 8192 tokens of 4 rows of 4096, 0.34 GB, 58 us (5.8 TB/s); rows of 512 5.3 TB/s,
// 256 3.9, 128 2.3.
__global__ __launch_bounds__(kThreads) void combine_rows_kernel(RowsArgs p) {
  constexpr int AT = 4;
  const int lane = threadIdx.x & 63;
  const long long unit = wave_index(p);
  const long long t = unit / p.parts;
  if (t >= p.T) return;
  const int part = static_cast<int>(unit - t * p.parts);
  for (int c = part * 64 + lane; c < p.chunks; c += p.parts * 64) {
    float acc[8] = {};
    for (int i0 = 0; i0 < p.K; i0 += AT) {
      uint4 v[AT];
      float w[AT];
      bool on[AT];
#pragma unroll
      for (int a = 0; a < AT; ++a) {
        const long long s = i0 + a < p.K ? slot_of(p, t, i0 + a) : -1;
        on[a] = s >= 0;
        if (on[a]) {
          w[a] = p.weights != nullptr ? p.weights[t * p.K + i0 + a] : 1.f;
          v[a] = nt_load(p.in + s * p.chunks + c);
        }
      }
#pragma unroll
      for (int a = 0; a < AT; ++a) {
        if (!on[a]) continue;
        const uint32_t u[4] = {v[a].x, v[a].y, v[a].z, v[a].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          acc[2 * q] += w[a] * bf_lo(u[q]);
          acc[2 * q + 1] += w[a] * bf_hi(u[q]);
        }
      }
    }
    p.out[t * p.chunks + c] = make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                                         pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
  }
}

// One wave per choice: dy[slot] = w g[t], dw = <g[t], y[slot]>, the products exact in float32 and added
// in float64 in a fixed order, so dw is the exact dot rounded once.  Bandwidth-bound: 8192 tokens of 4 rows of 4096,
// 0.60 GB (g's rows come from the caches after the first choice), 112 us (5.4 TB/s); rows of 512 5.5 TB/s, 256 3.6,
// 128 1.9.
__global__ __launch_bounds__(kThreads) void combine_rows_bwd_kernel(RowsArgs p) {
  const int lane = threadIdx.x & 63;
  const long long unit = wave_index(p);
  const long long t = unit / p.K;
  if (t >= p.T) return;
  const long long s = slot_of(p, t, static_cast<int>(unit - t * p.K));
  double acc = 0.0;
  if (s >= 0) {
    const float w = p.weights != nullptr ? p.weights[unit] : 1.f;
    for (int c = lane; c < p.chunks; c += 64) {
      const uint4 g = p.in[t * p.chunks + c], y = nt_load(p.y + s * p.chunks + c);
      const uint32_t gu[4] = {g.x, g.y, g.z, g.w}, yu[4] = {y.x, y.y, y.z, y.w};
      uint32_t o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        o[q] = pack_bf16x2(bf_lo(gu[q]) * w, bf_hi(gu[q]) * w);
        acc += static_cast<double>(bf_lo(gu[q]) * bf_lo(yu[q]));
        acc += static_cast<double>(bf_hi(gu[q]) * bf_hi(yu[q]));
      }
      nt_store(p.out + s * p.chunks + c, make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) acc += __shfl_xor(acc, d, 64);
  if (lane == 0) p.dw[unit] = static_cast<float>(acc);
}

// One wave a unit, in launches of 2^25: a launch takes fewer than 2^32 threads.  units < 2^31.
template <class Kernel>
int launch_waves(Kernel kernel, RowsArgs a, long long units, hipStream_t stream) {
  constexpr long long most = 1ll << 25, per = kThreads / 64;
  for (long long first = 0; first < units; first += most) {
    a.first = static_cast<int>(first);
    const long long n = units - first < most ? units - first : most;
    kernel<<<static_cast<int>((n + per - 1) / per), kThreads, 0, stream>>>(a);
    if (hipGetLastError() != hipSuccess) return RD_EHIP;
  }
  return RD_OK;
}

// per: chunks of a row that one wave carries
RowsArgs args_of(const RowsProblem& q, int per) {
  RowsArgs a{};
  a.in = static_cast<const uint4*>(q.in);
  a.y = static_cast<const uint4*>(q.y);
  a.slots = q.slots;
  a.weights = q.weights;
  a.out = static_cast<uint4*>(q.out);
  a.dw = q.dw;
  a.T = q.tokens;
  a.K = q.top_k;
  a.chunks = q.hidden / 8;
  a.rows = q.rows;
  a.parts = (a.chunks + per - 1) / per;
  return a;
}

}  // namespace

int launch_dispatch_rows(const RowsProblem& q, hipStream_t stream) {
  const long long choices = static_cast<long long>(q.tokens) * q.top_k;
  RowsArgs a = args_of(q, 64 * kChunks);
  const long long most = ((1ll << 31) - 8) / (choices > 0 ? choices : 1);  // waves are numbered in 32 bits
  if (a.parts > most) a.parts = static_cast<int>(most);  // >= 1: choices < 2^31, and a wave takes parts in turn
  return launch_waves(dispatch_rows_kernel, a, choices * a.parts, stream);
}

int launch_combine_rows(const RowsProblem& q, hipStream_t stream) {
  const RowsArgs a = args_of(q, 64);
  return launch_waves(combine_rows_kernel, a, static_cast<long long>(a.T) * a.parts, stream);
}

int launch_combine_rows_bwd(const RowsProblem& q, hipStream_t stream) {
  const RowsArgs a = args_of(q, 64);
  return launch_waves(combine_rows_bwd_kernel, a, static_cast<long long>(a.T) * a.K, stream);
}

}  // namespace rd
