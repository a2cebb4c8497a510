// Routing to experts for gfx950: scores, top-k choice and weights of each
// token, the gradient of the logits, and the stable sort of the chosen slots
// by expert.
//
// One row of logits x gives scores s = softmax(x) or sigmoid(x) and keys
// k = x (without a bias; s grows with x, so the order is that of s) or
// k = s + bias.  With groups, an expert takes part only if its group is among
// the top_groups groups with the largest sum of their two largest s (+ bias),
// masked experts left out.
// The top_k largest keys are chosen, ties to the lowest index; a key of -inf
// (a masked expert) is never chosen and leaves the slot empty (id -1, weight
// 0).  The weights are the chosen s, or s over their sum, times scale.
//
// Keys are float64: neighbours of the last chosen score decide whole numbers,
// and float32 would decide some of them wrongly.  (Float32 keys with a check
// that sends the doubtful rows to float64 were slower: 49 us against the 21 of its time at
// 15769 x 256 rows, because the few rows that go twice end the launch.)  The
// lowest four bits of a key's 52 are replaced by the element's number in its
// lane, so that one comparison finds the value and the element, and ties go
// to the lower expert; float32 and bf16 logits have zeros there.  +inf and
// NaN rank as the largest key, -inf as "cannot be chosen".
#include <utility>

#include "rd_device.h"
#include "rd_launch.h"

namespace rd {
namespace {

struct RouteArgs {
  const void* logits;
  const float* bias;
  const int32_t* limp;
  float* weights;
  int32_t* ids;
  int T, E, K, groups, top_groups;
  bool sigmoid, renorm;
  float scale;
  int first;  // the launch's first row
};

// ---------------------------------------------------------------- a row's lanes

// LPR lanes (16 or 64) share a row; element j of a lane is expert j * LPR + sub.

// Rotation by N within the 16-lane row: a DPP move, no LDS.
template <int N, class T>
__device__ __forceinline__ T ror(T v) {
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + N, 0xF, 0xF, false));
  } else {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = ror<N>(static_cast<uint32_t>(u)), hi = ror<N>(static_cast<uint32_t>(u >> 32));
    return __builtin_bit_cast(T, lo | (hi << 32));
  }
}

// All lanes of a row get op over its lanes.
template <int LPR, class T, class Op>
__device__ __forceinline__ T row_all(T v, Op op) {
  v = op(v, ror<8>(v));
  v = op(v, ror<4>(v));
  v = op(v, ror<2>(v));
  v = op(v, ror<1>(v));
  if constexpr (LPR == 64) {
    v = op(v, __shfl_xor(v, 16, 64));
    v = op(v, __shfl_xor(v, 32, 64));
  }
  return v;
}
template <class T>
struct Max {
  __device__ __forceinline__ T operator()(T a, T b) const { return __builtin_elementwise_max(a, b); }
};
template <class T>
struct Add {
  __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};

// ---------------------------------------------------------------- keys

constexpr double kLargest = 1e300;  // keys lie in [-1e300, 1e300]; the lower end cannot be chosen

// A logit as its own key (the order of the scores): fmin and fmax give the other operand for NaN.
__device__ __forceinline__ double logit_key(float x) {
  return x == -INFINITY ? -kLargest : fmin(static_cast<double>(x), kLargest);
}

struct Exp2Terms {  // (ln 2)^k / k!
  double c[14];
  constexpr Exp2Terms() : c() {
    c[0] = 1.0;
    for (int k = 1; k < 14; ++k) c[k] = c[k - 1] * 0.6931471805599453094 / k;
  }
};

// x log2(e) as a whole number n and the rest r, |r| <= 1: log2(e) in two parts (the second is log2(e) less its
// double), so that r is off by 2^-53 however large x is, where x log2(e) rounded once would be off by |x| 2^-53.
struct Power {
  double n, r;
};
__device__ __forceinline__ Power power_of(double x) {
  constexpr double hi = 1.4426950408889634, lo = 2.0355273740931033e-17;
  const double n = __builtin_rint(x * hi);
  return {n, __builtin_fma(x, lo, __builtin_fma(x, hi, -n))};
}
// 2^(n + r) for n in [-1100, 1022], |r| <= 1/2, NaN for NaN: the power series, whose term k = 14 is below 2^-57.
__device__ __forceinline__ double exp2_of(double n, double r) {
  constexpr Exp2Terms T;
  double v = T.c[13];
#pragma unroll
  for (int k = 12; k >= 0; --k) v = __builtin_fma(v, r, T.c[k]);
  return __builtin_ldexp(v, static_cast<int>(n));
}
// e^x, the argument cut to where the result and 1 / (1 + result) are normal numbers
__device__ __forceinline__ double exp_of(double x) {
  x = x > 708.0 ? 708.0 : x;
  const Power p = power_of(x < -762.0 ? -762.0 : x);
  return exp2_of(p.n, p.r);
}
// e^(x - m), m the power of the largest x: the difference is taken after the multiplication, since x - m itself
// may need more than 53 bits
__device__ __forceinline__ double exp_below(double x, double largest, const Power& m) {
  const Power p = power_of(x);
  const double r = p.r - m.r, k = __builtin_rint(r);
  const double v = exp2_of(p.n - m.n + k, r - k);
  return x - largest < -762.0 ? 0.0 : v;
}
// 1 / y for a normal y: the hardware's estimate and two Newton steps
__device__ __forceinline__ double inverse(double y) {
  double r = __builtin_amdgcn_rcp(y);
  r = __builtin_fma(__builtin_fma(-y, r, 1.0), r, r);
  return __builtin_fma(__builtin_fma(-y, r, 1.0), r, r);
}

// Scores of a lane's elements; true where they are all NaN (a softmax over NaN or +inf).
template <int EPL, int LPR>
__device__ __forceinline__ bool scores(const float (&x)[EPL], float row_max, bool sigmoid, int sub, int E,
                                       double (&s)[EPL]) {
  if (sigmoid) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) s[j] = inverse(1.0 + exp_of(-static_cast<double>(x[j])));
    return false;
  }
  double sum = 0.0;
  const double largest = row_max;
  const Power m = power_of(largest);
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    s[j] = j * LPR + sub < E ? exp_below(static_cast<double>(x[j]), largest, m) : 0.0;
    sum += s[j];
  }
  sum = row_all<LPR>(sum, Add<double>());
  const double r = 1.0 / sum;
#pragma unroll
  for (int j = 0; j < EPL; ++j) s[j] *= r;
  return sum != sum;
}

// Bit g of the result: group g stays.  keys: the row's keys by expert, in LDS.
template <int LPR>
__device__ __forceinline__ uint32_t chosen_groups(const double* keys, int E, int groups, int top_groups, int sub) {
  const int per = E / groups;
  const int lane = threadIdx.x & 63, base = lane & ~(LPR - 1);
  // 2^share lanes look at a group's elements in turn: lane (g << share) | part
  int share = 0;
  while ((groups << (share + 1)) <= 16) ++share;
  const int part = sub & ((1 << share) - 1), g = sub >> share;
  double a = -kLargest, b = -kLargest;  // the two largest
  if (g < groups) {
#pragma unroll 4
    for (int n = part; n < per; n += 1 << share) {
      const double v = keys[g * per + n];
      b = fmax(b, fmin(a, v));
      a = fmax(a, v);
    }
  }
  for (int i = 0; i < share; ++i) {  // join the lanes of the group
    const double oa = __shfl_xor(a, 1 << i, 64), ob = __shfl_xor(b, 1 << i, 64);
    b = fmax(fmin(a, oa), fmax(b, ob));
    a = fmax(a, oa);
  }
  const double sum = b == -kLargest ? a : a + b;  // masked experts add nothing
  int rank = 0;
  for (int o = 0; o < groups; ++o) {
    const double other = __shfl(sum, base + (o << share), 64);
    rank += other > sum || (other == sum && o < g);
  }
  const uint32_t lanes = static_cast<uint32_t>(__ballot(g < groups && rank < top_groups) >> base);
  uint32_t bits = 0;
  for (int o = 0; o < groups; ++o) bits |= ((lanes >> (o << share)) & 1) << o;
  return bits;
}

// ---------------------------------------------------------------- forward

template <bool BF16>
__device__ __forceinline__ float logit(const void* x, long long at) {
  if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(x)[at]);
  return static_cast<const float*>(x)[at];
}

// Compare-exchanges of an odd-even merge sort of N elements, in order.
template <int N>
struct SortNetwork {
  int a[64] = {}, b[64] = {}, n = 0;
  constexpr SortNetwork() {
    for (int p = 1; p < N; p *= 2)
      for (int k = p; k >= 1; k /= 2)
        for (int j = k % p; j + k < N; j += 2 * k)
          for (int i = 0; i < k && i + j + k < N; ++i)
            if ((i + j) / (2 * p) == (i + j + k) / (2 * p)) {
              a[n] = i + j;
              b[n] = i + j + k;
              ++n;
            }
  }
};
template <int N, int... I>
__device__ __forceinline__ void sort_descending(double (&v)[N], std::integer_sequence<int, I...>) {
  constexpr SortNetwork<N> net;
  const auto exchange = [&](int a, int b) {
    const double hi = fmax(v[a], v[b]), lo = fmin(v[a], v[b]);
    v[a] = hi;
    v[b] = lo;
  };
  (exchange(net.a[I], net.b[I]), ...);
}

// The choice of one row: lane i of the row gets the i-th chosen expert or -1.  Each lane sorts its keys once
// (63 exchanges of two instructions for 16); a step then takes the largest of the lanes' heads and moves one
// lane on, where a search would look at all keys twice.  A lane carries its first HEADS >= min(EPL, top_k) keys:
// with 8 of 16 the step moves half as many.  (With that, and the groups' masks by scalars below, 15769 x 256 rows and
// 4 of 8 groups went from 22.1 to 17.7 us, 8192 x 256 rows without groups from 9.3 to 6.3.)
template <int EPL, int LPR, int HEADS>
__device__ __forceinline__ int choose(const RouteArgs& p, const float (&x)[EPL], float row_max, int sub, double* lds,
                                      bool& all_nan) {
  double key[EPL];
  if (p.bias != nullptr || p.groups > 1) {
    all_nan = scores<EPL, LPR>(x, row_max, p.sigmoid, sub, p.E, key);
    if (p.bias != nullptr) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) key[j] += j * LPR + sub < p.E ? static_cast<double>(p.bias[j * LPR + sub]) : 0.0;
    }
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j) key[j] = static_cast<double>(x[j]);
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j)  // fmin and fmax give the other operand for NaN
    key[j] = x[j] == -INFINITY ? -kLargest : fmax(fmin(key[j], kLargest), -kLargest);
  if (p.groups > 1) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) lds[j * LPR + sub] = key[j];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const uint32_t keep = chosen_groups<LPR>(lds, p.E, p.groups, p.top_groups, sub);
    const int per = p.E / p.groups;
    // e / per as a product: exact for e < 1024 (the error e / 2^20 is below 1 / per)
    const uint32_t inv = ((1u << 20) + per - 1) / per;
    if (p.bias == nullptr) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) key[j] = logit_key(x[j]);
    }
    if (per % LPR == 0) {  // a lane's j-th elements all lie in one group: its number is a scalar
      int g = 0, left = per / LPR;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        key[j] = g < 16 && ((keep >> g) & 1) ? key[j] : -kLargest;
        if (--left == 0) {
          ++g;
          left = per / LPR;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const uint32_t g = (static_cast<uint32_t>(j * LPR + sub) * inv) >> 20;
        key[j] = g < 16 && ((keep >> g) & 1) ? key[j] : -kLargest;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const uint64_t u = __builtin_bit_cast(uint64_t, key[j] + 0.0);  // -0 becomes +0
    const uint32_t hi = static_cast<uint32_t>(u >> 32);
    // for negative keys a larger number is a smaller key
    const uint32_t low = (15u - j) ^ (static_cast<uint32_t>(static_cast<int32_t>(hi) >> 31) & 15u);
    key[j] = __builtin_bit_cast(double, (u & ~15ull) | low);
  }
  sort_descending(key, std::make_integer_sequence<int, SortNetwork<EPL>().n>());
  double head[HEADS];
#pragma unroll
  for (int j = 0; j < HEADS; ++j) head[j] = key[j];
  const int base = threadIdx.x & 63 & ~(LPR - 1);
  int my_id = -1;
  for (int i = 0; i < p.K; ++i) {
    const double m = row_all<LPR>(head[0], Max<double>());
    const uint64_t heads = __ballot(head[0] == m) >> base;
    const int first = LPR == 64 ? __ffsll(static_cast<unsigned long long>(heads)) - 1
                                : __ffs(static_cast<int>(heads & 0xFFFFu)) - 1;
    if (sub == first) {  // a branch: as a selection between neighbours it became an indexed read of the array
#pragma unroll
      for (int j = 0; j + 1 < HEADS; ++j) head[j] = head[j + 1];
      head[HEADS - 1] = -kLargest;
    }
    const uint64_t u = __builtin_bit_cast(uint64_t, m);
    const uint32_t j = 15u - ((static_cast<uint32_t>(u) ^ static_cast<uint32_t>(static_cast<int64_t>(u) >> 63)) & 15u);
    if (sub == i && m > -0.99 * kLargest) my_id = static_cast<int>(j) * LPR + first;
  }
  return my_id;
}

template <int EPL, int LPR, int HEADS, bool BF16, bool GROUPS>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs p) {
  constexpr int RPW = 64 / LPR, NW = kThreads / 64;
  __shared__ double s_keys[GROUPS ? NW * RPW : 1][GROUPS ? EPL * LPR : 1];
  const int lane = threadIdx.x & 63, sub = lane & (LPR - 1), wave = threadIdx.x >> 6;
  const int slot = wave * RPW + lane / LPR;
  const int row = p.first + blockIdx.x * (NW * RPW) + slot;
  int L = p.T;
  if (p.limp != nullptr) {
    const int v = *p.limp;
    L = v < 0 ? 0 : (v > p.T ? p.T : v);
  }
  const bool live = row < L;
  if (__ballot(live) == 0) {
    if (row < p.T && sub < p.K) {
      p.weights[static_cast<long long>(row) * p.K + sub] = 0.f;
      p.ids[static_cast<long long>(row) * p.K + sub] = -1;
    }
    return;
  }
  if (!GROUPS) p.groups = p.top_groups = 1;
  const long long base = static_cast<long long>(live ? row : 0) * p.E;
  float x[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = j * LPR + sub;
    x[j] = live && e < p.E ? logit<BF16>(p.logits, base + e) : -INFINITY;
  }
  float row_max = x[0];
#pragma unroll
  for (int j = 1; j < EPL; ++j) row_max = fmaxf(row_max, x[j]);
  row_max = row_all<LPR>(row_max, Max<float>());

  bool all_nan = false;
  const int my_id = choose<EPL, LPR, HEADS>(p, x, row_max, sub, s_keys[GROUPS ? slot : 0], all_nan);

  // weights of the chosen, float32: q = s, or s over a common factor where they are renormalised
  const bool chosen = live && my_id >= 0;
  const float xi = chosen ? logit<BF16>(p.logits, base + my_id) : -INFINITY;
  float w = 0.f;
  if (p.renorm) {
    float m = row_all<LPR>(xi, Max<float>());
    float q = 0.f;
    if (chosen) {
      if (!p.sigmoid) {
        q = all_nan ? NAN : expf(xi - m);
      } else {  // sigmoid(x) over exp(m): no underflow, however far below 0 the row lies
        m = fminf(m, 0.f);
        q = xi <= 0.f ? expf(xi - m) / (1.f + expf(xi)) : 1.f / (1.f + expf(-xi));
      }
    }
    const float sum = row_all<LPR>(q, Add<float>());
    if (chosen) w = q / sum * p.scale;
  } else if (p.sigmoid) {
    if (chosen) w = p.scale / (1.f + expf(-xi));
  } else {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) sum += j * LPR + sub < p.E ? expf(x[j] - row_max) : 0.f;
    sum = row_all<LPR>(sum, Add<float>());
    if (chosen) w = expf(xi - row_max) / sum * p.scale;
  }
  if (row < p.T && sub < p.K) {
    p.weights[static_cast<long long>(row) * p.K + sub] = w;
    p.ids[static_cast<long long>(row) * p.K + sub] = live ? my_id : -1;
  }
}

// ---------------------------------------------------------------- backward

struct RouteBwdArgs {
  const void* logits;
  const int32_t* ids;
  const float* d_weights;
  void* d_logits;
  int T, E, K;
  bool sigmoid, renorm;
  float scale;
  int first;  // the launch's first row
};

// d_logits of one row.  With q the chosen scores: softmax without renormalisation
// p_i (d_i - <d, p>) for every expert; sigmoid q (1 - q) d for the chosen;
// renormalised, with w = q / sum: w (d - <d, w>), times (1 - q) for sigmoid.
// Where one p is near 1, its d_i - <d, p> is a small difference of nearly equal
// numbers: the exponentials are float32, their sum and all that follows is
// float64, so the p of a row add up to 1 within 2^-50 and the difference keeps
// the exponentials' accuracy (in float32 a p of 1 - 3e-4 left 2e-4 of it).
// The lanes that share a row hold it in registers, so logits are read once:
// 8192 x 64 bf16 3.8 us, of which launching takes over half.
template <int EPL, int LPR, bool BF16>
__global__ __launch_bounds__(kThreads) void route_bwd_kernel(RouteBwdArgs p) {
  constexpr int RPW = 64 / LPR, NW = kThreads / 64;
  const int lane = threadIdx.x & 63, sub = lane & (LPR - 1), wave = threadIdx.x >> 6;
  const int row = p.first + blockIdx.x * (NW * RPW) + wave * RPW + lane / LPR;
  const bool in = row < p.T;
  const long long at = static_cast<long long>(in ? row : 0) * p.E;
  int id = -1;
  float d = 0.f, xi = -INFINITY;
  if (in && sub < p.K) {
    id = p.ids[static_cast<long long>(row) * p.K + sub];
    if (id < 0 || id >= p.E) id = -1;
  }
  const bool chosen = id >= 0;
  if (chosen) {
    d = p.d_weights[static_cast<long long>(row) * p.K + sub] * p.scale;
    xi = logit<BF16>(p.logits, at + id);
  }
  const uint64_t row_bits = (LPR == 64 ? ~0ull : ((1ull << (LPR & 63)) - 1)) << (lane & ~(LPR - 1));
  const bool live = (__ballot(chosen) & row_bits) != 0;  // a row without a choice has a zero gradient
  float grad[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) grad[j] = 0.f;
  double v = 0.0, base = 0.0;  // the chosen expert's own term, and its share of what all experts of the row get
  if (!p.sigmoid && !p.renorm) {
    float x[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = j * LPR + sub;
      x[j] = live && e < p.E ? logit<BF16>(p.logits, at + e) : -INFINITY;
    }
    float m = x[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) m = fmaxf(m, x[j]);
    m = row_all<LPR>(m, Max<float>());
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      grad[j] = live && j * LPR + sub < p.E ? expf(x[j] - m) : 0.f;
      sum += grad[j];
    }
    sum = row_all<LPR>(sum, Add<double>());
    const double r = live ? 1.0 / sum : 0.0;
    const double pk = chosen ? expf(xi - m) * r : 0.0;
    const double dot = row_all<LPR>(chosen ? d * pk : 0.0, Add<double>());
#pragma unroll
    for (int j = 0; j < EPL; ++j) grad[j] = live ? grad[j] * static_cast<float>(-dot * r) : 0.f;
    v = pk * d;  // joined below: p (d - dot)
    base = -pk * dot;
  } else {
    const float q = chosen ? 1.f / (1.f + expf(-xi)) : 0.f, not_q = chosen ? 1.f / (1.f + expf(xi)) : 0.f;
    if (p.renorm) {
      float m = row_all<LPR>(xi, Max<float>());
      float u = 0.f;
      if (chosen) {
        if (!p.sigmoid) {
          u = expf(xi - m);
        } else {
          m = fminf(m, 0.f);
          u = xi <= 0.f ? expf(xi - m) * not_q : q;
        }
      }
      const double sum = row_all<LPR>(static_cast<double>(u), Add<double>());
      const double w = chosen ? u / sum : 0.0;
      const double dot = row_all<LPR>(chosen ? d * w : 0.0, Add<double>());
      v = chosen ? w * (d - dot) * (p.sigmoid ? not_q : 1.f) : 0.0;
    } else {
      v = chosen ? d * q * not_q : 0.f;
    }
  }
  // the chosen experts' gradients take the place of their share; an expert that is named twice adds up
  const int first = lane & ~(LPR - 1);
  for (int i = 0; i < p.K; ++i) {
    const double other = __shfl(v, first + i, 64);
    base += __shfl(id, first + i, 64) == id ? other : 0.0;
  }
  const float own = static_cast<float>(base);
  for (int i = 0; i < p.K; ++i) {
    const int e = __shfl(id, first + i, 64);
    const float t = __shfl(own, first + i, 64);
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (e == j * LPR + sub) grad[j] = t;
  }
  if (!in) return;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = j * LPR + sub;
    if (e < p.E) {
      if constexpr (BF16)
        static_cast<uint16_t*>(p.d_logits)[at + e] = static_cast<uint16_t>(f32_to_bf16(grad[j]));
      else
        static_cast<float*>(p.d_logits)[at + e] = grad[j];
    }
  }
}

// ---------------------------------------------------------------- slots sorted by expert

// A stable counting sort of n ids: workgroup b owns ids [b * span, (b + 1) *
// span), span = 512 * R, wave w of it a contiguous part, R ids a lane, which
// stay in registers.  Class E collects the ids outside [0, E).  Counts are
// whole numbers, so the order in which they are added does not matter, and a
// slot's place is the number of slots before it: results do not depend on
// timing.  Up to 4096 ids are one workgroup and one launch; more take a first
// launch that counts each workgroup's classes, and many more a second that adds
// the counts up.  Latency sets the time of few ids, not the bytes: 512 ids of 256
// experts 3.3 us, 225280 ids (2.7 MB) 11.9.  4194304 ids (50 MB) take 44: they are
// read and classified twice, and the counts' reads lie a class apart.
constexpr int kSortThreads = 512, kSortWaves = kSortThreads / 64, kSortMaxR = 8;
constexpr int kSortClasses = (RD_MAX_GROUPS + kSortThreads) / kSortThreads;  // classes a thread carries at most
static_assert(kSortClasses * kSortThreads >= RD_MAX_GROUPS + 1, "every class has a thread");

// Lanes of the wave, among the active ones, with the same class as this one (c < 2^bits).
__device__ __forceinline__ uint64_t same_class(int c, int bits) {
  uint64_t m = __ballot(true);
  for (int b = 0; b < bits; ++b) {
    const bool on = (c >> b) & 1;
    const uint64_t set = __ballot(on);
    m &= on ? set : ~set;
  }
  return m;
}

__device__ __forceinline__ int class_of(const int32_t* ids, int i, int hi, int E) {
  const int v = i < hi ? ids[i] : 0;
  return v >= 0 && v < E ? v : E;
}

template <int R>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(const int32_t* __restrict__ ids, int n, int E,
                                                                  int32_t* __restrict__ counts) {
  __shared__ int s_count[RD_MAX_GROUPS + 1];
  for (int e = threadIdx.x; e <= E; e += kSortThreads) s_count[e] = 0;
  const int lo = blockIdx.x * kSortThreads * R;
  int c[R];
#pragma unroll
  for (int r = 0; r < R; ++r) c[r] = class_of(ids, lo + r * kSortThreads + threadIdx.x, n, E);
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (lo + r * kSortThreads + static_cast<int>(threadIdx.x) < n) atomicAdd(&s_count[c[r]], 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += kSortThreads) counts[static_cast<long long>(blockIdx.x) * (E + 1) + e] = s_count[e];
}

// For many workgroups, each class's counts as the sums before each workgroup, and the whole at ``all``: a wave a
// class.  Up to kSortDirect workgroups add up the counts of the others themselves, which spares a launch: 256
// experts, 131072 ids (32 workgroups) 10.8 us against 11.7, 225280 (55) 13.5 against 11.9, 4194304 122 against 44.
constexpr int kSortDirect = 40;
__global__ __launch_bounds__(kThreads) void sort_scan_kernel(int32_t* __restrict__ counts, int32_t* __restrict__ all,
                                                             int blocks, int C) {
  const int lane = threadIdx.x & 63, e = blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (e >= C) return;
  int sum = 0;
  for (int b0 = 0; b0 < blocks; b0 += 64) {
    int32_t* at = counts + static_cast<long long>(b0 + lane) * C + e;
    const int v = b0 + lane < blocks ? *at : 0;
    const int upto = static_cast<int>(wave_incl_scan(v));
    if (b0 + lane < blocks) *at = sum + upto - v;
    sum += __shfl(upto, 63, 64);
  }
  if (lane == 0) all[e] = sum;
}

// counts: each workgroup's class counts (null: this is the only workgroup); all_of: null, or each class's sum,
// and counts those of the workgroups before.
template <int R>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(const int32_t* __restrict__ ids, int n, int E,
                                                                  const int32_t* __restrict__ counts,
                                                                  const int32_t* __restrict__ all_of,
                                                                  int32_t* __restrict__ sizes,
                                                                  int32_t* __restrict__ rows,
                                                                  int32_t* __restrict__ slots,
                                                                  int32_t* __restrict__ total) {
  __shared__ int s_part[kSortWaves * (RD_MAX_GROUPS + 1)];  // each wave's class counts, then its next places
  __shared__ long long s_wave[kSortWaves];
  const int C = E + 1;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int lo = (blockIdx.x * kSortWaves + wave) * (64 * R);
  int c[R];
#pragma unroll
  for (int r = 0; r < R; ++r) c[r] = class_of(ids, lo + r * 64 + lane, n, E);
  for (int i = threadIdx.x; i < kSortWaves * C; i += kSortThreads) s_part[i] = 0;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (lo + r * 64 + lane < n) atomicAdd(&s_part[wave * C + c[r]], 1);
  __syncthreads();
  // consecutive classes a thread: the slots of each in earlier workgroups, and in all of them
  const int per = (C + kSortThreads - 1) / kSortThreads;
  int before[kSortClasses], all[kSortClasses], sum = 0;
#pragma unroll
  for (int q = 0; q < kSortClasses; ++q) {
    const int e = threadIdx.x * per + q;
    before[q] = all[q] = 0;
    if (q < per && e < C) {
      if (counts == nullptr) {
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) all[q] += s_part[w * C + e];
      } else if (all_of != nullptr) {
        all[q] = all_of[e];
        before[q] = counts[static_cast<long long>(blockIdx.x) * C + e];
      } else {
        const int32_t* p = counts + e;
        const int blocks = gridDim.x, here = blockIdx.x;
#pragma unroll 8
        for (int b = 0; b < blocks; ++b) {
          const int v = p[b * C];
          before[q] += b < here ? v : 0;
          all[q] += v;
        }
      }
    }
    sum += all[q];
  }
  int start = static_cast<int>(block_excl_scan<kSortThreads>(sum, s_wave));
#pragma unroll
  for (int q = 0; q < kSortClasses; ++q) {
    const int e = threadIdx.x * per + q;
    if (q < per && e < C) {
      int at = start + before[q];
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        const int v = s_part[w * C + e];
        s_part[w * C + e] = at;
        at += v;
      }
      if (blockIdx.x == 0) {
        if (e < E)
          sizes[e] = all[q];
        else
          total[0] = start;  // class E starts where the experts' rows end
      }
    }
    start += all[q];
  }
  __syncthreads();
  const int bits = 32 - __clz(E);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = lo + r * 64 + lane;
    if (i < n) {  // the active lanes are the first ones; ballots count only them
      const uint64_t same = same_class(c[r], bits);
      const int rank = __popcll(same & ((1ull << lane) - 1));
      const int next = s_part[wave * C + c[r]];
      rows[next + rank] = i;
      slots[i] = c[r] < E ? next + rank : -1;
      // every lane of the class has read its next place (a wave's LDS operations run in order)
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (rank == 0) s_part[wave * C + c[r]] = next + __popcll(same);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// LPR lanes a row, in launches of 2^23 workgroups: a launch takes fewer than 2^32 threads.
template <int LPR, class Kernel, class Args>
void launch_rows(Kernel kernel, Args a, hipStream_t stream) {
  constexpr int per = kThreads / LPR, blocks = 1 << 23;
  for (long long first = 0; first < a.T; first += static_cast<long long>(per) * blocks) {
    a.first = static_cast<int>(first);
    const long long want = (a.T - first + per - 1) / per;
    kernel<<<static_cast<int>(want < blocks ? want : blocks), kThreads, 0, stream>>>(a);
  }
}

template <int EPL, int LPR, int HEADS, bool BF16>
void launch_route_as(const RouteArgs& a, hipStream_t stream) {
  if (a.groups > 1)
    launch_rows<LPR>(route_kernel<EPL, LPR, HEADS, BF16, true>, a, stream);
  else
    launch_rows<LPR>(route_kernel<EPL, LPR, HEADS, BF16, false>, a, stream);
}
template <int EPL, int LPR, int HEADS>
void launch_route_as(const RouteArgs& a, bool bf16, hipStream_t stream) {
  if (bf16)
    launch_route_as<EPL, LPR, HEADS, true>(a, stream);
  else
    launch_route_as<EPL, LPR, HEADS, false>(a, stream);
}

template <int EPL, int LPR>
void launch_route_bwd_as(const RouteBwdArgs& a, bool bf16, hipStream_t stream) {
  if (bf16)
    launch_rows<LPR>(route_bwd_kernel<EPL, LPR, true>, a, stream);
  else
    launch_rows<LPR>(route_bwd_kernel<EPL, LPR, false>, a, stream);
}

int sort_blocks(long long n) {
  constexpr long long span = kSortThreads * kSortMaxR;
  return n <= span ? 1 : static_cast<int>((n + span - 1) / span);
}

template <int R>
void launch_sort(const int32_t* ids, int n, int experts, int blocks, int32_t* sizes, int32_t* rows, int32_t* slots,
                 int32_t* total, int32_t* counts, hipStream_t stream) {
  const int C = experts + 1, waves = kThreads / 64;
  int32_t* all = blocks > kSortDirect ? counts + static_cast<long long>(blocks) * C : nullptr;
  if (blocks > 1) sort_count_kernel<R><<<blocks, kSortThreads, 0, stream>>>(ids, n, experts, counts);
  if (all != nullptr) sort_scan_kernel<<<(C + waves - 1) / waves, kThreads, 0, stream>>>(counts, all, blocks, C);
  sort_place_kernel<R><<<blocks, kSortThreads, 0, stream>>>(ids, n, experts, blocks > 1 ? counts : nullptr, all, sizes,
                                                            rows, slots, total);
}

}  // namespace

int launch_route(const RouteProblem& q, hipStream_t stream) {
  RouteArgs a{q.logits, q.bias, q.limit, q.weights, q.ids, q.tokens, q.experts, q.top_k, q.groups, q.top_groups,
              q.sigmoid, q.renorm, q.scale, 0};
  if (q.experts <= 64)
    launch_route_as<4, 16, 4>(a, q.bf16, stream);
  else if (q.experts <= 128)
    launch_route_as<8, 16, 8>(a, q.bf16, stream);
  else if (q.experts <= 256)
    q.top_k <= 8 ? launch_route_as<16, 16, 8>(a, q.bf16, stream) : launch_route_as<16, 16, 16>(a, q.bf16, stream);
  else if (q.experts <= 512)
    launch_route_as<8, 64, 8>(a, q.bf16, stream);
  else
    q.top_k <= 8 ? launch_route_as<16, 64, 8>(a, q.bf16, stream) : launch_route_as<16, 64, 16>(a, q.bf16, stream);
  return hipGetLastError() == hipSuccess ? RD_OK : RD_EHIP;
}

int launch_route_bwd(const RouteProblem& q, const float* d_weights, void* d_logits, hipStream_t stream) {
  RouteBwdArgs a{q.logits, q.ids, d_weights, d_logits, q.tokens, q.experts, q.top_k, q.sigmoid, q.renorm, q.scale, 0};
  if (q.experts <= 64)
    launch_route_bwd_as<4, 16>(a, q.bf16, stream);
  else if (q.experts <= 128)
    launch_route_bwd_as<8, 16>(a, q.bf16, stream);
  else if (q.experts <= 256)
    launch_route_bwd_as<16, 16>(a, q.bf16, stream);
  else if (q.experts <= 512)
    launch_route_bwd_as<8, 64>(a, q.bf16, stream);
  else
    launch_route_bwd_as<16, 64>(a, q.bf16, stream);
  return hipGetLastError() == hipSuccess ? RD_OK : RD_EHIP;
}

size_t group_rows_workspace_size(long long n, int experts) {
  const int blocks = sort_blocks(n);
  // counts of every workgroup and class, and the classes' sums
  return blocks <= 1 ? 0 : (static_cast<size_t>(blocks + 1) * (experts + 1) * 4 + 15) / 16 * 16;
}

int launch_group_rows(const int32_t* ids, int n, int experts, int32_t* sizes, int32_t* rows, int32_t* slots,
                      int32_t* total, int32_t* counts, hipStream_t stream) {
  const int blocks = sort_blocks(n);
  // as few ids a lane as one workgroup needs, since a lane's ids follow each other: 2048 ids 4.6 us with four,
  // 6.3 with eight; many workgroups take eight, so that there are fewer counts: 131072 ids 10.6 us, 15.4 with four
  if (n <= kSortThreads)
    launch_sort<1>(ids, n, experts, blocks, sizes, rows, slots, total, counts, stream);
  else if (n <= kSortThreads * 3)
    launch_sort<3>(ids, n, experts, blocks, sizes, rows, slots, total, counts, stream);
  else if (n <= kSortThreads * 4)
    launch_sort<4>(ids, n, experts, blocks, sizes, rows, slots, total, counts, stream);
  else
    launch_sort<kSortMaxR>(ids, n, experts, blocks, sizes, rows, slots, total, counts, stream);
  return hipGetLastError() == hipSuccess ? RD_OK : RD_EHIP;
}

}  // namespace rd
