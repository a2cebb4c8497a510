// ragged_dot on MX operands for gfx950: out[rows of local group j] =
// x[rows] @ w[j]^T, w [num_local, n, k] in 4-bit E2M1 elements, x [m, k] in 4-
// or 8-bit (E4M3) ones, both with one E8M0 scale for every 32 along k.
//
// The matrix instructions take the codes and the scales as they lie in memory
// (v_mfma_scale_f32_16x16x128_f8f6f4: 128 products deep, float32 sums).  With
// an 8-bit operand it first adds eight neighbours in fewer bits: measured, and
// matched sum for sum by that rule, each product is cut off below 2^-13 of
// 2^e, e the largest sum of a product's two exponents in the eight (products
// that are zero left out; an exponent is at least that of the format's normal
// numbers).  E4M3 spans too many exponents for that: at 512 x 4096 normally
// distributed rows 5e-6 of the sums was lost.  So x is taken in two parts, the
// elements of 2 and more and those below.  In the first, exponents are 1 to 8
// for x and 0 to 2 for w: nothing is cut below 2^-3, and every product is a
// multiple of 2^-2 * 2^-1; in the second at most 0 and 2, nothing is cut below
// 2^-11, and products are multiples of 2^-9 * 2^-1.  With 4-bit operands
// products lie between 2^-2 and 36, and nothing is cut.  The second
// instruction and the split cost 8-bit rows 6 % where the weights' bandwidth
// is the bound (decode, below: 56.6 us to 60) and up to 44 % where it is not
// (8192 rows over 64 Zipf groups of 2048 x 4096: 137 to 173 us; 32768 rows of
// equal groups: 352 to 508; 8192^3: 680 to 894).
// The weights are its first operand, so a lane ends up with four neighbouring
// columns of one row.  Lane group q (16 lanes each) supplies the elements and
// the scale of the instruction's block q: neighbouring lanes hold different
// rows.  Both operands therefore come through LDS, by loads that go there
// directly, 1 KB of whole 64- to 256-byte pieces of rows at a time: loaded into the
// registers of those lanes they took 42 cache accesses an instruction, and
// the caches, not the memory, set the time (decode, 512 rows over 128 groups of
// 1536 x 4096 weights and 8-bit x in one part: 83 us against 56; a training step's
// up-projection, 8192 rows over 64 groups of 2048 x 4096 and 4-bit x: 119
// against 98).  A row's scales of a window are one 16-byte read, from which a
// lane shifts its own byte down.
#include "rd_device.h"
#include "rd_dma.h"
#include "rd_launch.h"

namespace rd {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

constexpr uint32_t kOutside = 0x80000000;  // a buffer offset past every operand: reads as zeros

struct MxArgs {
  const uint8_t *x, *xs, *w, *ws;
  const int32_t *gs, *offp, *limp;
  void* out;
  int G, gl, m, k, n;
  int out_f32;
};

// Rows [row0, row0 + rows) of an operand with row_bytes bytes a row: reads past them give zeros.
__device__ __forceinline__ u32x4_t rows_of(const uint8_t* base, long long row0, int rows, int row_bytes) {
  return uniform(make_rsrc(base + row0 * row_bytes, static_cast<unsigned long long>(rows) * row_bytes));
}

// All of this wave's LDS reads have returned.
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(vmcnt_imm(63) & ~(0xF << 8)); }

// A window of rows in LDS: CH 16-byte chunks a row, 64 / CH rows per 1 KB load, whose lane i writes place
// i % CH of row i / CH.  Chunk c of row r lies at place c ^ swizzle(r), so that 16 rows' reads of one chunk
// use different banks.
template <int CH>
struct Rows {
  static constexpr int kBytes = CH * 16, kPerLoad = 64 / CH;
  __device__ __forceinline__ static int swizzle(int row) {
    return CH >= 16 ? row & 15 : (CH == 8 ? (row >> 1) & 7 : (row >> 2) & 3);
  }
  __device__ __forceinline__ static int chunk_of_lane(int row) {
    return (threadIdx.x & (CH - 1)) ^ swizzle(row);
  }
  __device__ __forceinline__ static i32x4_t read(const char* rows, int row, int chunk) {
    return *reinterpret_cast<const i32x4_t*>(rows + row * kBytes + ((chunk ^ swizzle(row)) << 4));
  }
};

// Loads of N x 1 KB into LDS, rows row0 + (0 .. N * 64 / CH - 1) of the buffer, row0 a multiple of 16.
template <int CH, int N>
struct RowLoads {
  static constexpr int kPeriod = 16 / Rows<CH>::kPerLoad > 0 ? 16 / Rows<CH>::kPerLoad : 1;  // loads per 16 rows
  static constexpr int kKept = kPeriod < N ? kPeriod : N;
  uint32_t off[kKept];
  int left[kKept];  // bytes of the row from the lane's chunk to the row's end

  __device__ __forceinline__ void init(int row0, int row_bytes) {
#pragma unroll
    for (int s = 0; s < kKept; ++s) {
      const int row = row0 + s * Rows<CH>::kPerLoad + (threadIdx.x & 63) / CH;
      const int at = Rows<CH>::chunk_of_lane(row) * 16;
      off[s] = static_cast<uint32_t>(row) * row_bytes + at;
      left[s] = row_bytes - at;
    }
  }
  // kbyte: the window's first byte of each row; what lies past the row's end is read as zeros.  NT: data used
  // once, which is not to displace the rows of x in the caches.
  template <bool NT = false>
  __device__ __forceinline__ void issue(u32x4_t r, uint32_t lds, int row_bytes, int kbyte) const {
#pragma unroll
    for (int s = 0; s < N; ++s) {
      const uint32_t past = kbyte < left[s % kKept] ? 0u : kOutside;
      const uint32_t voff = (off[s % kKept] + (s / kKept) * (16 * row_bytes)) | past;
      if constexpr (NT)
        dma16_nt(r, lds + s * 1024, voff, uniform(kbyte));
      else
        dma16(r, lds + s * 1024, voff, uniform(kbyte));
    }
  }
};

// Rows below L outside the window's rows are written as +0.
template <int NT>
__device__ __forceinline__ void zero_other_rows(const MxArgs& p, const Window& win) {
  const long long row = static_cast<long long>(p.n) * (p.out_f32 ? 4 : 2) / 16;
  const long long a = static_cast<long long>(win.lo) * row, n = a + static_cast<long long>(win.L - win.hi) * row;
  uint4* out = static_cast<uint4*>(p.out);
  const long long hi = static_cast<long long>(win.hi) * row;
  for (long long i = static_cast<long long>(blockIdx.x) * NT + threadIdx.x; i < n;
       i += static_cast<long long>(gridDim.x) * NT)
    out[i < a ? i : hi + (i - a)] = make_uint4(0, 0, 0, 0);
}

template <int XB>
__device__ __forceinline__ f32x4_t mma(i32x8_t w, i32x8_t x, f32x4_t c, int ws, int xs) {
  // formats: 4 is E2M1, 0 is E4M3; the scale is the lowest byte
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 4, XB == 4 ? 4 : 0, 0, ws, 0, xs);
}

// The E4M3 elements of 2 and more (the top bit of the exponent is bit 6 of a byte), zeros for the others.
__device__ __forceinline__ i32x8_t large_part(i32x8_t v) {
  i32x8_t r;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = static_cast<uint32_t>(v[i]);
    // selectors 8 to 11 fill a byte with bit 15 or 31 of the second or of the first word
    r[i] = static_cast<int>(u & __builtin_amdgcn_perm(u << 9, u << 1, 0x090B080Au));
  }
  return r;
}

// acc[a] += w[a] x over one instruction's 128 elements.
template <int XB, int NI>
__device__ __forceinline__ void mma_columns(const i32x8_t (&w)[NI], i32x8_t x, f32x4_t (&acc)[NI],
                                            const uint32_t (&ws)[NI], uint32_t xs) {
  if constexpr (XB == 8) {
    const i32x8_t large = large_part(x);
#pragma unroll
    for (int a = 0; a < NI; ++a) acc[a] = mma<XB>(w[a], large, acc[a], ws[a], xs);
    x ^= large;
  }
#pragma unroll
  for (int a = 0; a < NI; ++a) acc[a] = mma<XB>(w[a], x, acc[a], ws[a], xs);
}

// An operand's registers: 16 bytes of E2M1 codes or two times 16 of E4M3 ones (elements 16 q on and 64 + 16 q on).
__device__ __forceinline__ i32x8_t operand(const i32x4_t& a) { return i32x8_t{a[0], a[1], a[2], a[3], 0, 0, 0, 0}; }
__device__ __forceinline__ i32x8_t operand(const i32x4_t (&v)[1]) { return operand(v[0]); }
__device__ __forceinline__ i32x8_t operand(const i32x4_t (&v)[2]) {
  return i32x8_t{v[0][0], v[0][1], v[0][2], v[0][3], v[1][0], v[1][1], v[1][2], v[1][3]};
}

// ---------------------------------------------------------------- few rows, few groups

// A few rows of a few groups make too few tiles for the CUs, so the contraction
// is split.  The work is counted in columns of blocks (16 rows of a group x 16
// columns), and every workgroup takes an equal run of them, two at a time.  Its
// four waves share the contraction: wave w multiplies windows w, w + 4, ... of
// 512 elements, and the four sums are added in the waves' order through LDS.  A
// wave has its part of LDS for itself: it waits for its own loads, reads the
// window into registers, starts the next window's loads (of the next pass
// too) and multiplies, so about 17 KB a wave are on their way at all times,
// with no barrier but the two of a pass's sums.
//
// The limits are the largest mean of rows a local group and the most tiles where
// this was faster: with 16 rows of 4-bit x and 4096 x 2048 weights, one group (16
// tiles) took 7.0 us against 11.9 in tiles (8-bit x 8.0 against 14.3), 4 groups (64)
// 8.6 against 12.2 (10.4, 14.7), 8 groups (128) 12.5 against 13.0 (14.5, 15.1), and
// 16 groups of 4096 x 1536 (192) 14.6 against 13.4 (17.5, 15.3); 1536 rows over 128
// groups of these took 98 us against 60.
constexpr int kFewRows = 24, kFewTiles = 128;
constexpr int kWin = 512, kFewN = 2;

template <int XB>
struct FewLds {  // bytes of a wave's part
  static constexpr int kXRow = kWin * XB / 8, kX = 16 * kFewN * 256, kWs = kX + 16 * kXRow, kXs = kWs + 16 * kFewN * 16,
                       kBytes = kXs + 256;
};

struct FewPass {
  int c0, cnt;     // first column block, how many
  int row0, rows;  // rows of x
  u32x4_t w, ws, x, xs;
};

template <int XB>
__global__ __launch_bounds__(kThreads, 2) void ragged_dot_mx_few(MxArgs p) {
  constexpr int BM = 16, NI = kFewN;
  typedef FewLds<XB> At;
  typedef Rows<16> WRows;
  typedef Rows<At::kXRow / 16> XRows;
  __shared__ __attribute__((aligned(1024))) char s_ops[4 * At::kBytes];
  __shared__ __attribute__((aligned(16))) float s_red[4][16 * 16 * NI];
  __shared__ int s_lb[kFewTiles + 1];
  __shared__ int s_tiles[kFewTiles + 1];
  __shared__ long long s_wave[kThreads / 64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
  const Window win = build_local_bounds(p.gs, p.G, p.offp, p.gl, p.limp, p.m, s_lb, s_wave);
  const int total_m = tile_prefix(s_lb, p.gl, BM, s_tiles, s_wave);
  const int nb = (p.n + 15) / 16;
  const long long total = static_cast<long long>(total_m) * nb;
  long long at = total * blockIdx.x / gridDim.x;
  const long long end = total * (blockIdx.x + 1) / gridDim.x;
  const int kb = p.k / 32, wbytes = p.k / 2, xbytes = p.k * XB / 8;  // scales and bytes a row

  const auto next_pass = [&](FewPass& t) -> bool {
    if (at >= end) return false;
    const int mt = static_cast<int>(at / nb);
    t.c0 = static_cast<int>(at - static_cast<long long>(mt) * nb);
    t.cnt = static_cast<int>(min(static_cast<long long>(min(NI, nb - t.c0)), end - at));
    at += t.cnt;
    const int j = __builtin_amdgcn_readfirstlane(upper_index(s_tiles, p.gl, mt));
    t.row0 = __builtin_amdgcn_readfirstlane(s_lb[j] + (mt - s_tiles[j]) * BM);
    t.rows = __builtin_amdgcn_readfirstlane(min(BM, s_lb[j + 1] - t.row0));
    const long long col0 = static_cast<long long>(j) * p.n + t.c0 * 16;
    const int cols = min(t.cnt * 16, p.n - t.c0 * 16);
    t.w = rows_of(p.w, col0, cols, wbytes);
    t.ws = rows_of(p.ws, col0, cols, kb);
    t.x = rows_of(p.x, t.row0, t.rows, xbytes);
    t.xs = rows_of(p.xs, t.row0, t.rows, kb);
    return true;
  };
  char* mine = s_ops + wave * At::kBytes;
  const uint32_t lds = lds_address(mine);
  RowLoads<16, 4 * NI> w_loads;
  RowLoads<At::kXRow / 16, At::kXRow / 64> x_loads;
  w_loads.init(0, wbytes);
  x_loads.init(0, xbytes);
  const uint32_t s_off = static_cast<uint32_t>(lane / 4) * kb + (lane & 3) * 4;  // scales: 4 words a row
  const auto load = [&](const FewPass& t, int k0) {
    w_loads.template issue<true>(t.w, lds, wbytes, k0 / 2);
    x_loads.issue(t.x, lds + At::kX, xbytes, k0 * XB / 8);
#pragma unroll
    for (int a = 0; a < NI; ++a) dma4(t.ws, lds + At::kWs + a * 256, s_off + a * 16 * kb, uniform(k0 / 32));
    dma4(t.xs, lds + At::kXs, s_off, uniform(k0 / 32));
  };

  // The rows' strides are often a power of two, and a window of all rows then lies in a few channels of the
  // caches and the memory: workgroups begin at different windows, or all would use the same ones at a time.
  const int windows = (p.k + kWin - 1) / kWin, turn = static_cast<int>(blockIdx.x / kXcds) % windows;
  const auto window = [&](int v) { return (v + turn >= windows ? v + turn - windows : v + turn) * kWin; };
  FewPass next;
  bool more = next_pass(next);
  if (more && wave < windows) load(next, window(wave));
  while (more) {
    const int c0 = next.c0, cnt = next.cnt, row0 = next.row0, rows = next.rows;
    f32x4_t acc[NI];
#pragma unroll
    for (int a = 0; a < NI; ++a) acc[a] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    int v = wave;
    do {
      const int deep = v < windows ? (p.k - window(v)) >> 7 : 0;  // instructions of the window that lie within k (a multiple of 128)
      i32x4_t wf[NI][4], xf[4][XB / 4];
      uint32_t ws[NI][4], xs[4];
      __builtin_amdgcn_sched_barrier(0);
      wait_vm<0>();
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // scales past k are another row's, which might be NaN: extracted with a width of 0
        const uint32_t width = i < deep ? 8 : 0;
#pragma unroll
        for (int a = 0; a < NI; ++a) {
          wf[a][i] = WRows::read(mine, a * 16 + r16, i * 4 + q);
          ws[a][i] = __builtin_amdgcn_ubfe(reinterpret_cast<const uint32_t*>(mine + At::kWs)[(a * 16 + r16) * 4 + i],
                                           8 * q, width);
        }
#pragma unroll
        for (int h = 0; h < XB / 4; ++h) xf[i][h] = XRows::read(mine + At::kX, r16, (i * (XB / 4) + h) * 4 + q);
        xs[i] = __builtin_amdgcn_ubfe(reinterpret_cast<const uint32_t*>(mine + At::kXs)[r16 * 4 + i], 8 * q, width);
      }
      wait_lds();
      __builtin_amdgcn_sched_barrier(0);
      const bool any = v < windows;  // a wave without a window has nothing in LDS
      v += 4;
      if (v < windows) {
        load(next, window(v));
      } else {
        more = next_pass(next);
        if (more && wave < windows) load(next, window(wave));
      }
      __builtin_amdgcn_sched_barrier(0);
      if (any) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          i32x8_t w[NI];
          uint32_t s[NI];
#pragma unroll
          for (int a = 0; a < NI; ++a) w[a] = operand(wf[a][i]), s[a] = ws[a][i];
          mma_columns<XB>(w, operand(xf[i]), acc, s, xs[i]);
        }
      }
    } while (v < windows);

    // barriers for LDS alone: the loads stay on their way
    const auto barrier = [] {
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    };
    barrier();  // the last pass's sums are read
#pragma unroll
    for (int a = 0; a < NI; ++a)
      *reinterpret_cast<f32x4_t*>(&s_red[wave][r16 * (16 * NI) + a * 16 + q * 4]) = acc[a];
    barrier();
    const int r = threadIdx.x >> 4, c = (threadIdx.x & 15) * 2;
    if (r < rows && c0 * 16 + c < p.n && c < cnt * 16) {
      const float* sum = &s_red[0][r * (16 * NI) + c];
      float v0 = sum[0], v1 = sum[1];
#pragma unroll
      for (int w = 1; w < 4; ++w) {
        v0 += sum[w * (16 * 16 * NI)];
        v1 += sum[w * (16 * 16 * NI) + 1];
      }
      const long long o = static_cast<long long>(row0 + r) * p.n + c0 * 16 + c;
      if (p.out_f32)
        *reinterpret_cast<float2*>(static_cast<float*>(p.out) + o) = make_float2(v0, v1);
      else
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + o) = pack_bf16x2(v0, v1);
    }
  }
  zero_other_rows<kThreads>(p, win);
}

// ---------------------------------------------------------------- many rows a group

// Tiles of up to 128 rows of a group by 128 columns, four waves, two
// workgroups a CU, each of which fills the gaps that the other's barriers,
// first loads and stores leave.  Both operands of a window lie in a ring of LDS
// stages; all but the one being multiplied are on their way.  A tile with more
// than 64 rows gives each wave 64 x 64 outputs (8-bit x: 32 x 128) and is bound by the
// loads into its CU (8192 rows of one group, 2048 x 4096, 4-bit x: 55 us, 2.5 PFLOP/s).
// One with fewer gives it all rows and 32 columns (8-bit x: 16 rows and more
// columns), its stages are smaller and there are
// more of them, so that a tile of a small group is a stream of its weights:
// decode takes 60 us for 300 MB, 5.0 TB/s.
constexpr int kTileM = 128, kTileN = 128, kTileThreads = 256, kTileWaves = 4;
// Workgroups a CU, and LDS for the ring: the share of the CU's 160 KB less the bounds of up to MAXL groups.
template <int MAXL>
constexpr int kTileWgs = MAXL <= 512 ? 2 : 1;
template <int MAXL>
constexpr int kRingBytes = (160 / kTileWgs<MAXL> * 1024 - 2 * (MAXL + 1) * 4 - 256) / 1024 * 1024;

struct TileAt {
  int j, row0, rows, n0;  // group, first row and rows, first column
  bool once;              // the group's only row block: no other tile reads its weights
};

// One tile with at most MW * MI * 16 rows: MW x (4 / MW) waves of 16 MI rows x 16 NI columns, windows S
// instructions deep.  S = 2 takes 128-byte pieces of the weights' rows; 8-bit x of 128 rows leaves room for S = 1.
template <int XB, int RING, int S, int MW, int MI, int NI>
__device__ __forceinline__ void mx_tile(const MxArgs& p, const TileAt& t, char* s_ops) {
  constexpr int W = 128 * S;  // elements deep a window is
  constexpr int kRows = MW * MI * 16, kXRow = W * XB / 8, kWRow = W / 2;
  static_assert((kTileWaves / MW) * NI * 16 == kTileN, "the waves cover the columns");
  typedef Rows<kXRow / 16> XRows;
  typedef Rows<kWRow / 16> WRows;
  // a stage: weights and x; a piece of the scales, two in turn: 16 bytes a column and row, for SP windows (the
  // 4 S bytes of one window would be fetched from as many cache lines)
  constexpr int kX = kTileN * kWRow, kStage = kX + kRows * kXRow;
  constexpr int SP = 512 / W, kXs = kTileN * 16, kPiece = kXs + kRows * 16;
  constexpr int kFit = (RING - 2 * kPiece) / kStage, NS = kFit < SP + 1 ? kFit : SP + 1;  // SP > NS - 2: see the waits
  static_assert(NS >= 2, "a stage to multiply and one on its way");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
  const int m_off = (wave % MW) * MI * 16, n_off = (wave / MW) * NI * 16;
  const int kb = p.k / 32, xbytes = p.k * XB / 8, wbytes = p.k / 2;
  const long long col0 = static_cast<long long>(t.j) * p.n + t.n0;
  const int cols = min(kTileN, p.n - t.n0);
  const u32x4_t rw = rows_of(p.w, col0, cols, wbytes), rws = rows_of(p.ws, col0, cols, kb);
  const u32x4_t rx = rows_of(p.x, t.row0, t.rows, xbytes), rxs = rows_of(p.xs, t.row0, t.rows, kb);
  const uint32_t lds = lds_address(s_ops);
  // Every wave loads 32 columns of the weights and a part of the rest, as many loads as the others: where there
  // is less than one load for each, some load the same bytes to the same place.
  constexpr int kXAll = kRows / XRows::kPerLoad, kXLoads = kXAll > kTileWaves ? kXAll / kTileWaves : 1;
  constexpr int kWLoads = 32 / WRows::kPerLoad, L = kWLoads + kXLoads;
  constexpr int kXsAll = kRows / 16, kXsLoads = kXsAll > kTileWaves ? kXsAll / kTileWaves : 1;  // 16 rows a load
  RowLoads<kXRow / 16, kXLoads> x_loads;
  RowLoads<kWRow / 16, kWLoads> w_loads;
  const int x_row = wave % (kXAll / kXLoads) * (kXLoads * XRows::kPerLoad), w_row = wave * 32;
  x_loads.init(x_row, xbytes);
  w_loads.init(w_row, wbytes);
  const int xs_row = wave % (kXsAll / kXsLoads) * (kXsLoads * 16);
  const uint32_t s_off = static_cast<uint32_t>(lane / 4) * kb + (lane & 3) * 4;
  const int nk = (p.k + W - 1) / W;
  const auto load = [&](int kt, int slot) {
    const uint32_t stage = lds + slot * kStage;
    // past the caches that hold x: decode with 8-bit x in one part, 62 us without, 56 with (whole cache lines only)
    if (S >= 2 && t.once)
      w_loads.template issue<true>(rw, stage + w_row * kWRow, wbytes, kt * kWRow);
    else
      w_loads.issue(rw, stage + w_row * kWRow, wbytes, kt * kWRow);
    x_loads.issue(rx, stage + kX + x_row * kXRow, xbytes, kt * kXRow);
  };
  const uint32_t pieces = lds + NS * kStage;
  const auto load_scales = [&](int piece) {
    const uint32_t at = pieces + (piece & 1) * kPiece;
#pragma unroll
    for (int s = 0; s < 2; ++s)
      dma4(rws, at + (w_row + 16 * s) * 16, s_off + static_cast<uint32_t>(w_row + 16 * s) * kb, uniform(piece * 16));
#pragma unroll
    for (int s = 0; s < kXsLoads; ++s)
      dma4(rxs, at + kXs + (xs_row + 16 * s) * 16, s_off + static_cast<uint32_t>(xs_row + 16 * s) * kb,
           uniform(piece * 16));
  };

  f32x4_t acc[MI][NI];
#pragma unroll
  for (int b = 0; b < MI; ++b)
#pragma unroll
    for (int a = 0; a < NI; ++a) acc[b][a] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  struct RowBlock {
    i32x4_t x[S][XB / 4];
    uint32_t xs[S];
  };
  const auto read_rows = [&](const char* stage, const uint32_t* scales, int b, RowBlock& f) {
    const int row = m_off + b * 16 + r16;
#pragma unroll
    for (int i = 0; i < S; ++i) {
#pragma unroll
      for (int h = 0; h < XB / 4; ++h) f.x[i][h] = XRows::read(stage + kX, row, (i * (XB / 4) + h) * 4 + q);
      f.xs[i] = scales[(kTileN + row) * 4 + i];
    }
  };
  __builtin_amdgcn_s_barrier();  // the last tile's readers are done
  load_scales(0);
#pragma unroll
  for (int s = 0; s < NS - 1; ++s)
    if (s < nk) load(s, s);
  int slot = 0;
  for (int kt = 0; kt < nk; ++kt) {
    __builtin_amdgcn_sched_barrier(0);
    wait_ladder<L, NS - 2>(min(nk - 1 - kt, NS - 2));
    __builtin_amdgcn_s_barrier();  // this window is in LDS, and every wave is done with the one before
    __builtin_amdgcn_sched_barrier(0);
    const char* stage = s_ops + slot * kStage;
    const uint32_t* scales =
        reinterpret_cast<const uint32_t*>(s_ops + NS * kStage + (kt / SP & 1) * kPiece) + kt % SP * S;
    // the next piece of the scales first: the waits below count the loads of windows, and are at most too long
    if (kt % SP == 0 && kt + SP < nk) load_scales(kt / SP + 1);
    if (kt + NS - 1 < nk) load(kt + NS - 1, slot == 0 ? NS - 1 : slot - 1);
    slot = slot + 1 == NS ? 0 : slot + 1;
    __builtin_amdgcn_sched_barrier(0);
    // scales past k are another row's, which might be NaN: their bytes are extracted with a width of 0
    const int deep = (p.k - kt * W) >> 7;
    uint32_t width[S];
#pragma unroll
    for (int i = 0; i < S; ++i) width[i] = i < deep ? 8 : 0;
    i32x8_t w[S][NI];
    uint32_t ws[S][NI];
#pragma unroll
    for (int a = 0; a < NI; ++a)
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const int col = n_off + a * 16 + r16;
        w[i][a] = operand(WRows::read(stage, col, i * 4 + q));
        ws[i][a] = __builtin_amdgcn_ubfe(scales[col * 4 + i], 8 * q, width[i]);
      }
    RowBlock f[2];
    read_rows(stage, scales, 0, f[0]);
#pragma unroll
    for (int b = 0; b < MI; ++b) {  // the next row block is read while this one is multiplied
      if (b + 1 < MI) read_rows(stage, scales, b + 1, f[(b + 1) & 1]);
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const uint32_t xs = __builtin_amdgcn_ubfe(f[b & 1].xs[i], 8 * q, width[i]);
        mma_columns<XB>(w[i], operand(f[b & 1].x[i]), acc[b], ws[i], xs);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if (p.out_f32) {
#pragma unroll
    for (int b = 0; b < MI; ++b) {
      const int r = m_off + b * 16 + r16;
      if (r >= t.rows) continue;
#pragma unroll
      for (int a = 0; a < NI; ++a) {
        const int c = t.n0 + n_off + a * 16 + q * 4;
        if (c < p.n)
          *reinterpret_cast<f32x4_t*>(static_cast<float*>(p.out) + static_cast<long long>(t.row0 + r) * p.n + c) =
              acc[b][a];
      }
    }
    return;
  }
  // bf16: through LDS, so that a store writes whole rows of the wave's 16 NI columns instead of 8 bytes a lane
  constexpr int kPer = 2 * NI, kLd = 16 * NI + 8;  // 16-byte chunks a row; halves a row, padded
  static_assert(MI * 16 * kLd * 2 * kTileWaves <= RING, "the outputs fit into the ring");
  __builtin_amdgcn_s_barrier();  // every wave is done with the ring
  uint16_t* mine = reinterpret_cast<uint16_t*>(s_ops) + wave * (MI * 16 * kLd);
#pragma unroll
  for (int b = 0; b < MI; ++b)
#pragma unroll
    for (int a = 0; a < NI; ++a)
      *reinterpret_cast<uint2*>(mine + (b * 16 + r16) * kLd + a * 16 + q * 4) =
          make_uint2(pack_bf16x2(acc[b][a][0], acc[b][a][1]), pack_bf16x2(acc[b][a][2], acc[b][a][3]));
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int i = 0; i < MI * 16 * kPer / 64; ++i) {
    const int at = i * 64 + lane, r = m_off + at / kPer, c = t.n0 + n_off + at % kPer * 8;
    if (r < t.rows && c < p.n)  // n is a multiple of 8
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + static_cast<long long>(t.row0 + r) * p.n + c) =
          *reinterpret_cast<const uint4*>(mine + at / kPer * kLd + at % kPer * 8);
  }
}

// The (group, strip) pairs are dealt round over the XCDs, and the row blocks of
// a pair, which share its weights, follow each other on one XCD: its L2 then
// reads the weights once (dealt over the XCDs, eight L2s read them, and what lies
// behind the L2s set the time).  They also read a window at about the same time:
// starting the workgroups at different windows, to spread rows of a power-of-two
// stride over the channels, cost up to 25 %.
//
// What bounds it now is what is read past the L2s: the up-projection (8192 rows
// over 64 Zipf groups of 2048 x 4096) with 4-bit x reads 501 MB there, of which the
// weights are 285 and x comes once for every XCD that has a strip, in 96 us (5.2
// TB/s), and as much again from the L2s; with 8-bit x 790 MB in 173 us, where
// the second instruction and the split add to the loads, since a stage or two is
// all that is on its way.  Other orders of the tiles do not change that: groups
// with the most rows first, large tiles before small ones, or one of each on
// every CU gained nothing there and lost where groups are of one size.
template <int XB, int MAXL>
__global__ __launch_bounds__(kTileThreads, kTileWgs<MAXL>) void ragged_dot_mx_tile(MxArgs p) {
  constexpr int RING = kRingBytes<MAXL>;
  __shared__ __attribute__((aligned(1024))) char s_ops[RING];
  __shared__ int s_lb[MAXL + 1];
  __shared__ int s_tiles[MAXL + 1];  // this XCD's tiles before each group
  __shared__ long long s_wave[kTileWaves];
  const Window win = build_local_bounds<kTileThreads>(p.gs, p.G, p.offp, p.gl, p.limp, p.m, s_lb, s_wave);
  const int strips = row_blocks(p.n, kTileN);
  const int xcd = blockIdx.x % kXcds, step = gridDim.x / kXcds;  // the grid is a multiple of kXcds
  // strips of group j on this XCD: s with (j * strips + s) % kXcds == xcd
  const auto first_strip = [&](int j) { return static_cast<int>((xcd + kXcds - (static_cast<long long>(j) * strips) % kXcds) % kXcds); };
  const auto strips_here = [&](int j) { return (strips - first_strip(j) + kXcds - 1) / kXcds; };
  {
    constexpr int PER = (MAXL + kTileThreads) / kTileThreads;
    int c[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int j = PER * threadIdx.x + i;
      c[i] = j < p.gl ? row_blocks(s_lb[j + 1] - s_lb[j], kTileM) * strips_here(j) : 0;
      sum += c[i];
    }
    int run = static_cast<int>(block_excl_scan<kTileThreads>(sum, s_wave));
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int j = PER * threadIdx.x + i;
      if (j <= p.gl) s_tiles[j] = run;
      run += c[i];
    }
    __syncthreads();
  }
  const int total = s_tiles[p.gl];
  for (int tile = blockIdx.x / kXcds; tile < total; tile += step) {
    TileAt t;
    t.j = __builtin_amdgcn_readfirstlane(upper_index(s_tiles, p.gl, tile));
    const int lb = __builtin_amdgcn_readfirstlane(s_lb[t.j]), ub = __builtin_amdgcn_readfirstlane(s_lb[t.j + 1]);
    const int mts = row_blocks(ub - lb, kTileM);
    const int local = tile - __builtin_amdgcn_readfirstlane(s_tiles[t.j]);
    const int unit = local / mts;
    t.once = mts == 1;
    t.row0 = lb + (local - unit * mts) * kTileM;
    t.rows = min(kTileM, ub - t.row0);
    t.n0 = (first_strip(t.j) + unit * kXcds) * kTileN;
    if constexpr (XB == 4) {
      if (t.rows > 64)
        mx_tile<XB, RING, 2, 2, 4, 4>(p, t, s_ops);
      else if (t.rows > 32)
        mx_tile<XB, RING, 2, 1, 4, 2>(p, t, s_ops);
      else if (t.rows > 16)
        mx_tile<XB, RING, 2, 1, 2, 2>(p, t, s_ops);
      else
        mx_tile<XB, RING, 2, 1, 1, 2>(p, t, s_ops);
    } else {  // fewer rows and more columns a wave, since a wave splits its rows: up to 1.24x faster than as above
      if (t.rows > 64)
        mx_tile<XB, RING, 1, 4, 2, 8>(p, t, s_ops);
      else if (t.rows > 32)
        mx_tile<XB, RING, 2, 4, 1, 8>(p, t, s_ops);
      else if (t.rows > 16)
        mx_tile<XB, RING, 2, 2, 1, 4>(p, t, s_ops);
      else
        mx_tile<XB, RING, 2, 1, 1, 2>(p, t, s_ops);
    }
  }
  zero_other_rows<kTileThreads>(p, win);
}

template <int XB>
void launch_mx(const MxArgs& a, hipStream_t stream) {
  const long long cus = device_cu_count();
  const long long strips = row_blocks(a.n, kTileN);
  if (a.m <= static_cast<long long>(kFewRows) * a.gl && a.gl * strips <= kFewTiles) {
    const long long passes = ((row_blocks(a.m, 16) + a.gl) * ((a.n + 15ll) / 16) + kFewN - 1) / kFewN;
    const int grid = static_cast<int>(passes < cus * 2 ? passes : cus * 2);
    ragged_dot_mx_few<XB><<<grid, kThreads, 0, stream>>>(a);
    return;
  }
  const long long tiles = (row_blocks(a.m, kTileM) + a.gl) * strips;
  const auto grid = [&](long long wgs) {
    const long long most = cus * wgs / kXcds * kXcds, want = tiles < most ? (tiles + kXcds - 1) / kXcds * kXcds : most;
    return static_cast<int>(want > 0 ? want : kXcds);
  };
  if (a.gl <= 512)
    ragged_dot_mx_tile<XB, 512><<<grid(kTileWgs<512>), kTileThreads, 0, stream>>>(a);
  else
    ragged_dot_mx_tile<XB, RD_MAX_GROUPS><<<grid(kTileWgs<RD_MAX_GROUPS>), kTileThreads, 0, stream>>>(a);
}

}  // namespace

int launch_forward_mx(const GemmProblem& p, const uint8_t* x_scales, const uint8_t* w_scales, int x_bits,
                      hipStream_t stream) {
  MxArgs a{};
  a.x = static_cast<const uint8_t*>(p.a);
  a.xs = x_scales;
  a.w = static_cast<const uint8_t*>(p.b);
  a.ws = w_scales;
  a.gs = p.group_sizes;
  a.offp = p.group_offset;
  a.limp = p.limit;
  a.out = p.out;
  a.G = p.num_groups;
  a.gl = p.num_local;
  a.m = p.m;
  a.k = p.k;
  a.n = p.n;
  a.out_f32 = p.out_f32;
  if (x_bits == 4)
    launch_mx<4>(a, stream);
  else
    launch_mx<8>(a, stream);
  return hipGetLastError() == hipSuccess ? RD_OK : RD_EHIP;
}

}  // namespace rd
