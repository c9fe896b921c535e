// Residual addition and root-mean-square norm for sm_103a, with the MXFP8 copy
// of the result that the block-scaled GEMMs read, and their gradient.
//
//   h = x + r,  rstd = (mean_K h^2 + eps)^(-1/2),  y = h rstd w
//
// The sum and its square mean are held in fp32; h and y are rounded to bf16
// once, each from its fp32 value.  The 8-bit output is the quantisation of the
// bf16 y, not of its fp32 value, so that it holds the bytes mpm_mxfp8_quantize
// makes of y: a rollout that reads these codes and a training step that
// quantises the stored y then run on the same operands.
//
// A row is held in the registers of the threads of one block, or of one warp, so
// every operand is read once.
#include <algorithm>
#include <atomic>
#include "norm.cuh"
#include "launch.cuh"
#include "mxfp8.cuh"
#include "packed.cuh"

namespace mpm {

constexpr int kNormMaxThreads = 512;
constexpr int kNormMaxWarps = kNormMaxThreads / 32;
constexpr int kNormTeams = 4;            // rows of one warp each in a block
constexpr int kRingStages = 8;           // most stages of the backward's ring
constexpr int kRingWords = 2;            // 16-byte words of each operand a thread takes there

MPM_DEV uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// VEC consecutive bf16 as loaded: pairs, or one in the low half
template <int VEC>
struct RawBf16 {
  static constexpr int W = (VEC + 1) / 2;
  uint32_t w[W];
  MPM_DEV void load(const uint16_t* p) {
    if constexpr (VEC == 8) {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    } else {
      w[0] = *p;
    }
  }
  MPM_DEV void zero() {
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = 0;
  }
  MPM_DEV float value(int j) const { return (j & 1) ? bf16hi(w[j / 2]) : bf16lo(w[j / 2]); }
  MPM_DEV void set(const float (&v)[VEC]) {
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = pack_bf16(v[2 * j], 2 * j + 1 < VEC ? v[2 * j + 1] : 0.0f);
  }
  MPM_DEV void store(uint16_t* p) const {
    if constexpr (VEC == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *p = (uint16_t)w[0];
  }
};

MPM_DEV float bf16_f(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// What a vector is computed in: pairs of fp32 (VEC = 8), or one
template <int VEC>
struct Lanes {
  using T = uint64_t;
  static constexpr int N = VEC / 2;
  static MPM_DEV T widen(uint32_t w) { return widen2(w); }
  static MPM_DEV T splat(float v) { return f32x2(v, v); }
  static MPM_DEV T pick(const float (&v)[VEC], int j) { return f32x2(v[2 * j], v[2 * j + 1]); }
  static MPM_DEV T add(T a, T b) { return add2(a, b); }
  static MPM_DEV T mul(T a, T b) { return mul_f32x2(a, b); }
  static MPM_DEV T fma(T a, T b, T c) { return fma2(a, b, c); }
  static MPM_DEV float sum(T v) { float lo, hi; f32x2_split(v, lo, hi); return __fadd_rn(lo, hi); }
  static MPM_DEV uint32_t bf16(T v) { float lo, hi; f32x2_split(v, lo, hi); return pack_bf16(lo, hi); }
};
template <>
struct Lanes<1> {
  using T = float;
  static constexpr int N = 1;
  static MPM_DEV T widen(uint32_t w) { return bf16lo(w); }
  static MPM_DEV T splat(float v) { return v; }
  static MPM_DEV T pick(const float (&v)[1], int) { return v[0]; }
  static MPM_DEV T add(T a, T b) { return __fadd_rn(a, b); }
  static MPM_DEV T mul(T a, T b) { return __fmul_rn(a, b); }
  static MPM_DEV T fma(T a, T b, T c) { return __fmaf_rn(a, b, c); }
  static MPM_DEV float sum(T v) { return v; }
  static MPM_DEV uint32_t bf16(T v) { return pack_bf16(v, 0.0f); }
};

template <int VEC>
MPM_DEV void load_weight(const void* w, int f32, int k, float (&v)[VEC]) {
  if (f32) {
    const float* p = static_cast<const float*>(w) + k;
    if constexpr (VEC == 8) {
      const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      v[0] = *p;
    }
  } else {
    RawBf16<VEC> r;
    r.load(static_cast<const uint16_t*>(w) + k);
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = r.value(j);
  }
}

// Rows that start anywhere are taken by the aligned words of 8 that they touch:
// where a row starts `off` columns into a word, word v holds columns 8 v - off
// and on, and the words at its ends have columns outside [0, K).  (Forward at
// 22524 x 4161: 146 us; by single elements 213, bound by their instructions.)
MPM_DEV int word_offset(const uint16_t* row) { return (int)(reinterpret_cast<uintptr_t>(row) & 15) >> 1; }
MPM_DEV bool whole_word(int k, int K) { return k >= 0 && k + 8 <= K; }

// Columns k .. k + VEC - 1 of a row, zero outside [0, K); OFF: k is one of a
// word as above, else K is a multiple of VEC
template <int VEC, bool OFF>
MPM_DEV void load_columns(RawBf16<VEC>& v, const uint16_t* row, int k, int K) {
  if constexpr (!OFF) {
    if (k < K) v.load(row + k);
  } else {
    if (whole_word(k, K)) {
      v.load(row + k);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if ((unsigned)(k + j) < (unsigned)K) v.w[j / 2] |= (uint32_t)row[k + j] << (j % 2 * 16);
    }
  }
}
template <int VEC, bool OFF>
MPM_DEV void store_columns(const RawBf16<VEC>& v, uint16_t* row, int k, int K) {
  if constexpr (!OFF) {
    if (k < K) v.store(row + k);
  } else {
    if (whole_word(k, K)) {
      v.store(row + k);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if ((unsigned)(k + j) < (unsigned)K) row[k + j] = (uint16_t)(v.w[j / 2] >> (j % 2 * 16));
    }
  }
}
// the weight's, zero outside; OFF: from any alignment
template <int VEC, bool OFF>
MPM_DEV void load_weight_columns(const void* w, int f32, int k, int K, float (&v)[VEC]) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) v[j] = 0.0f;
  if constexpr (!OFF) {
    if (k < K) load_weight<VEC>(w, f32, k, v);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if ((unsigned)(k + j) < (unsigned)K)
        v[j] = f32 ? static_cast<const float*>(w)[k + j] : bf16_f(static_cast<const uint16_t*>(w)[k + j]);
  }
}

// The threads that share a row: a block, or (WARP, rows short enough) a warp of
// a block of kNormTeams
template <bool WARP>
struct RowTeam {
  int t, nt;
  long long index;                       // of the grid's teams
  MPM_DEV RowTeam() {
    t = WARP ? threadIdx.x & 31 : threadIdx.x;
    nt = WARP ? 32 : blockDim.x;
    index = WARP ? (long long)blockIdx.x * kNormTeams + (threadIdx.x >> 5) : blockIdx.x;
  }
};

// R sums over a row's threads, in a fixed order; every thread gets them
template <bool WARP, int R>
MPM_DEV void row_sums(float (&v)[R], float (*sh)[kNormMaxWarps]) {
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[r] = __fadd_rn(v[r], __shfl_xor_sync(0xFFFFFFFFu, v[r], o));
  if constexpr (WARP) return;
  const int nw = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (lane == 0) sh[r][warp] = v[r];
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    v[r] = 0.0f;
    for (int i = 0; i < nw; ++i) v[r] = __fadd_rn(v[r], sh[r][i]);
  }
}

// Sum over the block's threads where every thread also says whether its wait
// went well; false if any did not.  sh: the caller
// alternates between two, so one barrier a call suffices.
MPM_DEV bool block_sum_ok(float& v, float* sh, bool ok) {
  const int nw = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  if (lane == 0) sh[warp] = v;
  if (__syncthreads_or(!ok)) return false;
  v = lane < nw ? sh[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return true;
}

// A ring of S stages whose copies are waited for in order; the place of row
// number `it` of a block
struct RingCursor {
  int s = 0;
  uint32_t phase = 0;
  MPM_DEV void next(int S) { if (++s == S) { s = 0; phase ^= 1; } }
  // lets the copies of the rows after a failed wait land (bounded), from thread 0
  MPM_DEV void drain(uint32_t bar0, int S, int outstanding, long long row, long long step, long long M) {
    for (int j = 0; j < outstanding && row < M; ++j, row += step) {
      mbar_wait(bar0 + 8 * s, phase, nullptr);
      next(S);
    }
  }
};

// VEC consecutive elements per load, IT loads per thread and operand, R rows per
// team, all their loads in flight together.  Bound by the bytes: with a residual
// and the 8-bit copy 9 + 1/32 bytes an element (x, r in; y, h, codes and scales
// out).  16384 x 2048 takes 46.0 us and 32768 x 7168 takes 306.7 us, 6.6 and 6.9
// TB/s.  The arithmetic is nearly as long as the copies, hence pairs of fp32:
// with single ones and 8 columns a thread the two took 48.6 and 315 us (16
// columns a thread alone: 47.6 and 312).
template <int VEC, int IT, int R, bool WARP, bool OFF>
__global__ void __launch_bounds__(WARP ? 32 * kNormTeams : kNormMaxThreads) add_rmsnorm_kernel(const NormFwd p) {
  using L = Lanes<VEC>;
  using T = typename L::T;
  __shared__ float sh[R][kNormMaxWarps];
  pdl_wait();
  pdl_launch_dependents();
  const RowTeam<WARP> team;
  const int t = team.t, nt = team.nt;
  const long long row0 = team.index * R;
  RawBf16<VEC> x[R][IT], res[R][IT];
  int off[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint16_t* px = p.x + (row0 + r) * p.ldx;
    const uint16_t* pr = p.r + (row0 + r) * p.ldr;
    off[r] = OFF ? word_offset(px) : 0;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int k = (i * nt + t) * VEC - off[r];
      x[r][i].zero();
      res[r][i].zero();
      if (row0 + r < p.M) {
        load_columns<VEC, OFF>(x[r][i], px, k, p.K);
        if (p.r) load_columns<VEC, OFF>(res[r][i], pr, k, p.K);
      }
    }
  }
  T h[R][IT][L::N];
  float ss[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    T s2 = L::splat(0.0f);
#pragma unroll
    for (int i = 0; i < IT; ++i)
#pragma unroll
      for (int j = 0; j < L::N; ++j) {
        // x + 0 is x: no branch on whether there is a residual
        h[r][i][j] = L::add(L::widen(x[r][i].w[j]), L::widen(res[r][i].w[j]));
        s2 = L::fma(h[r][i][j], h[r][i][j], s2);
      }
    ss[r] = L::sum(s2);
  }
  row_sums<WARP, R>(ss, sh);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    ss[r] = rsqrtf(__fmaf_rn(ss[r], p.rk, p.eps));
    if (t == 0 && p.rstd && row0 + r < p.M) p.rstd[row0 + r] = ss[r];
  }
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    T w[L::N];
    auto weight = [&](int k) {
      float v[VEC];
      load_weight_columns<VEC, OFF>(p.w, p.w_f32, k, p.K, v);
#pragma unroll
      for (int j = 0; j < L::N; ++j) w[j] = L::pick(v, j);
    };
    if (!OFF) weight((i * nt + t) * VEC);          // the same for all rows
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long row = row0 + r;
      const int k = (i * nt + t) * VEC - off[r];
      if (OFF) weight(k);
      const bool live = k < p.K && row < p.M;
      const T rstd = L::splat(ss[r]);
      RawBf16<VEC> oh, o;
#pragma unroll
      for (int j = 0; j < L::N; ++j) {
        oh.w[j] = L::bf16(h[r][i][j]);
        o.w[j] = L::bf16(L::mul(L::mul(h[r][i][j], rstd), w[j]));
      }
      if (p.h && live) store_columns<VEC, OFF>(oh, p.h + row * p.ldh, k, p.K);
      if (p.y && live) store_columns<VEC, OFF>(o, p.y + row * p.ldy, k, p.K);
      if (OFF || !p.q) continue;
      // K % 32 == 0: a block of 32 lies in 32 / VEC neighbouring lanes.  The
      // quantiser's maximum, also of NaN: over the even columns and over the odd
      // ones, where a number passes over a NaN, then of the two by their bits.
      uint32_t m;
      if constexpr (VEC == 8) {
        m = absmax_bf16x2_halves(o.w);
#pragma unroll
        for (int d = 2; d > 0; d >>= 1) m = max_bf16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
        m = larger_half(m);
      } else {
        constexpr uint32_t kEven = 0x55555555u;
        m = o.w[0] & 0x7FFFu;
        const uint32_t nan = __ballot_sync(0xFFFFFFFFu, m > 0x7F80u);
        m = __reduce_max_sync(0xFFFFFFFFu, m > 0x7F80u ? 0u : m);
        if ((nan & kEven) == kEven || (nan & ~kEven) == ~kEven) m = 0x7FFFu;
      }
      const int e = mx_exponent(m << 16);
      if (!live) continue;
      const uint64_t sc = f32x2_splat(pow2_neg(e));
      uint8_t* dst = p.q + row * (long long)p.K + k;
      if constexpr (VEC == 8) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(e4m3x2_scaled(o.w[0], sc) | (e4m3x2_scaled(o.w[1], sc) << 16),
                                                    e4m3x2_scaled(o.w[2], sc) | (e4m3x2_scaled(o.w[3], sc) << 16));
      } else {
        *dst = (uint8_t)e4m3x2_scaled(o.w[0], sc);
      }
      if (k % 32 == 0) p.s[sf_offset(row, k >> 5, p.s_cols_pad)] = (uint8_t)(e + 127);
    }
  }
  if (OFF || !p.q) return;
  // zero the padding of the scale tiles: past K, and rows past M
  const int nblk = p.K >> 5;
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (row0 + r < (p.M + 127) / 128 * 128)
      for (int c = (row0 + r < p.M ? nblk : 0) + t; c < (int)p.s_cols_pad; c += nt)
        p.s[sf_offset(row0 + r, c, p.s_cols_pad)] = 0;
}

// ---------------------------------------------------------------- backward
// With xh = h rstd and g = dy w:
//   dx = rstd (g - xh mean_K(g xh)) + dh,   dw = sum over rows of dy xh,
// computed from u = dy rstd as t = u w, c = sum_K t h,
//   dx = t - h (rstd^2 c / K) + dh,         dw += u h.
// Blocks walk rows blockIdx.x, blockIdx.x + gridDim.x, ...; each keeps its
// columns' share of dw in fp32 registers and writes it to its row of the
// workspace, which a second kernel sums in a fixed order (no atomics: the same
// bytes every time).

// What bounds a thread's registers: 512 threads, but with two operands alone the
// compiler then takes 97, one too many for two blocks of 320 (4000 x 4480: 33.8
// against 22.9 us, 8192 x 2048: 22.3 against 21.2)
constexpr int ring_most_threads(int c, bool more) { return more ? 1024 / c : 640; }

// Rows of 16-byte aligned operands stream through a ring of S stages in shared
// memory, one row's operands each, by bulk copies that thread 0 issues: S - 1
// rows are in flight whatever the threads are doing.  A thread takes C words of
// 8 columns.  A stage is refilled after the block barrier of the next row's
// reduction, by when every thread is past its last read of it.
//
// Bound by the bytes, 8 an element with dh, 10 with dy2 too: 8192 x 2048 with
// both takes 30.1 us, the sum of the partials included (floor 24.8), 4093 x 1544
// with dh 14.5 (7.5).  Rows held in registers with one in flight took
// 89.6 and 45.6; one block of 1024 threads an SM in teams, 31.1 and 17.4.
//
// OFF: rows that start anywhere, by their words.  A block's rows start at one
// place of a word (the blocks are a multiple of 8, or have one row each), so its
// threads keep their columns (8000 x 1003 takes 19.4 us, 43 by single elements).
// A copy takes whole words, and with them a few
// elements of the rows beside it, which are masked; at the ends of the operand,
// where there may be nothing beside it, it takes the row's own elements.
template <int C, bool TWO, bool RES, bool OFF>
__global__ void __launch_bounds__(ring_most_threads(C, TWO || RES || OFF)) add_rmsnorm_bwd_ring_kernel(const NormBwd p, int S) {
  constexpr int NT = 2 + (TWO ? 1 : 0) + (RES ? 1 : 0);
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float sh[2][32];
  __shared__ __align__(8) uint64_t bars[kRingStages];
  const int t = threadIdx.x, nt = blockDim.x;
  const int off = OFF ? word_offset(p.dy + blockIdx.x * p.lddy) : 0;
  const int end = off + p.K;                               // in elements of the row's words
  const uint32_t row_bytes = OFF ? (uint32_t)(end + 7) / 8 * 16 : (uint32_t)p.K * 2;
  const uint32_t stage_bytes = NT * row_bytes;
  const uint32_t base = smem_u32(ring), bar0 = smem_u32(bars);
  if (t == 0) {
    for (int s = 0; s < S; ++s) mbar_init(bar0 + 8 * s, 1);
    fence_mbar_init();
    fence_proxy_async();
  }
  pdl_wait();
  auto issue = [&](long long row, int s) {
    const uint32_t bar = bar0 + 8 * s;
    uint32_t lo = 0, hi = row_bytes;                       // of the words, what is copied whole
    if (OFF) {
      if (row == 0 && off > 0) lo = 16;
      if (row == p.M - 1 && end % 8 != 0) hi -= 16;
    }
    auto copy = [&](int operand, const uint16_t* src) {
      const uint32_t to = s * stage_bytes + operand * row_bytes;
      if (OFF && hi - lo != row_bytes) {
        uint16_t* dst = reinterpret_cast<uint16_t*>(ring + to);
        for (int j = off; j < (int)lo / 2; ++j) dst[j] = src[j - off];
        for (int j = (int)hi / 2; j < end; ++j) dst[j] = src[j - off];
        fence_proxy_async();                               // before a later copy over them
      }
      return base + to;
    };
    const uint16_t* src[NT];
    src[0] = p.dy + row * p.lddy;
    src[1] = p.h + row * p.ldh;
    if (TWO) src[2] = p.dy2 + row * p.lddy2;
    if (RES) src[NT - 1] = p.dh + row * p.lddh;
    uint32_t dst[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) dst[i] = copy(i, src[i]);
    mbar_arrive_expect_tx(bar, NT * (hi - lo));            // releases the elements above
#pragma unroll
    for (int i = 0; i < NT; ++i)
      bulk_load(dst[i] + lo, reinterpret_cast<const uint8_t*>(src[i] - off) + lo, hi - lo, bar);
  };
  const long long step = gridDim.x;
  if (t == 0) {
    long long row = blockIdx.x;
    for (int s = 0; s < S && row < p.M; ++s, row += step) issue(row, s);
  }
  uint64_t w[C][4], dw[C][4];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    float v[8];
    load_weight_columns<8, OFF>(p.w, p.w_f32, (i * nt + t) * 8 - off, p.K, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) { w[i][j] = f32x2(v[2 * j], v[2 * j + 1]); dw[i][j] = 0; }
  }
  __syncthreads();
  const float rk = __fdiv_rn(1.0f, (float)p.K);
  RingCursor cur;
  int it = 0;
  long long row = blockIdx.x;
  float rstd = row < p.M ? p.rstd[row] : 0.0f;
  for (; row < p.M; row += step, ++it) {
    const float next_rstd = row + step < p.M ? p.rstd[row + step] : 0.0f;
    const bool ok = mbar_wait(bar0 + 8 * cur.s, cur.phase, p.status);
    const uint8_t* st = ring + cur.s * stage_bytes;
    RawBf16<8> h[C];
    uint64_t u[C][4], c2 = 0;
    const uint64_t rstd2 = f32x2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int at = (i * nt + t) * 8;
      RawBf16<8> a, b;
      a.zero(); b.zero(); h[i].zero();
      if (at < end) {
        a.load(reinterpret_cast<const uint16_t*>(st) + at);
        h[i].load(reinterpret_cast<const uint16_t*>(st + row_bytes) + at);
        if (TWO) b.load(reinterpret_cast<const uint16_t*>(st + 2 * row_bytes) + at);
        if (OFF && !whole_word(at - off, p.K)) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int k = at - off + 2 * j;
            const uint32_t m = ((unsigned)k < (unsigned)p.K ? 0xFFFFu : 0u) |
                               ((unsigned)(k + 1) < (unsigned)p.K ? 0xFFFF0000u : 0u);
            a.w[j] &= m; b.w[j] &= m; h[i].w[j] &= m;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t y = TWO ? add2(widen2(a.w[j]), widen2(b.w[j])) : widen2(a.w[j]);
        const uint64_t hh = widen2(h[i].w[j]), v = mul_f32x2(y, rstd2);
        dw[i][j] = fma2(v, hh, dw[i][j]);
        u[i][j] = mul_f32x2(v, w[i][j]);
        c2 = fma2(u[i][j], hh, c2);
      }
    }
    float c, chi;
    f32x2_split(c2, c, chi);
    c = __fadd_rn(c, chi);
    if (!block_sum_ok(c, sh[it & 1], ok)) {
      // a copy did not arrive in time (reported): no result
      if (t == 0) cur.drain(bar0, S, it > 0 ? S - 1 : S, row, step, p.M);
      return;
    }
    // the previous row's stage has been read by every thread
    if (t == 0 && it > 0) {
      const long long ahead = row + (long long)(S - 1) * step;
      if (ahead < p.M) issue(ahead, cur.s == 0 ? S - 1 : cur.s - 1);
    }
    const float f = -__fmul_rn(rstd, __fmul_rn(rstd, __fmul_rn(c, rk)));      // rstd^2 may leave fp32
    const uint64_t f2 = f32x2(f, f);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int at = (i * nt + t) * 8;
      if (at >= end) continue;
      RawBf16<8> r, o;
      if (RES) r.load(reinterpret_cast<const uint16_t*>(st + (NT - 1) * row_bytes) + at);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint64_t d = fma2(widen2(h[i].w[j]), f2, u[i][j]);
        if (RES) d = add2(d, widen2(r.w[j]));
        float lo, hi;
        f32x2_split(d, lo, hi);
        o.w[j] = pack_bf16(lo, hi);
      }
      store_columns<8, OFF>(o, p.dx + row * p.lddx, at - off, p.K);
    }
    rstd = next_rstd;
    cur.next(S);
  }
  pdl_launch_dependents();
  if (!p.dw) return;
  float* out = gridDim.x == 1 ? p.dw : p.part + (long long)blockIdx.x * p.K;
  if constexpr (OFF) {
    // through the ring, whose copies have all been read, for stores in a row
    float* sum = reinterpret_cast<float*>(ring);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) f32x2_split(dw[i][j], v[2 * j], v[2 * j + 1]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = (i * nt + t) * 8 - off + j;
        if ((unsigned)k < (unsigned)p.K) sum[k] = v[j];
      }
    }
    __syncthreads();
    for (int k = t; k < p.K; k += nt) out[k] = sum[k];
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int k = (i * nt + t) * 8;
      if (k >= p.K) continue;
      if (reinterpret_cast<uintptr_t>(out) % 16 == 0) {
        reinterpret_cast<ulonglong2*>(out + k)[0] = make_ulonglong2(dw[i][0], dw[i][1]);
        reinterpret_cast<ulonglong2*>(out + k)[1] = make_ulonglong2(dw[i][2], dw[i][3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) f32x2_split(dw[i][j], out[k + 2 * j], out[k + 2 * j + 1]);
      }
    }
  }
}

// What the ring does not take (few short rows, rows of more than 8192 columns and
// operands that start at different places of a word) has two kernels: dx from
// one row a block (short rows: one a warp), held in registers with all its loads
// in flight, and dw's partials from blocks of columns.  They read dy and h
// twice; short rows are bound by latency there (2000 x 256: 6.9 us), single
// elements by instructions (3000 x 4161 at different offsets: 72 us, where a
// register form that kept dw beside one row at a time took 216 and the ring, at
// equal offsets, takes 30).  WIDE rows (32 values a thread) would not fit in
// registers with all operands: there the gradients of y are added as they
// arrive and dh is loaded after the reduction.
template <int VEC, int IT, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kNormTeams : kNormMaxThreads) rmsnorm_dx_kernel(const NormBwd p) {
  constexpr bool WIDE = VEC * IT > 16;
  constexpr int ITR = WIDE ? 1 : IT;
  __shared__ float sh[1][kNormMaxWarps];
  pdl_wait();
  pdl_launch_dependents();
  const RowTeam<WARP> team;
  const int t = team.t, nt = team.nt;
  const long long row = team.index;
  const bool live = row < p.M;
  const float rstd = live ? p.rstd[row] : 0.0f;
  RawBf16<VEC> dy[ITR], dy2[ITR], h[IT], dh[ITR];
  float u[IT][VEC], c[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int k = (i * nt + t) * VEC, iw = WIDE ? 0 : i;
    dy[iw].zero(); dy2[iw].zero(); h[i].zero(); dh[iw].zero();
    if (k < p.K && live) {
      dy[iw].load(p.dy + row * p.lddy + k);
      h[i].load(p.h + row * p.ldh + k);
      if (p.dy2) dy2[iw].load(p.dy2 + row * p.lddy2 + k);
      if (!WIDE && p.dh) dh[iw].load(p.dh + row * p.lddh + k);
    }
    if constexpr (WIDE) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) u[i][j] = __fadd_rn(dy[0].value(j), dy2[0].value(j));
    }
  }
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int k = (i * nt + t) * VEC, iw = WIDE ? 0 : i;
    float w[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) w[j] = 0.0f;
    if (k < p.K) load_weight<VEC>(p.w, p.w_f32, k, w);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      if (!WIDE) u[i][j] = __fadd_rn(dy[iw].value(j), dy2[iw].value(j));
      u[i][j] = __fmul_rn(__fmul_rn(u[i][j], rstd), w[j]);
      c[0] = __fmaf_rn(u[i][j], h[i].value(j), c[0]);
    }
  }
  row_sums<WARP, 1>(c, sh);
  const float f = -__fmul_rn(rstd, __fmul_rn(rstd, __fdiv_rn(c[0], (float)p.K)));      // rstd^2 may leave fp32
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int k = (i * nt + t) * VEC, iw = WIDE ? 0 : i;
    if (k >= p.K || !live) continue;
    if (WIDE && p.dh) dh[0].load(p.dh + row * p.lddh + k);
    float d[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) d[j] = __fadd_rn(__fmaf_rn(h[i].value(j), f, u[i][j]), dh[iw].value(j));
    RawBf16<VEC> o;
    o.set(d);
    o.store(p.dx + row * p.lddx + k);
  }
}

// Partials of dw = sum over rows of dy h rstd: one column a thread, the rows
// blockIdx.y, blockIdx.y + gridDim.y, ..., eight of them in flight, which is
// what its time goes by: 95 of the 256 us at 12000 x 4161 by single elements
__global__ void __launch_bounds__(256) rmsnorm_dw_rows_kernel(const NormBwd p) {
  pdl_wait();
  pdl_launch_dependents();
  const int k = blockIdx.x * blockDim.x + threadIdx.x;
  if (k >= p.K) return;
  const long long step = gridDim.y;
  float s = 0.0f;
  for (long long row0 = blockIdx.y; row0 < p.M; row0 += 8 * step) {
    float y[8], h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const long long row = row0 + i * step;
      y[i] = h[i] = 0.0f;
      if (row < p.M) {
        y[i] = bf16_f(p.dy[row * p.lddy + k]);
        if (p.dy2) y[i] = __fadd_rn(y[i], bf16_f(p.dy2[row * p.lddy2 + k]));
        h[i] = __fmul_rn(bf16_f(p.h[row * p.ldh + k]), p.rstd[row]);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s = __fmaf_rn(y[i], h[i], s);
  }
  (gridDim.y == 1 ? p.dw : p.part + (long long)blockIdx.y * p.K)[k] = s;
}

// dw = the sum of the partials: C columns a block, 1024 / C partials at a time.
// 608 partials, 5 MB in L2, at K = 2048; with the writing of the partials it adds
// 3.4 us, most of it latency: the end of one kernel and a chain of two steps.
template <int C>
__global__ void __launch_bounds__(1024) rmsnorm_dw_kernel(const float* part, int parts, int K, float* dw) {
  constexpr int G = 1024 / C;
  __shared__ float sh[C][G + 1];
  pdl_wait();
  pdl_launch_dependents();
  const int c = threadIdx.x % C, g = threadIdx.x / C, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int k = blockIdx.x * C + c;
  float s = 0.0f;
  if (k < K) {
#pragma unroll 8
    for (int i = g; i < parts; i += G) s = __fadd_rn(s, part[(long long)i * K + k]);
  }
  sh[c][g] = s;
  __syncthreads();
  if (warp >= C || blockIdx.x * C + warp >= K) return;
  s = 0.0f;                              // warp w: column w
#pragma unroll
  for (int i = lane; i < G; i += 32) s = __fadd_rn(s, sh[warp][i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, o));
  if (lane == 0) dw[blockIdx.x * C + warp] = s;
}

// ---------------------------------------------------------------- launchers
static bool vec8(const void* p, long long ld) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0);
}
// whether every row of both starts at the same place of a 16-byte word
static bool same_words(const void* a, long long lda, const void* b, long long ldb) {
  return b == nullptr || ((reinterpret_cast<uintptr_t>(a) ^ reinterpret_cast<uintptr_t>(b)) % 16 == 0 &&
                          (lda - ldb) % 8 == 0);
}
static unsigned norm_threads(int K, int per_thread) {
  const int n = (K + per_thread - 1) / per_thread;
  return (unsigned)((n + 31) / 32 * 32);
}

// The ring form: blocks an SM, and the stages that fit beside one another
struct NormRing { unsigned threads; int blocks, stages, smem; };
// 512 threads an SM, 16 columns each (8 columns and 1024 threads: 15.8 against
// 15.1 us at 4093 x 1544, the same at 8192 x 2048); but two blocks of up to 320
// where their registers fit beside one another and there are rows for them (4000
// x 4480: 27.4 against 31.3 us, 4000 x 5120: 30.6 and 32.9; 200 x 4480: 7.7 and 6.7)
constexpr int kRingPair = 320;
static int ring_blocks(long long M, int K, int pair) {    // K: columns of the words that a row touches
  const int threads = (int)norm_threads(K, 8 * kRingWords), n = 512 / threads;
  return n <= 1 && threads <= pair && M >= 1024 ? 2 : (n < 1 ? 1 : n);
}
static NormRing norm_ring(int blocks, int K, int per_thread, int stage) {
  NormRing r{norm_threads(K, per_thread), blocks, 0, 0};
  r.stages = (222 * 1024 / r.blocks - 1024) / stage;
  if (r.stages > kRingStages) r.stages = kRingStages;
  r.smem = r.stages * stage;
  return r;
}
template <auto kernel, typename P>
static cudaError_t launch_ring(const NormRing& r, long long blocks, const P& p, cudaStream_t st) {
  static std::atomic<bool> set[64];      // per device
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64 || !set[dev].load()) {
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 222 * 1024);
    if (err != cudaSuccess) return err;
    if (dev < 64) set[dev].store(true);
  }
  return launch_serial(kernel, dim3((unsigned)blocks), dim3(r.threads), (size_t)r.smem, st, p, r.stages);
}

template <int VEC, int IT, int R, bool WARP, bool OFF>
static cudaError_t norm_fwd(const NormFwd& p, cudaStream_t st) {
  const long long rows = p.q ? (p.M + 127) / 128 * 128 : p.M, per = WARP ? R * kNormTeams : R;
  return launch_serial(add_rmsnorm_kernel<VEC, IT, R, WARP, OFF>, dim3((unsigned)((rows + per - 1) / per)),
                       dim3(WARP ? 32 * kNormTeams : norm_threads(OFF ? p.K + 7 : p.K, VEC * IT)), 0, st, p);
}

// Short rows leave most of a block idle at its barrier: a warp each, two at a
// time where one has a load each at most.  Warp against block: 18.0 and 20.1
// us at 16384 x 768, but 25.6 and 24.4 at 16384 x 1024; two rows against one:
// 11.5 and 12.2 us at 32768 x 256, 9.1 and 10.1 at 32768 x 128.
template <bool OFF>
static cudaError_t norm_fwd_words(const NormFwd& p, cudaStream_t st) {
  const int n = OFF ? p.K + 7 : p.K;     // columns of the words that a row touches
  if (n <= 256) return norm_fwd<8, 1, 2, true, OFF>(p, st);
  if (n <= 512) return norm_fwd<8, 2, 1, true, OFF>(p, st);
  if (n <= 768) return norm_fwd<8, 3, 1, true, OFF>(p, st);
  return n <= 16 * kNormMaxThreads ? norm_fwd<8, 2, 1, false, OFF>(p, st) : norm_fwd<8, 4, 1, false, OFF>(p, st);
}

cudaError_t launch_add_rmsnorm(const NormFwd& p, cudaStream_t st) {
  if (p.K % 8 == 0 && vec8(p.x, p.ldx) && vec8(p.r, p.ldr) && vec8(p.h, p.ldh) && vec8(p.y, p.ldy) && vec8(p.w, 0))
    return norm_fwd_words<false>(p, st);
  // by words, but the shortest rows by single elements, where few lanes would
  // have a word (18434 rows of 127: 6.2 and 7.7 us; of 143: 19.3 and 7.8)
  if (!p.q && p.K > 128 && p.K + 7 <= 32 * kNormMaxThreads && same_words(p.x, p.ldx, p.r, p.ldr) &&
      same_words(p.x, p.ldx, p.h, p.ldh) && same_words(p.x, p.ldx, p.y, p.ldy))
    return norm_fwd_words<true>(p, st);
  if (p.K <= 128) return norm_fwd<1, 4, 1, true, false>(p, st);
  if (p.K <= 4 * kNormMaxThreads) return norm_fwd<1, 4, 1, false, false>(p, st);
  return p.K <= 16 * kNormMaxThreads ? norm_fwd<1, 16, 1, false, false>(p, st)
                                     : norm_fwd<1, 32, 1, false, false>(p, st);
}

// Blocks of the backward's ring, each with its own partial dw (the two-kernel
// form makes no more)
long long rmsnorm_backward_parts(long long M, int K) {
  const long long most = 152ll * ring_blocks(M, K, kRingPair);
  return M < most ? M : most;
}

static cudaError_t norm_dw(const NormBwd& p, long long parts, cudaStream_t st) {
  if (!p.dw || parts == 1) return cudaSuccess;
  // the fewest columns a block that need no more blocks than there are SMs (8, 16
  // and 32: 9.8, 11.5, 13.4 us in all at 8192 x 512; 14.7, 13.8, 14.5 at 4093 x
  // 1544; 26.5, 25.7, 24.6 at 2000 x 7168)
  auto sum = [&](auto kernel, int columns) {
    return launch_serial(kernel, dim3((unsigned)((p.K + columns - 1) / columns)), dim3(1024), 0, st,
                         (const float*)p.part, (int)parts, p.K, p.dw);
  };
  if (p.K <= 8 * 152) return sum(rmsnorm_dw_kernel<8>, 8);
  return p.K <= 16 * 152 ? sum(rmsnorm_dw_kernel<16>, 16) : sum(rmsnorm_dw_kernel<32>, 32);
}

template <auto kernel, bool OFF>
static cudaError_t norm_bwd_ring(const NormBwd& p, int operands, cudaStream_t st) {
  const int n = OFF ? (p.K + 14) / 8 * 8 : p.K;      // columns of the words that a row touches, at most
  // by words a thread has 128 registers: no room for a second block
  const NormRing r = norm_ring(ring_blocks(p.M, n, OFF ? 0 : kRingPair), n, 8 * kRingWords, 2 * n * operands);
  const long long blocks = std::min(p.M, 152ll * r.blocks);      // no more than the workspace has parts
  const cudaError_t err = launch_ring<kernel>(r, blocks, p, st);
  return err != cudaSuccess ? err : norm_dw(p, blocks, st);
}

template <int VEC, int IT, bool WARP>
static cudaError_t norm_bwd_two(const NormBwd& p, cudaStream_t st) {
  if (p.dw) {
    // First dw: dx may replace one of its operands.  About 2048 threads an SM,
    // eight rows a block at least.
    const unsigned threads = p.K < 256 ? norm_threads(p.K, 1) : 256u, gx = ((unsigned)p.K + threads - 1) / threads;
    long long parts = 152ll * (2048 / threads) / gx;
    const long long most = rmsnorm_backward_parts(p.M, p.K);
    if (parts > (p.M + 7) / 8) parts = (p.M + 7) / 8;
    if (p.M <= 16) parts = 1;            // no sum: 4.0 against 4.8 us at 16 x 248 (24 rows: 4.8 and 4.6)
    if (parts > most) parts = most;
    if (parts < 1) parts = 1;
    cudaError_t err = launch_serial(rmsnorm_dw_rows_kernel, dim3(gx, (unsigned)parts), dim3(threads), 0, st, p);
    if (err == cudaSuccess) err = norm_dw(p, parts, st);
    if (err != cudaSuccess) return err;
  }
  const long long per = WARP ? kNormTeams : 1;
  return launch_serial(rmsnorm_dx_kernel<VEC, IT, WARP>, dim3((unsigned)((p.M + per - 1) / per)),
                       dim3(WARP ? 32 * kNormTeams : norm_threads(p.K, VEC * IT)), 0, st, p);
}

template <bool OFF>
static cudaError_t norm_bwd_words(const NormBwd& p, cudaStream_t st) {
  if (p.dy2)
    return p.dh ? norm_bwd_ring<add_rmsnorm_bwd_ring_kernel<kRingWords, true, true, OFF>, OFF>(p, 4, st)
                : norm_bwd_ring<add_rmsnorm_bwd_ring_kernel<kRingWords, true, false, OFF>, OFF>(p, 3, st);
  return p.dh ? norm_bwd_ring<add_rmsnorm_bwd_ring_kernel<kRingWords, false, true, OFF>, OFF>(p, 3, st)
              : norm_bwd_ring<add_rmsnorm_bwd_ring_kernel<kRingWords, false, false, OFF>, OFF>(p, 2, st);
}

cudaError_t launch_add_rmsnorm_backward(const NormBwd& p, cudaStream_t st) {
  const bool v = p.K % 8 == 0 && vec8(p.dy, p.lddy) && vec8(p.dy2, p.lddy2) && vec8(p.h, p.ldh) &&
                 vec8(p.dh, p.lddh) && vec8(p.dx, p.lddx) && vec8(p.w, 0);
  // few short rows are quicker in two kernels (2000 x 256: 6.9 against 7.6 us;
  // 32768 x 256: 32.8 against 19.9; 2000 x 143: 6.9 and 8.3; 18434 x 143: 30.1 and
  // 16.0), and the shortest at any number (30000 x 64: 15.9 and 16.6)
  const bool ring = p.K > 256 || (p.K > 128 && p.M >= 4096);
  if (v) {
    if (ring && p.K <= 8192) return norm_bwd_words<false>(p, st);
    return p.K <= 256 ? norm_bwd_two<8, 1, true>(p, st) : norm_bwd_two<8, 4, false>(p, st);
  }
  if (ring && p.K + 7 <= 8192 && same_words(p.dy, p.lddy, p.dy2, p.lddy2) && same_words(p.dy, p.lddy, p.h, p.ldh) &&
      same_words(p.dy, p.lddy, p.dh, p.lddh) && same_words(p.dy, p.lddy, p.dx, p.lddx))
    return norm_bwd_words<true>(p, st);
  if (p.K <= 128) return norm_bwd_two<1, 4, true>(p, st);
  if (p.K <= 4 * kNormMaxThreads) return norm_bwd_two<1, 4, false>(p, st);
  return p.K <= 16 * kNormMaxThreads ? norm_bwd_two<1, 16, false>(p, st) : norm_bwd_two<1, 32, false>(p, st);
}

}  // namespace mpm
