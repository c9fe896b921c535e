// Log probabilities of given tokens over the vocabulary, with the
// log-sum-exp, the entropy and the most likely alternatives, and the gradient
// of log probability and entropy, for sm_103a.
//
// With z = logits / temperature, M the largest z of a row and
//   rest = sum over all tokens but one with z = M of e^(z - M)
//   w    = sum of e^(z - M) (l - L), l the logits and L their largest
// a row's results are
//   lse = M + log1p(rest),  logp_t = (z_t - M) - log1p(rest),
//   H   = log1p(rest) - w / temperature / (1 + rest).
// The sum is kept without its largest term, which is 1: where a token is
// nearly certain (most positions of a rollout) log p is as small as rest, and
// 1 + rest in fp32 would lose it.  w is of differences that are finite wherever they weigh anything (masked tokens
// stand at the lowest value, and their quotient by a temperature may overflow): above 2^100 the next logit is more than
// 2^76 away, only tokens equal to L weigh anything and w is 0.
//
// Forward: one pass over the logits, bound by reading them (8192 x 32768 bf16 82.6 us, 0.97 of a plain copy's rate; 64 x
// 131072 with 8 alternatives 9.7 us and 1 x 131072 with 20 7.8, latency).  Batches of 32 KB come by bulk copies through a
// ring of three in shared memory, which runs on from row to row; a warp keeps one running maximum, raised once a batch,
// so an element costs one difference, one product, one exponential and two accumulations.  A row goes to a block, or,
// when there are few rows, to a cluster of up to 8 blocks that join through distributed shared memory; a short row to the
// registers of one to four warps.  The alternatives are found in the same pass: after a row's first batch the k-th largest of 32 or 64 group maxima is
// a bound that at least k elements reach, and only what reaches it is put on a list, which the warp that closes the row
// ranks while the next one is read (2047 x 50001 fp32, all rows: 60.6 us without alternatives, 64.5 with one, 68.8 with 4, 81
// with 20; 8192 x 32768 bf16: 82.6, 109, 122, 145: instructions and the waits of the first batch, with 16 reading warps an SM).
//
// Gradient: one read and one write (8192 x 32768 bf16 165 us, 0.98 of a plain copy's rate).
#include <atomic>
#include "logprob.cuh"
#include "packed.cuh"

namespace mpm {
namespace {

constexpr int NT = 256;              // reading threads of a block
constexpr int U = 4;                 // gradient: 16-byte vectors a thread and batch
constexpr int UF = 8;                // forward
constexpr int BATCH = UF * NT;       // vectors of a batch: 32 KB, a stage of the ring
constexpr int STAGES = 3;
constexpr int MAX_TOP = 32;
constexpr int NW = NT / 32;
constexpr int CAP = 768;             // listed candidates of a row (or of a block's part of it): as many as leave an SM two blocks
constexpr int FEW = 128;             // candidates that the closing warp ranks by counting
constexpr int SHORT = 64;            // longer lists are first reduced by the row's own bound (k = 20 at 2047 x 50001: 65.7 -> 61.7 us)
constexpr int MAX_CLUSTER = 8;
constexpr int QUEUE = 4;              // rows handed on ahead
constexpr float LOW = -0x1.FEp127f;  // bf16's lowest finite value: logits at or below it are out of reach
constexpr float FAR = -0x1p100f;     // no probability is left there, unless all logits are as low (lse is -2^90 or less then)
constexpr float MOST = 0x1.FFp127f;  // an lse past it is NaN
constexpr float kLog2e = 1.4426950408889634f;

MPM_DEV float ex2(float t) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return r;
}
MPM_DEV float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
MPM_DEV uint32_t max_nan2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// the largest of a warp's numbers
MPM_DEV float warp_max(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
MPM_DEV float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
MPM_DEV uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// A row of V elements as 16-byte vectors counted from the 16-byte boundary at
// or before its first element: vector q holds elements q * VE - off ...  The
// first and last one may reach past the row.
template <bool F32> struct Row {
  static constexpr int ES = F32 ? 4 : 2, VE = 16 / ES;
  const uint8_t* base;               // the boundary
  long long V;
  int off;                           // elements between the boundary and the row
  int nv;
  MPM_DEV Row(const void* logits, long long row, long long ld, long long v) : V(v) {
    const uint8_t* b = static_cast<const uint8_t*>(logits) + row * ld * ES;
    off = (int)(reinterpret_cast<uintptr_t>(b) & 15) / ES;
    base = b - off * ES;
    nv = (int)((off + V + VE - 1) / VE);
  }
  MPM_DEV long long first(int q) const { return (long long)q * VE - off; }
  // the vectors that lie in the row as a whole: [full0, full1)
  MPM_DEV int full0() const { return off ? 1 : 0; }
  MPM_DEV int full1() const { return (int)((off + V) / VE); }
  // vector q; elements outside of the row are -inf
  MPM_DEV uint4 load(int q) const {
    const long long e = first(q);
    if (e >= 0 && e + VE <= V) return load16(base + (long long)q * 16);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (F32) {
        const bool in = e + i >= 0 && e + i < V;
        w[i] = in ? *(reinterpret_cast<const uint32_t*>(base) + (long long)q * 4 + i) : 0xFF800000u;
      } else {
        uint32_t h[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const bool in = e + 2 * i + j >= 0 && e + 2 * i + j < V;
          h[j] = in ? *(reinterpret_cast<const uint16_t*>(base) + (long long)q * 8 + 2 * i + j) : 0xFF80u;
        }
        w[i] = h[0] | (h[1] << 16);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // this thread's vectors q, q + team, ... below `end` of a batch of a team of threads; a batch that lies inside the row
  // (and below `end`), which is known for the team as a whole, takes plain loads
  MPM_DEV void load_batch(uint4 (&v)[U], int batch, int end, int team) const {
    const int q = batch + ((int)threadIdx.x & (team - 1));
    if (batch * VE >= off && batch + team * U <= end && (long long)(batch + team * U) * VE <= off + V) {
      const uint8_t* p = base + (long long)q * 16;
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = load16(p + u * (team * 16));
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = q + u * team < end ? load(q + u * team) : none();
    }
  }
  static MPM_DEV uint4 none() {
    const uint32_t w = F32 ? 0xFF800000u : 0xFF80FF80u;
    return make_uint4(w, w, w, w);
  }
};

MPM_DEV float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// the words of a vector raised to LOW (a NaN stays), or to FAR, and their largest
template <bool F32, bool TO_FAR = false>
MPM_DEV float clamp_max(uint4& v) {
  if (F32) {
    float f[4] = {__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w)};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = max_nan(f[i], TO_FAR ? FAR : LOW);
    v = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    return fmaxf(max3(f[0], f[1], f[2]), f[3]);
  }
  const uint32_t low2 = TO_FAR ? 0xF180F180u : 0xFF7FFF7Fu;           // the bound twice
  v = make_uint4(max_nan2(v.x, low2), max_nan2(v.y, low2), max_nan2(v.z, low2), max_nan2(v.w, low2));
  const uint32_t a = max_nan2(max_nan2(v.x, v.y), max_nan2(v.z, v.w));
  return fmaxf(bf16lo(a), bf16hi(a));
}
// element pair i of a vector
template <bool F32>
MPM_DEV uint64_t pair(const uint4& v, int i) {
  if (F32) return i == 0 ? f32x2(__uint_as_float(v.x), __uint_as_float(v.y)) : f32x2(__uint_as_float(v.z), __uint_as_float(v.w));
  return widen2(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
}
template <bool F32>
MPM_DEV float element(const uint4& v, int i) {
  float lo, hi;
  f32x2_split(pair<F32>(v, i >> 1), lo, hi);
  return (i & 1) ? hi : lo;
}

// One step of a bitonic sort across a warp: the smaller (low) or the larger of this lane's number and that of the lane
// that differs in bit d.
MPM_DEV float exchange(float v, int d, bool low) {
  const float o = __shfl_xor_sync(0xffffffffu, v, d);
  return low ? fminf(v, o) : fmaxf(v, o);
}
// a warp's 32 numbers in descending order
MPM_DEV float sort_down(float v, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size *= 2)
#pragma unroll
    for (int d = size / 2; d; d /= 2) v = exchange(v, d, ((lane & d) != 0) != ((lane & size) != 0));
  return v;
}

// numbers in descending order, equal ones by ascending index (both zeros equal)
MPM_DEV uint64_t rank_key(float z, long long idx) {
  const uint32_t u = __float_as_uint(z + 0.0f);
  const uint32_t k = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return ((uint64_t)k << 32) | (uint32_t)(0xFFFFFFFFu - (uint32_t)idx);
}
MPM_DEV float key_value(uint64_t key) {
  const uint32_t k = (uint32_t)(key >> 32);
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

// the target of a row as it is given, and what it stands for; -1: not scored
MPM_DEV long long given_target(const void* targets, int i64, long long row) {
  if (!targets) return 0;
  return i64 ? static_cast<const long long*>(targets)[row] : static_cast<const int*>(targets)[row];
}
MPM_DEV long long target_of(long long given, long long V, int* status) {
  if (given >= V) {
    set_status(status, MPM_ERR_DEVICE_BOUNDS);
    return -1;
  }
  return given < 0 ? -1 : given;
}

template <bool F32>
MPM_DEV float logit(const void* logits, long long at) {
  return F32 ? static_cast<const float*>(logits)[at]
             : __uint_as_float((uint32_t)static_cast<const uint16_t*>(logits)[at] << 16);
}

struct Stats { float m, rest, w; };            // of a row or of a part of it

struct Shared {
  // of the row (by its parity among the block's) that the closing warp works on while the next one is read
  struct Half {
    float m[NW], other[NW], own[NW], w[NW];
    int lane[NW];
    unsigned count;                            // listed candidates
    uint64_t best[MAX_TOP];
    uint64_t full, empty;                      // mbarriers
    uint64_t posted;                           // and one of the readers' first maxima
  } half[2];
  // the cluster's first block: the other blocks' parts and their mbarrier
  alignas(16) float4 stats[MAX_CLUSTER];
  uint64_t keys[MAX_CLUSTER][MAX_TOP];
  uint64_t got;
  uint64_t full[STAGES], empty[STAGES];        // mbarriers of the ring
  // the block's rows, handed from the copying warp to the others, and the mbarriers of each place
  struct { long long row, t; uint64_t full, empty; } queue[QUEUE];
  alignas(16) uint4 claim;                     // the answer to a request for another row
  uint64_t claimed;                            // its mbarrier
  alignas(16) float group[2][64];              // of the two rows in work: maxima of four threads each, as far as they have read
};

// stores into another block of the cluster that count as bytes of its mbarrier
MPM_DEV void store_remote(uint32_t addr, const Stats& v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %3}, [%4];"
               :: "r"(addr), "f"(v.m), "f"(v.rest), "f"(v.w), "r"(bar) : "memory");
}
MPM_DEV void store_remote(uint32_t addr, uint64_t v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u64 [%0], %1, [%2];"
               :: "r"(addr), "l"(v), "r"(bar) : "memory");
}
// The 32 best of two descending lists, lane i's the i-th of each, in descending order: the larger of a's i-th and b's
// (31 - i)-th are a bitonic sequence of them.
MPM_DEV uint64_t merge_best(uint64_t a, uint64_t b, int lane) {
  a = max(a, (uint64_t)__shfl_sync(0xffffffffu, (unsigned long long)b, 31 - lane));
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const uint64_t o = __shfl_xor_sync(0xffffffffu, (unsigned long long)a, d);
    a = ((lane & d) != 0) == (o > a) ? a : o;
  }
  return a;
}

// The closing warp: the block's statistics from the readers'.  Where the largest term
// dominates, the elements of the thread that read it are read once more (they
// are in L2) and summed without it.
template <bool F32>
MPM_DEV Stats block_stats(const Shared::Half& h, const Row<F32>& r, int q0, int q1, float c, int lane) {
  const float m = lane < NW ? h.m[lane] : LOW;
  const float M = warp_max(m);
  const float d = m - M;
  const float sc = lane < NW ? ex2(d * c) : 0.0f;
  const float own = lane < NW ? h.own[lane] : 0.0f, other = lane < NW ? h.other[lane] : 0.0f;
  const int ow = __ffs(__ballot_sync(0xffffffffu, lane < NW && m == M)) - 1;
  const float s_all = warp_sum((other + own) * sc);
  // a part of weight 0 (nothing in reach, among others) adds 0: its distance times its number of elements may overflow
  const float w = warp_sum(sc > 0.0f ? sc * fmaf(d, other + own, h.w[lane]) : 0.0f);
  float rest = s_all - 1.0f;
  if (s_all < 1.5f && M > LOW) {
    const int owner = ow * 32 + h.lane[ow];
    float sum = 0.0f, hits = 0.0f;
    for (int q = q0 + owner + NT * lane; q < q1; q += NT * 32) {
      uint4 v = r.load(q);
      clamp_max<F32>(v);
#pragma unroll
      for (int i = 0; i < Row<F32>::VE; ++i) {
        const float z = element<F32>(v, i);
        if (z == M) hits += 1.0f;
        else sum += ex2((z - M) * c);
      }
    }
    const float others = warp_sum((other + (lane == ow ? 0.0f : own)) * sc);
    rest = others + warp_sum(sum) + (warp_sum(hits) - 1.0f);
  }
  return Stats{M, rest, w};
}

// the k-th largest of a warp's 64 numbers, two a lane
MPM_DEV float kth_of_64(float a, float b, int k, int lane) {
  float v = fmaxf(sort_down(a, lane), __shfl_sync(0xffffffffu, sort_down(b, lane), 31 - lane));
#pragma unroll
  for (int d = 16; d; d >>= 1) v = exchange(v, d, (lane & d) != 0);
  return __shfl_sync(0xffffffffu, v, k - 1);
}
// the k-th largest of a warp's 32 numbers: a few are taken off one by one, more are sorted
MPM_DEV float kth_of_32(float v, int k, int lane) {
  if (k > 8) return __shfl_sync(0xffffffffu, sort_down(v, lane), k - 1);
  float top = warp_max(v);
  for (int j = 1; j < k; ++j) {
    // one number at the maximum leaves
    v = lane == __ffs(__ballot_sync(0xffffffffu, v == top)) - 1 ? LOW : v;
    top = warp_max(v);
  }
  return top;
}

// The closing warp, for a row of which more than CAP elements were listed (it rises, or has many equal ones): the list
// anew, by the bound that the whole row gives, in one pass in the order of the row, so that of elements equal to the
// bound the first k are enough.  Returns their number; more than CAP: they do not fit.
template <bool F32>
__device__ __noinline__ unsigned list_again(uint64_t* list, const volatile float* group, const void* logits, long long row,
                                            long long ld, long long V, int q0, int q1, int k, int lane) {
  constexpr int VE = Row<F32>::VE, AHEAD = 4, ROOM = CAP - MAX_TOP;      // the equal ones from the end
  const Row<F32> r(logits, row, ld, V);
  const float bound = kth_of_64(group[2 * lane], group[2 * lane + 1], k, lane);
  unsigned n = 0, equal = 0;
  for (int q = q0 + lane; q - lane < q1; q += 32 * AHEAD) {
    uint4 v[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) v[j] = q + 32 * j < q1 ? r.load(q + 32 * j) : Row<F32>::none();
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const float top = clamp_max<F32>(v[j]);
      if (!__any_sync(0xffffffffu, top > LOW && top >= bound)) continue;
      unsigned above = 0, same = 0;
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float z = element<F32>(v[j], i);
        above |= (unsigned)(z > LOW && z > bound) << i;
        same |= (unsigned)(z > LOW && z == bound) << i;
      }
      const unsigned mine = (unsigned)__popc(above) | ((unsigned)__popc(same) << 16);
      unsigned incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      unsigned at = n + ((incl - mine) & 0xFFFF), eq = equal + ((incl - mine) >> 16);
      const long long e = r.first(q + 32 * j);
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const uint64_t key = rank_key(element<F32>(v[j], i), e + i);
        if (above >> i & 1) {
          if (at < ROOM) list[at] = key;
          ++at;
        }
        if (same >> i & 1) {
          if (eq < (unsigned)k) list[CAP - 1 - eq] = key;
          ++eq;
        }
      }
      const unsigned all = __shfl_sync(0xffffffffu, incl, 31);
      n += all & 0xFFFF;
      equal = min(equal + (all >> 16), (unsigned)k);
    }
  }
  if (n > ROOM) return CAP + 1;
  __syncwarp();
  const uint64_t key = (unsigned)lane < equal ? list[CAP - 1 - lane] : 0;
  __syncwarp();
  if ((unsigned)lane < equal) list[n + lane] = key;
  __syncwarp();
  return n + equal;
}

// The closing warp: what of n listed elements reaches the bound that the whole row gives, in the list's front.
MPM_DEV unsigned shorten(uint64_t* list, unsigned n, const volatile float* group, int k, int lane) {
  const float bound = kth_of_64(group[2 * lane], group[2 * lane + 1], k, lane);
  unsigned m = 0;
  for (unsigned i = lane; i - lane < n; i += 32) {
    const uint64_t key = i < n ? list[i] : 0;
    const bool keep = i < n && key_value(key) >= bound;
    const unsigned all = __ballot_sync(0xffffffffu, keep);
    if (keep) list[m + __popc(all & ((1u << lane) - 1u))] = key;
    m += __popc(all);
  }
  __syncwarp();
  return m;
}

// The closing warp: the k best of n listed elements, or, where they are too many for the list, of the block's part of
// the row, by k rounds of the best below the last.
template <bool F32>
__device__ __noinline__ void select_by_rounds(uint64_t* best_of, const uint64_t* list, unsigned n, const void* logits,
                                              long long row, long long ld, long long V, int q0, int q1, int k, int lane) {
  const Row<F32> r(logits, row, ld, V);
  uint64_t last = ~0ull;
  for (int i = 0; i < k; ++i) {
    uint64_t best = 0;
    if (n <= CAP) {
      for (unsigned j = lane; j < n; j += 32) {
        const uint64_t key = list[j];
        if (key < last && key > best) best = key;
      }
    } else {
      for (int q = q0 + lane; q < q1; q += 32) {
        uint4 v = r.load(q);
        if (!(clamp_max<F32>(v) > LOW)) continue;
#pragma unroll
        for (int j = 0; j < Row<F32>::VE; ++j) {
          const float z = element<F32>(v, j);
          const uint64_t key = rank_key(z, r.first(q) + j);
          if (z > LOW && key < last && key > best) best = key;
        }
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) best = max(best, (uint64_t)__shfl_xor_sync(0xffffffffu, (unsigned long long)best, o));
    if (lane == 0) best_of[i] = best;
    last = best;
    if (!best) break;                          // the entries after it are 0 already
  }
}

// A row's results, by one warp; key: lane i's the i-th alternative
MPM_DEV void write_row(const LogprobFwd& p, long long row, const Stats& st, float zt, uint64_t key, int lane) {
  const bool some = st.m > LOW || st.rest != st.rest;
  // NaN and +inf make every result of the row NaN
  const float lr = st.m < INFINITY ? log1pf(st.rest) : NAN;
  // (of halves: the difference of two logits may overflow where its quotient by the temperature does not)
  auto logp = [&](float z) { return fmaf(0.5f * z - 0.5f * st.m, 2.0f * p.inv_t, -lr); };
  if (lane == 0) {
    const float lse = fmaf(st.m, p.inv_t, lr);
    p.lse[row] = some ? (fabsf(lse) <= MOST ? lse : NAN) : -INFINITY;       // (tested in lr instead: 1 to 2 % in short rows)
    if (p.logp) p.logp[row] = some ? (zt <= LOW ? (lr == lr ? -INFINITY : lr) : logp(zt)) : -INFINITY;
    if (p.entropy) {
      const float h = lr - (st.m > -FAR ? 0.0f : st.w * p.inv_t / (1.0f + st.rest));
      p.entropy[row] = some ? (h < 0.0f ? 0.0f : h) : 0.0f;       // a NaN passes
    }
  }
  if (lane < p.top) {
    p.top_ids[row * p.top + lane] = key ? (int)(0xFFFFFFFFu - (uint32_t)key) : -1;
    p.top_logp[row * p.top + lane] = key ? logp(key_value(key)) : lr == lr ? -INFINITY : lr;
  }
}

// A row that is not scored, by one warp
MPM_DEV void write_unscored(const LogprobFwd& p, long long row, int lane) {
  if (lane == 0) {
    if (p.logp) p.logp[row] = 0.0f;
    p.lse[row] = 0.0f;
    if (p.entropy) p.entropy[row] = 0.0f;
  }
  if (lane < p.top) {
    p.top_ids[row * p.top + lane] = -1;
    p.top_logp[row * p.top + lane] = -INFINITY;
  }
}
// The k best of n listed elements, by one warp: each has as many above it as its place.
MPM_DEV void rank_by_counting(uint64_t* best_of, const uint64_t* list, int n, int k, int lane) {
  for (int i = lane; i - lane < n; i += 64) {
    const uint64_t one = i < n ? list[i] : 0, two = i + 32 < n ? list[i + 32] : 0;
    int above1 = 0, above2 = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) {
      const uint64_t x = list[j];
      above1 += x > one;
      above2 += x > two;
    }
    if (one && above1 < k) best_of[above1] = one;
    if (two && above2 < k) best_of[above2] = two;
  }
  __syncwarp();
}

// A block that has not begun yet is taken over by one that runs: its index is the row to go on with.  So rows
// that are not scored, or a grid that does not divide by the SMs, leave none idle (rows dealt out beforehand: 97 us at
// 2047 x 50001 with 30 % not scored at random; counted out over the blocks beforehand: 8 us for reading 8192 targets
// in each block).
MPM_DEV void request_block(uint32_t answer, uint32_t bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
               :: "r"(answer), "r"(bar) : "memory");
}
// the block taken over; -1: none is left, and none may be asked for again
MPM_DEV long long requested_block(uint32_t answer) {
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .b128 a;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 a, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\t}"
      : "=r"(got), "=r"(x) : "r"(answer) : "memory");
  return got ? (long long)x : -1;
}

// One warp copies batches of the block's rows into a ring in shared memory,
// eight warps read them, and a tenth closes rows (joins the warps' sums, ranks
// the alternatives, writes the results) while the next one is read.
template <bool F32, bool TOP>
__global__ void __launch_bounds__(NT + 64, 2) token_logprob_kernel(const LogprobFwd p, const int lcs) {
  constexpr int VE = Row<F32>::VE, S = STAGES;
  __shared__ Shared sh;
  extern __shared__ uint4 ring[];              // S batches, then (TOP) CAP candidates a half
  uint64_t* const lists = reinterpret_cast<uint64_t*>(ring + S * BATCH);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cs = 1 << lcs, rank = lcs ? (int)cluster_ctarank() : 0;
  const float c = __fmul_rn(kLog2e, p.inv_t);
  if (TOP) {
    for (int i = tid; i < 2 * MAX_TOP; i += NT + 64) sh.half[i / MAX_TOP].best[i % MAX_TOP] = 0;
    if (tid < 2) sh.half[tid].count = 0;
    if (tid < 2 * 64) sh.group[tid / 64][tid % 64] = LOW;
  }
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 1);
      mbar_init(smem_u32(&sh.empty[i]), NW);
    }
    for (int i = 0; i < QUEUE; ++i) {
      mbar_init(smem_u32(&sh.queue[i].full), 1);
      mbar_init(smem_u32(&sh.queue[i].empty), NW + 1);
    }
    mbar_init(smem_u32(&sh.claimed), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.half[i].full), NW);
      mbar_init(smem_u32(&sh.half[i].empty), 1);
      mbar_init(smem_u32(&sh.half[i].posted), NW);
    }
    mbar_init(smem_u32(&sh.got), 1);
    fence_mbar_init();
    fence_proxy_async();
  }
  __syncthreads();
  if (cs > 1) cluster_arrive();                // waited for where a peer's memory is reached
  pdl_wait();
  int par = 0;                                 // of the next scored row
  uint32_t qs = 0, qph = 0;                    // place in the queue
  bool ok = true;
  long long row, t;
  // the next row of the queue; false at its end
  auto next_row = [&]() {
    ok = warp_agrees(ok && mbar_wait(smem_u32(&sh.queue[qs].full), qph, p.status));
    row = sh.queue[qs].row;
    t = sh.queue[qs].t;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.queue[qs].empty));
    if (++qs == QUEUE) {
      qs = 0;
      qph ^= 1u;
    }
    return ok && row >= 0;
  };
  if (warp == NW) {
    // ---------------------------------------------------------------- closing
    uint32_t use = 0;                          // scored rows so far
    if (cs > 1) cluster_wait();                // the peers' barriers are there
    while (next_row()) {
      if (t < 0) {
        if (rank == 0) write_unscored(p, row, lane);
        continue;
      }
      Shared::Half& h = sh.half[par];
      const Row<F32> r(p.logits, row, p.ld, p.V);
      const int q0 = (int)((long long)r.nv * rank >> lcs), q1 = (int)((long long)r.nv * (rank + 1) >> lcs);
      const float zt = p.targets ? logit<F32>(p.logits, row * p.ld + t) : 0.0f;
      ok = warp_agrees(ok && mbar_wait(smem_u32(&h.full), (use >> 1) & 1u, p.status));
      Stats st = block_stats<F32>(h, r, q0, q1, c, lane);
      uint64_t key = 0;
      if (TOP) {
        uint64_t* list = lists + par * CAP;
        unsigned listed = h.count;
        if (listed > CAP && ok)
          listed = list_again<F32>(list, sh.group[par], p.logits, row, p.ld, p.V, q0, q1, p.top, lane);
        else if (listed > SHORT && ok)
          listed = shorten(list, listed, sh.group[par], p.top, lane);
        if (listed > FEW && ok) {
          select_by_rounds<F32>(h.best, list, listed, p.logits, row, p.ld, p.V, q0, q1, p.top, lane);
          __syncwarp();
        } else {
          rank_by_counting(h.best, list, (int)min(listed, (unsigned)FEW), p.top, lane);
        }
        key = lane < p.top ? h.best[lane] : 0;
        __syncwarp();
        if (lane < MAX_TOP) h.best[lane] = 0;
        reinterpret_cast<float2*>(sh.group[par])[lane] = make_float2(LOW, LOW);
        if (lane == 0) h.count = 0;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&h.empty));
      if (cs > 1) {
        const uint32_t got = smem_u32(&sh.got);
        if (rank) {
          // this block's part into the first block's memory
          const uint32_t bar = map_to_rank(got, 0);
          if (lane == 0) store_remote(map_to_rank(smem_u32(&sh.stats[rank]), 0), st, bar);
          if (lane < p.top) store_remote(map_to_rank(smem_u32(&sh.keys[rank][lane]), 0), key, bar);
        } else {
          if (lane == 0) mbar_arrive_expect_tx(got, (uint32_t)(cs - 1) * (16 + 8 * (uint32_t)p.top));
          __syncwarp();
          if (ok) ok = mbar_wait_cluster(got, 0, p.status);
          // lane i: block i's part
          float4 o = make_float4(lane ? LOW : st.m, lane ? 0.0f : st.rest, lane ? 0.0f : st.w, 0.0f);
          if (lane && lane < cs) o = sh.stats[lane];
          const float M = warp_max(o.x);
          const int first = __ffs(__ballot_sync(0xffffffffu, lane < cs && o.x == M)) - 1;
          const float d = o.x - M, sc = lane < cs ? ex2(d * c) : 0.0f;
          const float rest = warp_sum(sc * (lane == first ? o.y : 1.0f + o.y));
          const float w_all = warp_sum(sc > 0.0f ? sc * fmaf(d, 1.0f + o.y, o.z) : 0.0f);
          st = Stats{M, rest, w_all};
          if (TOP) {
            // the blocks' alternatives, each in descending order
            uint64_t of[MAX_CLUSTER];
#pragma unroll
            for (int i = 0; i < MAX_CLUSTER; ++i) of[i] = i == 0 ? key : i < cs && lane < p.top ? sh.keys[i][lane] : 0;
#pragma unroll
            for (int half = MAX_CLUSTER / 2; half; half /= 2)
#pragma unroll
              for (int i = 0; i < half; ++i) of[i] = merge_best(of[i], of[i + half], lane);
            key = of[0];
          }
        }
      }
      if (rank == 0) write_row(p, row, st, zt, key, lane);
      ++use;
      par ^= 1;
    }
    // after a wait that ran out: the peers' stores into this block's memory are given their time to come
    if (cs > 1 && rank == 0 && !ok) mbar_wait_cluster(smem_u32(&sh.got), 0, p.status);
  } else if (warp == NW + 1) {
    // ---------------------------------------------------------------- copying
    uint32_t st = 0, ph = 0, turn = 0;
    auto hand_on = [&](long long r, long long target) {
      ok = ok && mbar_wait(smem_u32(&sh.queue[qs].empty), qph ^ 1u, p.status);
      if (lane == 0) {
        sh.queue[qs].row = r;
        sh.queue[qs].t = target;
        mbar_arrive(smem_u32(&sh.queue[qs].full));
      }
      if (++qs == QUEUE) {
        qs = 0;
        qph ^= 1u;
      }
    };
    row = blockIdx.x >> lcs;
    while (ok && row >= 0) {
      if (!lcs && lane == 0) request_block(smem_u32(&sh.claim), smem_u32(&sh.claimed));
      const long long given = given_target(p.targets, p.targets_i64, row);
      const Row<F32> r(p.logits, row, p.ld, p.V);
      const int q0 = (int)((long long)r.nv * rank >> lcs), q1 = (int)((long long)r.nv * (rank + 1) >> lcs);
      int q = q0;
      auto copy = [&](int end) {
        for (; q < end; q += BATCH) {
          ok = mbar_wait(smem_u32(&sh.empty[st]), ph ^ 1u, p.status);
          if (!ok) break;
          // the whole vectors of the batch; a row's ends are read by their threads
          const int a = max(q, r.full0()), b = min(min(q + BATCH, q1), r.full1());
          const uint32_t bar = smem_u32(&sh.full[st]);
          if (lane == 0) {
            if (b > a) {
              mbar_arrive_expect_tx(bar, (uint32_t)(b - a) * 16);
              bulk_load(smem_u32(ring + st * BATCH + (a - q)), r.base + (long long)a * 16, (uint32_t)(b - a) * 16, bar);
            } else {
              mbar_arrive(bar);
            }
          }
          if (++st == S) {
            st = 0;
            ph ^= 1u;
          }
        }
      };
      // With few rows the first batches are asked for before it is known that the row is scored (0.5 us)
      if (lcs) copy(min(q1, q0 + S * BATCH));
      t = target_of(given, p.V, p.status);
      hand_on(row, t);
      if (t >= 0 && ok) copy(q1);
      if (lcs) break;                          // one row a cluster
      const bool answered = mbar_wait(smem_u32(&sh.claimed), turn, p.status);
      turn ^= 1u;
      row = answered ? requested_block(smem_u32(&sh.claim)) : -1;
      __syncwarp();
      fence_proxy_async();                     // read before the next answer is written
    }
    hand_on(-1, -1);
    // no block leaves before its copies have come, those that nobody reads among them
    for (int i = 0; i < S; ++i) {
      mbar_wait(smem_u32(&sh.full[st]), ph ^ 1u, p.status);
      if (++st == S) {
        st = 0;
        ph ^= 1u;
      }
    }
  } else {
    // ---------------------------------------------------------------- reading
    const uint64_t c2 = f32x2(c, c);
    uint32_t stage = 0, ph = 0, use = 0;        // use: scored rows so far
    while (next_row()) {
      if (t < 0) continue;
      Shared::Half& h = sh.half[par];
      const Row<F32> r(p.logits, row, p.ld, p.V);
      const int q0 = (int)((long long)r.nv * rank >> lcs), q1 = (int)((long long)r.nv * (rank + 1) >> lcs);
      const int nb = (q1 - q0 + BATCH - 1) / BATCH;
      auto post = [&](float v) {                 // the maxima of four threads each so far
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
        if ((lane & 3) == 0) *(volatile float*)&sh.group[par][tid >> 2] = v;
      };
      // the row before the last is closed
      ok = ok && mbar_wait(smem_u32(&h.empty), ((use >> 1) & 1u) ^ 1u, p.status);
      float m = LOW, tmax = LOW, bound = LOW;
      uint64_t s2[2] = {0, 0}, w2[2] = {0, 0};
      for (int b = 0; b < nb; ++b) {
        const int qb = q0 + b * BATCH;
        uint4 v[UF];
        ok = ok && mbar_wait(smem_u32(&sh.full[stage]), ph, p.status);
        const uint4* from = ring + stage * BATCH + tid;
        if (qb >= r.full0() && qb + BATCH <= min(q1, r.full1())) {
#pragma unroll
          for (int u = 0; u < UF; ++u) v[u] = from[u * NT];
        } else {
#pragma unroll
          for (int u = 0; u < UF; ++u) {
            const int q = qb + u * NT + tid;
            v[u] = q >= q1 ? Row<F32>::none() : q >= r.full0() && q < r.full1() ? from[u * NT] : r.load(q);
          }
        }
        if (!TOP) {
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.empty[stage]));
        }
        float vm[UF];
#pragma unroll
        for (int u = 0; u < UF; ++u) vm[u] = clamp_max<F32>(v[u]);
        const float bm = max3(max3(vm[0], vm[1], vm[2]), max3(vm[3], vm[4], vm[5]), fmaxf(vm[6], vm[7]));
        tmax = fmaxf(tmax, bm);
        const float mw = warp_max(bm);
        if (mw > m) {
          // 2^((z - m) c) -> 2^((z - mw) c): s f and (w - D s) f, f = 2^(-D c)
          const float D = fminf(mw - m, 0x1p90f), f = ex2(-D * c);         // f is 0 there, and D s finite
          const uint64_t f2 = f32x2(f, f), nD2 = f32x2(-D, -D);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            w2[i] = mul_f32x2(fma2(nD2, s2[i], w2[i]), f2);
            s2[i] = mul_f32x2(s2[i], f2);
          }
          m = mw;
        }
        if (TOP) {
          // The bound: the k-th largest of group maxima, which that many elements are at or above.  Taken after the first
          // batch, when all warps have posted theirs, and anew at batches 1, 3, 7, ... (k > 8; not at a row's last) or 3, 15, 63, ... from
          // what is posted by then: all of it is of this row, so a warp that is behind makes the bound lower, not
          // wrong, and nobody waits (a barrier each time, with one at the row's end: 56.3 us at 2047 x 50001, k = 4, fp32, against
          // 52.0; 135 against 119 at 8192 x 32768 bf16).  A few are taken off one by one, more are sorted.
          if ((b & (b + 1)) == 0 && (p.top > 8 ? b == 0 || b + 1 < nb : (__popc(b) & 1) == 0)) {
            post(tmax);
            __syncwarp();
            if (b == 0) {
              if (lane == 0) mbar_arrive(smem_u32(&h.posted));
              ok = ok && mbar_wait(smem_u32(&h.posted), (use >> 1) & 1u, p.status);
            }
            const volatile float* group = sh.group[par];
            const float x = group[2 * lane], y = group[2 * lane + 1];
            bound = p.top <= 24 ? kth_of_32(fmaxf(x, y), p.top, lane) : kth_of_64(x, y, p.top, lane);
          }
          // Vectors that reach the bound, found in the ring again: few, and their code is small (unrolled over a
          // thread's vectors it took 14 of 71 us at 2047 x 50001, fetching instructions).
          unsigned reach = 0;
#pragma unroll
          for (int u = 0; u < UF; ++u) reach |= (unsigned)(vm[u] > LOW && vm[u] >= bound) << u;
          while (reach) {
            const int u = __ffs(reach) - 1, q = qb + u * NT + tid;
            reach &= reach - 1;
            const uint4 x = q >= r.full0() && q < r.full1() ? from[u * NT] : r.load(q);
            const long long e = r.first(q);
            unsigned hit = 0;
#pragma unroll
            for (int i = 0; i < VE; ++i) {
              const float z = element<F32>(x, i);
              hit |= (unsigned)(z > LOW && z >= bound) << i;
            }
            unsigned at = hit ? atomicAdd(&h.count, (unsigned)__popc(hit)) : 0;
            for (; hit; hit &= hit - 1, ++at) {
              const int i = __ffs(hit) - 1, j = F32 ? i : i >> 1;
              const uint32_t w = j == 0 ? x.x : j == 1 ? x.y : j == 2 ? x.z : x.w;
              const float z = __uint_as_float(F32 ? w : (i & 1) ? w & 0xFFFF0000u : w << 16);
              if (at < CAP) lists[par * CAP + at] = rank_key(z, e + i);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.empty[stage]));
        }
        if (++stage == S) {
          stage = 0;
          ph ^= 1u;
        }
        const uint64_t nm2 = f32x2(-m, -m);
        auto add = [&](const uint4& x) {
#pragma unroll
          for (int i = 0; i < VE / 2; ++i) {
            const uint64_t d2 = add2(pair<F32>(x, i), nm2);
            float lo, hi;
            f32x2_split(mul_f32x2(d2, c2), lo, hi);
            const uint64_t e2 = f32x2(ex2(lo), ex2(hi));
            w2[i & 1] = fma2(d2, e2, w2[i & 1]);
            s2[i & 1] = add2(e2, s2[i & 1]);
          }
        };
#pragma unroll
        for (int u = 0; u < UF / 2; ++u) add(v[u]);
        if (qb + UF / 2 * NT < q1) {               // a row's last batch is often short
#pragma unroll
          for (int u = UF / 2; u < UF; ++u) add(v[u]);
        }
      }
      // the warp's sums; the lane that holds its largest element apart
      float a, bb, s, w;
      f32x2_split(add2(s2[0], s2[1]), a, bb);
      s = a + bb;
      f32x2_split(add2(w2[0], w2[1]), a, bb);
      w = warp_sum(a + bb);
      const unsigned holds = __ballot_sync(0xffffffffu, tmax == m);
      const int ol = holds ? __ffs(holds) - 1 : 0;
      const float so = warp_sum(lane == ol ? 0.0f : s);
      s = __shfl_sync(0xffffffffu, s, ol);
      if (lane == 0) {
        h.m[warp] = m;
        h.other[warp] = so;
        h.own[warp] = s;
        h.w[warp] = w;
        h.lane[warp] = ol;
      }
      if (TOP) post(tmax);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&h.full));
      ++use;
      par ^= 1;
    }
  }
  if (cs > 1) {
    __syncwarp();
    if (warp != NW) cluster_wait();
    cluster_sync();                            // no block leaves while another may still reach its memory
  }
}

// ---------------------------------------------------------------- short rows
// Rows of up to VL vectors a lane, each by a warp, two or four (W) that hold it in registers: no ring, at most two meetings
// a row, and the sum without its largest term is taken there.  A block of the kernel above takes 1.5 us (3 with
// alternatives) a row whatever its length (8192 x 1000 bf16: 46 us, with 5 alternatives 80).
constexpr int SHORT_WARPS = 4;                 // of a block
constexpr int SHORT_CAP = 256;                 // listed candidates of a row

// the first element of a bf16 vector that is m becomes LOW
MPM_DEV void leave_out(uint4& v, float m) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  bool found = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (!found && element<false>(v, i) == m) {
      found = true;
      w[i >> 1] = (i & 1) ? (w[i >> 1] & 0xFFFFu) | 0xFF7F0000u : (w[i >> 1] & 0xFFFF0000u) | 0xFF7Fu;
    }
  }
  v = make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool F32, bool TOP, int VL, int W>
__global__ void __launch_bounds__(SHORT_WARPS * 32, VL > 4 ? 4 : 8) token_logprob_short_kernel(const LogprobFwd p, const bool ahead) {
  constexpr int VE = Row<F32>::VE, TEAM = 32 * W;
  struct Mine {
    uint4 row[TOP ? VL * TEAM : 1];
    uint64_t list[TOP ? SHORT_CAP : 1], best[MAX_TOP];
    float group[64], m[W], s[W], w[W], hits[W];
    unsigned count;
  };
  __shared__ Mine sh[SHORT_WARPS / W];
  const int lane = threadIdx.x & 31, wi = (threadIdx.x >> 5) % W, team = threadIdx.x / TEAM, tl = threadIdx.x % TEAM;
  const long long row = (long long)blockIdx.x * (SHORT_WARPS / W) + team;
  auto meet = [&]() {
    if (W == 1) __syncwarp();
    else named_sync(1 + team, TEAM);
  };
  pdl_wait();
  if (row >= p.T) return;
  Mine& my = sh[team];
  const float c = __fmul_rn(kLog2e, p.inv_t);
  const Row<F32> r(p.logits, row, p.ld, p.V);
  uint4 v[VL];
  auto load = [&]() {
    const int f0 = r.full0(), f1 = r.full1();
    // the last vector where it reaches past the row (and is not the first one too)
    uint4 e = Row<F32>::none();
    if (f1 < r.nv && f1 >= f0 && tl == f1 % TEAM) e = r.load(f1);
#pragma unroll
    for (int u = 0; u < VL; ++u) {
      const int q = u * TEAM + tl;
      v[u] = q == f1 ? e : Row<F32>::none();
      if (q >= f0 && q < f1) v[u] = load16(r.base + q * 16);
    }
    if (tl == 0 && f0) v[0] = r.load(0);
  };
  const long long given = given_target(p.targets, p.targets_i64, row);
  if (ahead) load();                           // few rows: before it is known that the row is scored
  const long long t = target_of(given, p.V, p.status);
  if (t < 0) {
    if (wi == 0) write_unscored(p, row, lane);
    return;
  }
  if (!ahead) load();
  const float zt = p.targets ? logit<F32>(p.logits, row * p.ld + t) : 0.0f;
  float a = LOW, b = LOW, vm[VL];              // this lane's largest in even and odd vectors, and of each
  if (TOP) {
#pragma unroll
    for (int u = 0; u < VL; ++u)
      if (u * TEAM < r.nv) my.row[u * TEAM + tl] = v[u];
  }
#pragma unroll
  for (int u = 0; u < VL; ++u) {
    if (u * TEAM < r.nv) {
      vm[u] = clamp_max<F32>(v[u]);
      if (u & 1) b = fmaxf(b, vm[u]);
      else a = fmaxf(a, vm[u]);
    }
  }
  // the team's largest element, and the first warp that has it
  float m = warp_max(fmaxf(a, b));
  bool mine = true;
  if (W > 1) {
    if (lane == 0) my.m[wi] = m;
    if (TOP) {
      float gm = fmaxf(a, b);
      if (W == 4) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 1));
      if (W == 2 || (lane & 1) == 0) my.group[W == 2 ? tl : tl >> 1] = gm;
    }
  }
  if (TOP && wi == 0) {
    my.best[lane] = 0;
    if (lane == 0) my.count = 0;
  }
  meet();
  if (W > 1) {
    const float own = m;
    int first = W;
#pragma unroll
    for (int i = W - 1; i >= 0; --i) m = fmaxf(m, my.m[i]);
#pragma unroll
    for (int i = W - 1; i >= 0; --i) first = my.m[i] == m ? i : first;
    mine = own == m && first == wi;
  }
  uint64_t key = 0;
  if (TOP) {
    if (W > 1) {
      a = my.group[2 * lane];
      b = my.group[2 * lane + 1];
    }
    const float bound = p.top <= 24 ? kth_of_32(fmaxf(a, b), p.top, lane) : kth_of_64(a, b, p.top, lane);
    unsigned reach = 0;
#pragma unroll
    for (int u = 0; u < VL; ++u)
      if (u * TEAM < r.nv) reach |= (unsigned)(vm[u] > LOW && vm[u] >= bound) << u;
    for (; reach; reach &= reach - 1) {
      const int q = (__ffs(reach) - 1) * TEAM + tl;
      const uint4 x = my.row[q];
      const long long e = r.first(q);
      unsigned hit = 0;
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float z = element<F32>(x, i);
        hit |= (unsigned)(z > LOW && z >= bound) << i;
      }
      unsigned at = hit ? atomicAdd(&my.count, (unsigned)__popc(hit)) : 0;
      for (; hit; hit &= hit - 1, ++at) {
        const int i = __ffs(hit) - 1, j = F32 ? i : i >> 1;
        const uint32_t w = j == 0 ? x.x : j == 1 ? x.y : j == 2 ? x.z : x.w;
        const float z = __uint_as_float(F32 ? w : (i & 1) ? w & 0xFFFF0000u : w << 16);
        if (at < SHORT_CAP) my.list[at] = rank_key(z, e + i);
      }
    }
  }
  // bf16: one largest element leaves the sum (25.3 -> 17.5 us at 8192 x 4000; fp32 instead sums again where that element is more than
  // the others together: 12.3 against 17.6 at 8192 x 1000)
  bool left = F32 || !mine || !(m > LOW);
#pragma unroll
  for (int u = 0; u < VL; ++u) {
    if (u * TEAM < r.nv && !left) {
      const unsigned holds = __ballot_sync(0xffffffffu, vm[u] == m);
      left = holds != 0;
      if (holds && lane == __ffs(holds) - 1) leave_out(v[u], m);
    }
  }
  const uint64_t c2 = f32x2(c, c), nm2 = f32x2(-m, -m);
  uint64_t s2[2] = {0, 0}, w2[2] = {0, 0};
#pragma unroll
  for (int u = 0; u < VL; ++u) {
    if (u * TEAM < r.nv) {
#pragma unroll
      for (int i = 0; i < VE / 2; ++i) {
        const uint64_t d2 = add2(pair<F32>(v[u], i), nm2);
        float lo, hi;
        f32x2_split(mul_f32x2(d2, c2), lo, hi);
        const uint64_t e2 = f32x2(ex2(lo), ex2(hi));
        s2[i & 1] = add2(s2[i & 1], e2);
        w2[i & 1] = fma2(e2, d2, w2[i & 1]);
      }
    }
  }
  float x, y;
  f32x2_split(add2(s2[0], s2[1]), x, y);
  float s = warp_sum(x + y);
  f32x2_split(add2(w2[0], w2[1]), x, y);
  float w = warp_sum(x + y);
  if (W > 1) {
    if (lane == 0) my.s[wi] = s, my.w[wi] = w;
  }
  if (W > 1 || TOP) meet();
  if (W > 1) {
    s = w = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) s += my.s[i], w += my.w[i];
  }
  Stats st{m, F32 ? s - 1.0f : s, w};
  if (F32 && s < 1.5f && m > LOW) {
    float sum = 0.0f, hits = 0.0f;
#pragma unroll
    for (int u = 0; u < VL; ++u) {
      if (u * TEAM < r.nv) {
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          const float z = element<F32>(v[u], i);
          if (z == m) hits += 1.0f;
          else sum += ex2((z - m) * c);
        }
      }
    }
    sum = warp_sum(sum);
    hits = warp_sum(hits);
    if (W > 1) {
      meet();                                  // the sums before have been read
      if (lane == 0) my.s[wi] = sum, my.hits[wi] = hits;
      meet();
      sum = hits = 0.0f;
#pragma unroll
      for (int i = 0; i < W; ++i) sum += my.s[i], hits += my.hits[i];
    }
    st.rest = sum + (hits - 1.0f);
  }
  if (wi) return;
  if (TOP) {
    const unsigned n = my.count;
    if (n <= SHORT_CAP) rank_by_counting(my.best, my.list, (int)n, p.top, lane);
    else select_by_rounds<F32>(my.best, my.list, CAP + 1, p.logits, row, p.ld, p.V, 0, r.nv, p.top, lane);
    __syncwarp();
    key = lane < p.top ? my.best[lane] : 0;
  }
  write_row(p, row, st, zt, key, lane);
}

// ---------------------------------------------------------------- gradient
//   dz_i = g_l ([i = t] - p_i) - g_h p_i (log p_i + H),  p_i = e^(z_i - lse)
// in one read and one write; the given token's own 1 - p is -expm1(log p), of the forward's log p where that is given: lse
// rounded to fp32 holds no 1 - p of a nearly certain token.  An item, a row's chunk of
// 2^lt U vectors, goes to a team of 2^lt threads: a block, or, where rows are short, down to a warp.
// (A team of the whole block is known as such, so that what is the same for the block stays out of the threads'
// registers: with the team's size as an argument alone 8192 x 32768 bf16 took 269 us instead of 163.)
// A vector of a row whose lse is -2^90 or less: the scaled logits next to it are 2^66 away or more, so p is 1 at lse and 0
// elsewhere, as it is of 0, FAR and (out of reach) -inf with an lse of 0.
template <bool F32>
MPM_DEV uint4 at_lse(const uint4& v, float inv_t, float lse) {
  uint32_t w[4];
  auto bits = [&](int i) {
    const float z = element<F32>(v, i);
    return z * inv_t == lse ? 0u : (F32 ? 0x10000u : 1u) * (z > LOW ? 0xF180u : 0xFF80u);
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = F32 ? bits(i) : bits(2 * i) | (bits(2 * i + 1) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The same as a call: where registers are short (teams; in line its code spills: 14.0 us at 8192 x 1000 bf16)
template <bool F32>
__device__ __noinline__ uint4 at_lse_called(const uint4 v, float inv_t, float lse) { return at_lse<F32>(v, inv_t, lse); }

// (Whether log p is given is known as such too: tested at the target it cost the teams' registers 21 % at 8192 x 2000 fp32.)
template <bool F32, bool OUT32, bool PARTS, bool LOGP>
__global__ void __launch_bounds__(NT, PARTS ? 3 : 4) token_logprob_backward_kernel(const LogprobBwd p, const int chunks, const int lt) {
  constexpr int VE = Row<F32>::VE, OS = OUT32 ? 4 : 2;
  // What an item needs besides its logits
  struct Item {
    long long row, t;
    int chunk;
    float lse, gl, gh, H;
  };
  pdl_wait();
  const int team = PARTS ? 1 << lt : NT;
  const long long items = p.T * chunks, first = PARTS ? (long long)blockIdx.x * (NT >> lt) + (threadIdx.x >> lt) : blockIdx.x;
  const long long step = PARTS ? (long long)gridDim.x * (NT >> lt) : gridDim.x;
  auto fetch = [&](long long i) {
    Item x;
    x.row = chunks == 1 ? i : i / chunks;
    x.chunk = (int)(i - x.row * chunks);
    x.t = -1;
    x.lse = x.gl = x.gh = x.H = 0.0f;
    if (i < items) {
      x.t = target_of(given_target(p.targets, p.targets_i64, x.row), p.V, p.status);
      x.lse = p.lse[x.row];
      if (p.dlogp) x.gl = p.dlogp[x.row];
      if (p.dentropy) {
        x.gh = p.dentropy[x.row];
        x.H = p.entropy[x.row];
      }
    }
    return x;
  };
  auto load = [&](const Item& x, uint4 (&v)[U]) {
    if (x.t >= 0 && x.lse != -INFINITY) {
      const Row<F32> r(p.logits, x.row, p.ld, p.V);
      r.load_batch(v, x.chunk * (team * U), r.nv, team);
    }
  };
  // an item's logits are on their way while the one before is worked on, and its row's numbers before that
  uint4 v[U];
  Item x = fetch(first), nx = fetch(first + step);
  load(x, v);
  for (long long i = first; i < items; i += step) {
    uint4 nv[U];
    const Item nnx = fetch(i + 2 * step);
    if (i + step < items) load(nx, nv);
    const Row<F32> r(p.logits, x.row, p.ld, p.V);
    const bool zero = x.t < 0 || x.lse == -INFINITY;
    if (__builtin_expect(!zero && x.lse <= -0x1p90f, 0)) {
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = PARTS ? at_lse_called<F32>(v[u], p.inv_t, x.lse) : at_lse<F32>(v[u], p.inv_t, x.lse);
      x.lse = 0.0f;
    }
    // -p (g_l + g_h (log p + H)) / temperature = p (A log p + B)
    const float A = -x.gh * p.inv_t, G = x.gl * p.inv_t, K = x.gh * x.H * p.inv_t, B = -(G + K);
    const uint64_t it2 = f32x2(p.inv_t, p.inv_t), zero2 = f32x2(p.zero, p.zero), nl2 = f32x2(-x.lse, -x.lse), k2 = f32x2(kLog2e, kLog2e);
    const uint64_t A2 = f32x2(A, A), B2 = f32x2(B, B);
    uint8_t* out = static_cast<uint8_t*>(p.out) + x.row * p.ldo * OS;
    constexpr int OA = VE * OS > 16 ? 15 : VE * OS - 1;
    // vectors of the row that can be stored whole
    const bool wide = ((reinterpret_cast<uintptr_t>(out) - (uintptr_t)r.off * OS) & OA) == 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = x.chunk * (team * U) + u * team + ((int)threadIdx.x & (team - 1));
      if (q >= r.nv) break;
      const long long e = r.first(q);
      float d[VE];
      if (zero) {
#pragma unroll
        for (int j = 0; j < VE; ++j) d[j] = 0.0f;
      } else {
        uint4 near = v[u];
        clamp_max<F32, true>(near);
#pragma unroll
        for (int j = 0; j < VE / 2; ++j) {
          // The scaled logit is rounded before lse is taken off, as lse was: so no p comes out above 1 (at logits of 1e9
          // lse's rounding is 32), and where a token is nearly certain the difference is 0 rather than what that left.
          // (A zero that the compiler does not know: a product would be drawn into the sum.)
          const uint64_t lp2 = add2(fma2(pair<F32>(near, j), it2, zero2), nl2);
          float lo, hi;
          f32x2_split(mul_f32x2(lp2, k2), lo, hi);
          const uint64_t e2 = f32x2(ex2(lo), ex2(hi));         // p log p first: 0 where p is
          f32x2_split(fma2(mul_f32x2(e2, lp2), A2, mul_f32x2(e2, B2)), d[2 * j], d[2 * j + 1]);
        }
        if (p.targets && (unsigned long long)(x.t - e) < (unsigned long long)VE) {
#pragma unroll
          for (int j = 0; j < VE; ++j)
            if (x.t == e + j) {
              const float z = element<F32>(v[u], j), own = LOGP ? p.logp[x.row] : __fsub_rn(__fmul_rn(z, p.inv_t), x.lse);
              const float lp = max_nan(own, FAR), pt = expf(lp);         // p log p first: 0 where p is
              d[j] = z <= LOW && x.lse == x.lse ? 0.0f : -fmaf(G, expm1f(lp), fmaf(-A, pt * lp, pt * K));
            }
        }
      }
      uint8_t* o = out + e * OS;
      if (wide && e >= 0 && e + VE <= p.V) {
        uint32_t w[VE * OS / 4];
#pragma unroll
        for (int j = 0; j < VE * OS / 4; ++j) {
          if (OUT32) {
            w[j] = __float_as_uint(d[j]);
          } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(d[2 * j], d[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&h);
          }
        }
        if (VE * OS == 8) {
          __stcs(reinterpret_cast<uint2*>(o), make_uint2(w[0], w[1]));
        } else {
#pragma unroll
          for (int j = 0; j < VE * OS / 16; ++j)
            __stcs(reinterpret_cast<uint4*>(o + 16 * j), make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]));
        }
      } else {
#pragma unroll
        for (int j = 0; j < VE; ++j)
          if (e + j >= 0 && e + j < p.V) {
            if (OUT32) *reinterpret_cast<float*>(o + 4 * j) = d[j];
            else *reinterpret_cast<__nv_bfloat16*>(o + 2 * j) = __float2bfloat16_rn(d[j]);
          }
      }
    }
    x = nx;
    nx = nnx;
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = nv[u];
  }
}

int sm_count() {
  static std::atomic<int> sms[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  if (!sms[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) n = 152;
    sms[dev] = n;
  }
  return sms[dev];
}

}  // namespace

template <int VL, int W>
static cudaError_t launch_short(const LogprobFwd& p, cudaStream_t st) {
  auto kern = p.f32 ? (p.top ? token_logprob_short_kernel<true, true, VL, W> : token_logprob_short_kernel<true, false, VL, W>)
                    : (p.top ? token_logprob_short_kernel<false, true, VL, W> : token_logprob_short_kernel<false, false, VL, W>);
  const long long blocks = (p.T + SHORT_WARPS / W - 1) / (SHORT_WARPS / W);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(SHORT_WARPS * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p, blocks <= sm_count() * (VL > 4 ? 4 : 8));
}

cudaError_t launch_token_logprob(const LogprobFwd& p, cudaStream_t st) {
  // By the registers of up to four warps where a row, wherever its first vector begins, fits in them; rows above 2 KB only where
  // there are more than blocks at once (5 alternatives, so against by blocks: 8192 x 1000 bf16 12.3 / 80 us, 100 x 1000 3.8 / 5.5,
  // 8192 x 4000 31.6 / 83, x 8000 49.0 / 84, 4000 x 16000 43.9 / 50.9, but 64 x 4000 11 / 5.5).
  const long long most = p.V * (p.f32 ? 4 : 2) + 15;
  if (most <= 4 * 512) return launch_short<4, 1>(p, st);
  const long long slots = (long long)sm_count() * 2;
  if (most <= 16 * 512 && p.T > slots) return launch_short<16, 1>(p, st);
  if (most <= 16 * 1024 && p.T > slots) return launch_short<16, 2>(p, st);
  if (most <= 16 * 2048 && p.T > slots) return launch_short<16, 4>(p, st);
  auto kern = p.f32 ? (p.top ? token_logprob_kernel<true, true> : token_logprob_kernel<true, false>)
                    : (p.top ? token_logprob_kernel<false, true> : token_logprob_kernel<false, false>);
  const int smem = p.top ? STAGES * BATCH * 16 + 2 * CAP * (int)sizeof(uint64_t) : STAGES * BATCH * 16;
  static std::atomic<bool> ready[64][4];        // by device and kernel
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  std::atomic<bool>* done = dev >= 0 && dev < 64 ? &ready[dev][(p.f32 ? 2 : 0) + (p.top ? 1 : 0)] : nullptr;
  if (!done || !*done) {
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    if (done) *done = true;
  }
  const long long nv = (p.V * (p.f32 ? 4 : 2) + 15) / 16;
  int lcs = 0;                                  // log2 of the blocks a row
  while ((1 << lcs) < MAX_CLUSTER && p.T << (lcs + 1) <= slots && nv >> (lcs + 1) >= BATCH / 4) ++lcs;
  const int cs = 1 << lcs;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.T << lcs));   // a row a block, or a cluster (then all of them fit at once)
  cfg.blockDim = dim3(NT + 64);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cs;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cs > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p, lcs);
}

template <bool F32, bool OUT32>
static cudaError_t launch_backward(const LogprobBwd& p, cudaStream_t st) {
  // a row's bytes from the 16-byte boundary before it: the same for all rows where the pitch is a multiple of 16
  const long long es = p.f32 ? 4 : 2, off = (long long)(reinterpret_cast<uintptr_t>(p.logits) % 16);
  const long long nv = (p.V * es + (p.ld * es % 16 == 0 || p.T == 1 ? off : 16 - es) + 15) / 16;
  const long long slots = (long long)sm_count() * 4;
  // Rows of up to 2048 elements leave most of a block idle; where there are more of them than blocks at once, the smallest
  // team that holds a row takes it (8192 x 100 bf16: 8.8 us against 28.8 by blocks, x 1000 13.1 / 26.0, x 2000 25.0 / 29.8;
  // fp32 x 2000 26.0 / 31.8; bf16 x 4000 43.5 / 36.1; few rows, 96 x 1000: 3.1 / 2.5).
  int lt = 8;
  if (nv * 16 <= 2048 * es)
    while (lt > 5 && nv <= (long long)U << (lt - 1) && p.T << lt > slots * NT) --lt;
  const int chunks = (int)((nv + ((long long)U << lt) - 1) / ((long long)U << lt));
  const long long blocks = (p.T * chunks + (NT >> lt) - 1) / (NT >> lt);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks < slots ? blocks : slots));
  cfg.blockDim = dim3(NT);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kern = lt < 8 ? (p.logp ? token_logprob_backward_kernel<F32, OUT32, true, true> : token_logprob_backward_kernel<F32, OUT32, true, false>)
                     : (p.logp ? token_logprob_backward_kernel<F32, OUT32, false, true> : token_logprob_backward_kernel<F32, OUT32, false, false>);
  return cudaLaunchKernelEx(&cfg, kern, p, chunks, lt);
}

cudaError_t launch_token_logprob_backward(const LogprobBwd& p, cudaStream_t st) {
  if (p.f32) return p.out_f32 ? launch_backward<true, true>(p, st) : launch_backward<true, false>(p, st);
  return p.out_f32 ? launch_backward<false, true>(p, st) : launch_backward<false, false>(p, st);
}

}  // namespace mpm
