// The whole expert layer for a few tokens (decode and rollout batches) in one
// kernel, on NVFP4 or MXFP8 weights:
//
//   xq = quantise(x_t),  c = xq W1_e^T,  D = bf16(silu(gate) * up * prob),
//   dq = quantise(D),    y = dq W2_e^T,  out_t = bf16(sum over t's experts of y)
//
// the operands and roundings of the layers' own steps but for y, which stays in
// fp32 until the sum.  It is bound by reading the weights of the experts that
// tokens go to once from HBM, so everything else is arranged around one stream
// of weight tiles that never stops: one persistent block an SM, launched
// cooperatively; a ring of TMA loads (about 200 KB a block, more than HBM's
// latency times an SM's share of its rate) that runs ahead across tasks and
// from the first product's weights into the second's while rows are quantised,
// partial sums are joined or another block's D is waited for.
//
// Each block sorts the routed rows by expert for itself (at most 1024 of them, in shared memory); slots of weight 0
// are left out, experts without rows are never touched.  A group is an expert with up to `nb` of its rows.  A task is 256
// weight rows of a group (FC1: 128 gate and the 128 up rows beside them, FC2: 256 output features) over the whole
// reduction; tasks go around the blocks whole, and where few are left over, those are cut along the reduction into
// parts, whose fp32 partials the last block to finish adds in order.
//
//   tcgen05.mma, block scaled, M = 128 weight rows, N = the group's rows padded
//   to 16, accumulators and scales in TMEM; warp 0 loads weights, warp 10 rows,
//   warp 1 issues MMAs, warps 6-9 put scale tiles into TMEM, warps 2-5 are the
//   epilogue.
//
// Waits between blocks (a group's D, before its second product) are on blocks
// that are resident (the launch is cooperative) and never wait for later work;
// they are bounded like every wait here.
//
// Measured (weights alone over the time, of the 6.67 TB/s of a plain copy): 671B-shaped NVFP4, 1 token 43.7 us (0.68), 7
// tokens 188 to 196 (0.96 to 1.0), 64 tokens and 124 to 152 experts 503 to 522 (1.0); 30B-shaped MXFP8, 1 token 20 us (0.29),
// 33 tokens 77 to 80 (0.89 to 0.92).
// With one token the chain counts: the launch and the meeting of the blocks 4.7 us, the first rows 3, D between the products
// 5 to 8 (partials, D and its quantised rows each pass from block to block through L2), FC2's last steps 3.
#include <atomic>
#include <cooperative_groups.h>
#include <utility>

#include "moe_few.cuh"
#include "nvfp4.cuh"
#include "team_wait.cuh"

namespace mpm {
namespace few {
namespace {

constexpr int NT = 352;                       // 11 warps
constexpr int TILE = 128 * 128;               // 128 weight rows x 128 bytes of K
constexpr uint32_t TMEM_COLS = 512;
constexpr int MAX_STAGES = 6, MIN_STAGES = 2;
constexpr int PRE = 2;                        // steps asked for before the blocks have met (at most MIN_STAGES)
constexpr int SMEM_LIMIT = 227 * 1024;

template <int KIND> struct Fmt;
template <> struct Fmt<MPM_KIND_NVFP4> {
  static constexpr int kStep = 256, kAtoms = 4, kBlock = 16;       // elements a k-step, scale tiles of it
  static constexpr uint32_t kFmt = 1, kUe8m0 = 0;
};
template <> struct Fmt<MPM_KIND_MXFP8> {
  static constexpr int kStep = 128, kAtoms = 1, kBlock = 32;
  static constexpr uint32_t kFmt = 0, kUe8m0 = 1;
};
// a stage: two weight tiles, their scale tiles, the rows' codes, their scales (64 bytes
// for 16 rows and four scale blocks)
constexpr int w_bytes(int kind) { return 2 * TILE + 2 * (kind == MPM_KIND_NVFP4 ? 4 : 1) * 512; }
constexpr int row_scales(int kind) { return (kind == MPM_KIND_NVFP4 ? 4 : 1) * 64; }
constexpr int stage_bytes(int kind, int nb) {
  return (w_bytes(kind) + nb * 128 + nb / 16 * row_scales(kind) + 1023) / 1024 * 1024;
}

// The routed rows sorted by expert, in shared memory.
struct Groups {
  int n;                                      // groups
  uint16_t expert[MAX_R], start[MAX_R], block[MAX_R];   // of each group: expert, first entry of `slot`, first 16-row block
  uint8_t rows[MAX_R];
  uint16_t slot[MAX_R], group[MAX_R];         // grouped rows -> slot t * k + j, and their group
  uint16_t row[MAX_R];                        // slot -> row of dq (0xFFFF: left out)
};
struct Bars {
  uint64_t w[MAX_STAGES], x[MAX_STAGES], sf[MAX_STAGES], empty[MAX_STAGES], acc_full[2], acc_empty[2];
};

MPM_DEV void fence_proxy_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }
MPM_DEV int load_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
MPM_DEV void add_release(int* p, int v) {
  asm volatile("red.release.gpu.global.add.s32 [%0], %1;" :: "l"(p), "r"(v) : "memory");
}
MPM_DEV int add_acq_rel(int* p, int v) {
  int r;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(r) : "l"(p), "r"(v) : "memory");
  return r;
}
// until *p reaches v (bounded)
MPM_DEV bool wait_count(const int* p, int v, int* status) {
  if (load_acquire(p) >= v) return true;
  const long long t0 = clock64();
  while (load_acquire(p) < v) {
    __nanosleep(64);
    if (clock64() - t0 > kWaitLimitCycles) {
      set_status(status, MPM_ERR_DEVICE_TIMEOUT);
      return false;
    }
  }
  return true;
}
// Teams that wait as one: a warp, and the epilogue's four.
struct WarpTeam {
  int lane;
  MPM_DEV bool first() const { return lane == 0; }
  MPM_DEV bool share(bool v) const {
    v = __shfl_sync(0xffffffffu, v, 0);
    __syncwarp();                               // a shuffle alone orders no memory
    return v;
  }
};
struct EpilogueTeam {
  int et;
  MPM_DEV bool first() const { return et == 0; }
  MPM_DEV bool share(bool v) const {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"((uint32_t)v) : "memory");
    return r != 0;
  }
};
// Weights are read once: they leave L2 first, and what the next call finds there
// (its code among it) stays.
MPM_DEV uint64_t once_policy() {
  uint64_t v;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(v));
  return v;
}
MPM_DEV void tma_load_2d_once(uint32_t dst, const void* tmap, int x, int y, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;"
      :: "r"(dst), "l"(tmap), "r"(x), "r"(y), "r"(bar), "l"(policy) : "memory");
}
MPM_DEV void bulk_load_once(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
      :: "r"(dst), "l"(src), "r"(bytes), "r"(bar), "l"(policy) : "memory");
}
// one lane of a converged warp, known as such to the compiler
MPM_DEV bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}
MPM_DEV uint32_t tmem_ld_32x32b_x1(uint32_t taddr) {
  uint32_t v;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(v) : "r"(taddr));
  return v;
}

// One product's tasks over the blocks.  Block b takes tasks b, b + blocks, ... whole: a
// group's tasks lie side by side on neighbouring blocks, so that groups of many rows
// burden no block alone and groups are finished one after the other.  Tasks that
// are left over, at most a third of the blocks', are cut along K into so many parts that
// all blocks take one, before anything else (more than a third: a block alone can pull
// about twice its share of HBM's rate, so uncut they take no longer).
constexpr int PHASES = 2;
constexpr int MAX_PARTS = 8;
struct Cut {
  int nk, tiles;                              // steps a task, tasks a group
  int tasks, cut, parts;                      // the first `cut` tasks are in `parts` parts
  MPM_DEV Cut() {}
  MPM_DEV Cut(int groups, int tiles_, int nk_) : nk(nk_), tiles(tiles_), tasks(groups * tiles_) {
    const int B = (int)gridDim.x, left = tasks % B;
    parts = left ? min(min(B / left, MAX_PARTS), nk / 2) : 1;
    cut = parts >= 3 ? left : 0;
  }
};
// A block's run, part by part (a part: steps k0 .. k1 of one task).
struct Part {
  int group, tile, k0, k1;
  int task;                                   // a cut task's number, or -1
};
struct Walk {
  Cut c[PHASES];
  int phase, next_task;                       // -1: this block's part of a cut task
  MPM_DEV Walk(const Cut& first, const Cut& second) {
    c[0] = first;
    c[1] = second;
    enter(0);
  }
  MPM_DEV const Cut& cut() const { return phase ? c[1] : c[0]; }
  MPM_DEV void enter(int ph) {
    phase = ph;
    next_task = (int)blockIdx.x < cut().cut * cut().parts ? -1 : cut().cut + (int)blockIdx.x;
  }
  // the next part of this phase
  MPM_DEV bool next_here(Part& p) {
    const Cut& u = cut();
    int task = next_task;
    p.k0 = 0;
    p.k1 = u.nk;
    p.task = -1;
    if (task < 0) {
      task = (int)blockIdx.x / u.parts;
      const int piece = (int)blockIdx.x - task * u.parts;
      p.k0 = u.nk * piece / u.parts;
      p.k1 = u.nk * (piece + 1) / u.parts;
      p.task = task;
      next_task = u.cut + (int)blockIdx.x;
    } else {
      if (task >= u.tasks) return false;
      next_task += (int)gridDim.x;
    }
    p.group = task / u.tiles;
    p.tile = task - p.group * u.tiles;
    return true;
  }
  MPM_DEV bool next(Part& p) {
    while (!next_here(p)) {
      if (phase == PHASES - 1) return false;
      enter(phase + 1);
    }
    return true;
  }
};

// A role's place in the ring: the stage, and the parity of its current use.
struct Ring {
  uint32_t s = 0, ph = 0, n = 0;              // n: steps so far
  MPM_DEV void next(uint32_t stages) {
    ++n;
    if (++s == stages) {
      s = 0;
      ph ^= 1u;
    }
  }
  // given up: wait for what is under way in the last uses of `bar`
  MPM_DEV void drain(uint32_t bar, uint32_t stages, int* status) {
    for (uint32_t i = n < stages ? n : stages; i > 0; --i) {
      if (s == 0) { s = stages; ph ^= 1u; }
      --s;
      mbar_wait(bar + 8 * s, ph, status);
    }
  }
};

constexpr int PER_R = (MAX_R + NT - 1) / NT;           // slots a thread, at most
// The slots begin with warp 2: thread 0 announces the block to the others meanwhile (its fence takes 0.7 us).
MPM_DEV int slot_thread() { return (int)threadIdx.x >= 64 ? (int)threadIdx.x - 64 : (int)threadIdx.x + NT - 64; }

// All threads: the groups of the call's rows, from the experts and weights of this
// thread's slots tid, tid + NT, ...
MPM_DEV void build_groups(const FewArgs& a, Groups& g, int (&my)[PER_R], const float (&weight)[PER_R], int* cnt,
                          uint8_t* hist, uint64_t* sums) {
  const int tid = slot_thread(), lane = tid & 31, R = a.T * a.k;
#pragma unroll
  for (int i = 0; i < PER_R; ++i) {
    if (tid + i * NT >= R || weight[i] == 0.0f) {
      my[i] = -1;
    } else if (my[i] < 0 || my[i] >= a.E) {
      set_status(a.status, MPM_ERR_DEVICE_BOUNDS);
      my[i] = -1;
    }
  }
  if (R <= 32) {
    // a warp's worth of slots: groups in the order of their first slots, by ballots alone
    if (tid < 32) {
      const int e = my[0];
      const unsigned same = __match_any_sync(0xffffffffu, e), before = same & ((1u << lane) - 1u);
      const int n = __popc(same), first = __ffs(same) - 1, rank = __popc(before);
      const bool lead = e >= 0 && rank == 0;
      const unsigned mine = lead ? (unsigned)n | ((n > a.nb ? (unsigned)(n + a.nb - 1) / a.nb : 1u) << 8) | ((n + 15) / 16 << 16) : 0u;
      unsigned incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) g.n = (int)(incl >> 8 & 0xFF);
      const unsigned at = __shfl_sync(0xffffffffu, incl - mine, first);
      const int dense = (int)(at & 0xFF), grp = (int)(at >> 8 & 0xFF), blk = (int)(at >> 16);
      if (lead)
        for (int c = 0; c < n; c += a.nb) {
          const int to = grp + c / a.nb;
          g.expert[to] = (uint16_t)e;
          g.start[to] = (uint16_t)(dense + c);
          g.block[to] = (uint16_t)(blk + c / 16);
          g.rows[to] = (uint8_t)min(a.nb, n - c);
        }
      if (e >= 0) {
        g.slot[dense + rank] = (uint16_t)lane;
        g.group[dense + rank] = (uint16_t)(grp + (rank < a.nb ? 0 : rank / a.nb));
      }
      if (lane < R) g.row[lane] = e >= 0 ? (uint16_t)(blk * 16 + rank) : (uint16_t)0xFFFF;
    }
    __syncthreads();
    return;
  }
  for (int e = tid; e < a.E; e += NT) cnt[e] = 0;
  for (int i = tid; i < (R + 31) / 32 * a.E; i += NT) hist[i] = 0;
  __syncthreads();
  int rank[PER_R];
#pragma unroll
  for (int i = 0; i < PER_R; ++i) {
    const int c = (tid + i * NT) / 32;        // a warp has one chunk
    if (c * 32 >= R) break;
    const unsigned same = __match_any_sync(0xffffffffu, my[i]);
    rank[i] = __popc(same & ((1u << lane) - 1u));
    if (my[i] >= 0 && rank[i] == 0) {
      hist[c * a.E + my[i]] = (uint8_t)__popc(same);
      atomicAdd(&cnt[my[i]], __popc(same));
    }
  }
  __syncthreads();
  // rows, groups and 16-row blocks before each expert: one scan of the three in fields of 20 bits
  const int per = (a.E + NT - 1) / NT, e0 = min(tid * per, a.E), e1 = min(e0 + per, a.E);
  uint64_t sum = 0;
  for (int e = e0; e < e1; ++e) {
    const int n = cnt[e];
    const int groups = n <= a.nb ? (n > 0) : (n + a.nb - 1) / a.nb;
    sum += (uint64_t)n | ((uint64_t)groups << 20) | ((uint64_t)((n + 15) >> 4) << 40);
  }
  uint64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sums[tid >> 5] = incl;
  __syncthreads();
  uint64_t at = incl - sum;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w)
    if (w < (tid >> 5)) at += sums[w];
  if (tid == NT - 1) g.n = (int)(((at + sum) >> 20) & 0xFFFFF);
  int dense = (int)(at & 0xFFFFF), grp = (int)((at >> 20) & 0xFFFFF), blk = (int)(at >> 40);
  for (int e = e0; e < e1; ++e) {
    const int n = cnt[e];
    cnt[e] = dense | (blk << 16);             // where its rows start
    for (int c = 0; c < n; c += a.nb) {
      const int m = min(a.nb, n - c);
      g.expert[grp] = (uint16_t)e;
      g.start[grp] = (uint16_t)(dense + c);
      g.block[grp] = (uint16_t)(blk + c / 16);
      g.rows[grp] = (uint8_t)m;
      for (int i = 0; i < m; ++i) g.group[dense + c + i] = (uint16_t)grp;
      ++grp;
    }
    dense += n;
    blk += (n + 15) >> 4;
  }
  __syncthreads();
  // an expert's rows in the order of their slots: those of earlier chunks of 32 slots, then earlier ones of this chunk
#pragma unroll
  for (int i = 0; i < PER_R; ++i) {
    const int r = tid + i * NT, e = my[i];
    if (r >= R) break;
    if (e < 0) {
      g.row[r] = 0xFFFF;
      continue;
    }
    int before = rank[i];
    for (int c = 0; c < r / 32; ++c) before += hist[c * a.E + e];
    g.slot[(cnt[e] & 0xFFFF) + before] = (uint16_t)r;
    g.row[r] = (uint16_t)((cnt[e] >> 16) * 16 + before);
  }
  fence_proxy_async();                        // cnt and hist lie where the ring's loads go
  __syncthreads();
}

// where a row's scale byte of 4-block word `word` goes: [16-row block][step][tile of it][16 rows][4]
template <int KIND>
MPM_DEV size_t scale_at(int row, int nk, int block) {
  constexpr int ATOMS = Fmt<KIND>::kAtoms;
  const int word = block >> 2;
  return ((size_t)(row >> 4) * nk * ATOMS + word) * 64 + (row & 15) * 4 + (block & 3);
}

// All threads: the largest magnitude of token t's row (NVFP4), as bf16 bits of this warp's lanes.
MPM_DEV unsigned row_top(const FewArgs& a, int t) {
  const uint4* src = reinterpret_cast<const uint4*>(a.x + (long long)t * a.ldx);
  unsigned m = 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < a.H / 8; i += NT) {
    const uint4 v = __ldg(src + i);
    m = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(m, v.x), v.y), v.z), v.w);
  }
  return max(m & 0xFFFFu, m >> 16);
}
// All threads: blocks [b0, b1) of token t quantised; the row's largest magnitude `top`.
template <int KIND>
MPM_DEV void quantise_token(const FewArgs& a, int t, int b0, int b1, unsigned top,
                            uint4 (&pre)[Fmt<KIND>::kBlock / 8]) {
  constexpr int VB = Fmt<KIND>::kBlock / 8;   // 16-byte words of a block
  const int tid = threadIdx.x, nk = a.H / Fmt<KIND>::kStep;
  const uint4* src = reinterpret_cast<const uint4*>(a.x + (long long)t * a.ldx);
  const float sg = nvfp4_outer(__uint_as_float(top << 16)), six = __fmul_rn(6.0f, sg);
  for (int b = b0 + tid; b < b1; b += NT) {
    uint4 v[VB];
#pragma unroll
    for (int j = 0; j < VB; ++j) v[j] = b == b0 + tid ? pre[j] : __ldg(src + b * VB + j);
    uint32_t sb;
    if (KIND == MPM_KIND_NVFP4) {
      uint4(&w)[2] = *reinterpret_cast<uint4(*)[2]>(v);
      uint32_t bm = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        bm = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(bm, w[j].x), w[j].y), w[j].z), w[j].w);
      const uint2 code = nvfp4_encode_block(w, max(bm & 0xFFFFu, bm >> 16), sg, six, sb);
      *reinterpret_cast<uint2*>(a.xq + (size_t)t * (a.H / 2) + b * 8) = code;
    } else {
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < VB; ++j) {
        w[4 * j] = v[j].x; w[4 * j + 1] = v[j].y; w[4 * j + 2] = v[j].z; w[4 * j + 3] = v[j].w;
      }
      const int e = mx_exponent(absmax_bf16x2_packed(w) << 16);
      const uint64_t sc = f32x2_splat(pow2_neg(e));
      uint32_t q[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = e4m3x2_scaled(w[2 * j], sc) | (e4m3x2_scaled(w[2 * j + 1], sc) << 16);
      sb = (uint32_t)(e + 127);
      uint4* dst = reinterpret_cast<uint4*>(a.xq + (size_t)t * a.H + b * 32);
      dst[0] = make_uint4(q[0], q[1], q[2], q[3]);
      dst[1] = make_uint4(q[4], q[5], q[6], q[7]);
    }
    a.xs[scale_at<KIND>(t, nk, b)] = (uint8_t)sb;
  }
}

// A team of threads: one row of D in NVFP4 against its whole-row maximum.
MPM_DEV void quantise_d_row(const FewArgs& a, int slot, int row, int member, int team) {
  const int nblk = a.I / 16, nk = a.I / Fmt<MPM_KIND_NVFP4>::kStep;
  const float sg = nvfp4_outer(__uint_as_float(__ldcg(a.amax + slot))), six = __fmul_rn(6.0f, sg);
  const uint4* src = reinterpret_cast<const uint4*>(a.d + (size_t)slot * a.I);
#pragma unroll 4
  for (int b = member; b < nblk; b += team) {
    uint4 v[2] = {__ldcg(src + 2 * b), __ldcg(src + 2 * b + 1)};
    uint32_t bm = 0, sb;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      bm = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(bm, v[j].x), v[j].y), v[j].z), v[j].w);
    const uint2 code = nvfp4_encode_block(v, max(bm & 0xFFFFu, bm >> 16), sg, six, sb);
    *reinterpret_cast<uint2*>(a.dq + (size_t)row * (a.I / 2) + b * 8) = code;
    a.ds[scale_at<MPM_KIND_NVFP4>(row, nk, b)] = (uint8_t)sb;
  }
}

template <int KIND>
__global__ void __launch_bounds__(NT, 1) moe_few_kernel(const __grid_constant__ FewMaps maps, const FewArgs a) {
  using F = Fmt<KIND>;
  constexpr bool NV = KIND == MPM_KIND_NVFP4;
  constexpr int SF = F::kAtoms * 512, RS = F::kAtoms * 64;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Groups g;
  __shared__ float s_prob[MAX_R];
  __shared__ float s_xts[MAX_T];
  __shared__ Bars bars;
  __shared__ uint32_t s_tmem;
  __shared__ int s_flag;
  __shared__ float s_alpha[64], s_p[64];                 // of a task's rows: scale of the product, routing weight
  __shared__ uint16_t s_slot[64];
  __shared__ uint8_t s_col[64];
  __shared__ uint64_t s_sums[NT / 32];
  __shared__ unsigned s_red[NT / 32];
  __shared__ volatile int s_fail;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool leader = elect_one();
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const int S = a.stages, STB = a.stage_bytes;
  const int off_sf = 2 * TILE, off_x = off_sf + 2 * SF, off_xs = off_x + a.nb * 128;
  const uint32_t bar_w = smem_u32(bars.w), bar_x = smem_u32(bars.x), bar_sf = smem_u32(bars.sf),
                 bar_empty = smem_u32(bars.empty), bar_accf = smem_u32(bars.acc_full),
                 bar_acce = smem_u32(bars.acc_empty);
  // The routing and this block's token row are asked for first: once the weights
  // stream, a load waits behind them (about 4 us).  A token's row is shared by as many
  // blocks as there are for it.
  const int R = a.T * a.k;
  int my[PER_R];
  float weight[PER_R];
#pragma unroll
  for (int i = 0; i < PER_R; ++i) {
    const int r = slot_thread() + i * NT;
    my[i] = r < R ? a.ids[r] : -1;
    weight[i] = r < R ? a.prob[r] : 0.0f;
  }
  const int slices = (int)gridDim.x / a.T, t_own = (int)blockIdx.x / slices, slice = (int)blockIdx.x - t_own * slices;
  const int nblk_x = a.H / F::kBlock, xb0 = nblk_x * slice / slices, xb1 = nblk_x * (slice + 1) / slices;
  uint4 pre[F::kBlock / 8] = {};
  unsigned top = 0;
  if (t_own < a.T) {
    const uint4* src = reinterpret_cast<const uint4*>(a.x + (long long)t_own * a.ldx);
    if (xb0 + tid < xb1)
#pragma unroll
      for (int j = 0; j < F::kBlock / 8; ++j) pre[j] = __ldg(src + (xb0 + tid) * (F::kBlock / 8) + j);
    if (NV) top = row_top(a, t_own);
  }
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(bar_w + 8 * s, 1);
      mbar_init(bar_x + 8 * s, 1);
      mbar_init(bar_sf + 8 * s, 4);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_accf + 8 * b, 1);
      mbar_init(bar_acce + 8 * b, 4);
    }
    s_fail = 0;
    fence_mbar_init();
    fence_proxy_async();
    prefetch_tmap(&maps.w1);
    prefetch_tmap(&maps.w2);
    prefetch_tmap(&maps.xq);
    prefetch_tmap(&maps.dq);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&s_tmem), TMEM_COLS);
    tmem_relinquish();
  }
  // Tokens in 8 or 4 bits, and the counters cleared; the blocks meet while they sort the rows.
  if (NV) {
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) s_red[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) top = max(top, s_red[w]);
  }
  for (int i = blockIdx.x * NT + tid; i < a.count_ints; i += gridDim.x * NT) a.count[i] = 0;
  for (int i = blockIdx.x * NT + tid; i < R; i += gridDim.x * NT) a.amax[i] = 0;
  if (t_own < a.T) {
    if (NV && tid == 0 && slice == 0) a.xts[t_own] = nvfp4_outer(__uint_as_float(top << 16));
    quantise_token<KIND>(a, t_own, xb0, xb1, top, pre);
  }
  fence_proxy_global();
  auto met = cooperative_groups::this_grid().barrier_arrive();
#pragma unroll
  for (int i = 0; i < PER_R; ++i)
    if (slot_thread() + i * NT < R) s_prob[slot_thread() + i * NT] = weight[i];
  // the sort's scratch lies in the ring, which is empty until it is done
  build_groups(a, g, my, weight, reinterpret_cast<int*>(gbase), gbase + MAX_E * 4, s_sums);
  int* grp_done = a.count;                               // first product's tasks of a group that are finished
  int* grp_ready = a.count + MAX_R;                      // NVFP4: rows of the group whose D is quantised
  int* part_done = a.count + 2 * MAX_R;                  // parts of a cut task, by phase and first block
  int* tile_done = part_done + PHASES * MAX_CTAS;        // groups whose 256 features are in y

  // ---------------------------------------------------------------- weights
  Walk walk(Cut(g.n, a.I / 128, a.H / F::kStep), Cut(g.n, a.H / 256, a.I / F::kStep));
  Part p{};
  const uint64_t once = once_policy();
  // The weights' producer, step by step: the step's two tiles (rows y0, y1 at byte x) and their scale tiles.
  struct Load {
    const void* map;
    const uint8_t *s0, *s1;
    int x, y0, y1, left;
  } load{};
  Ring ring;
  auto load_part = [&]() {
    load.left = 0;
    if (!walk.next(p)) return;
    const bool second = walk.phase;
    const long long e = g.expert[p.group];
    const long long r0 = second ? e * a.H + p.tile * 256 : e * 2 * a.I + p.tile * 128;
    const long long r1 = second ? r0 + 128 : r0 + a.I;
    const uint8_t* sf = second ? a.w2_s : a.w1_s;
    const long long per_row = (long long)walk.cut().nk * F::kAtoms;        // 512-byte scale tiles of 128 rows
    load.map = second ? &maps.w2 : &maps.w1;
    load.s0 = sf + ((r0 >> 7) * per_row + p.k0 * F::kAtoms) * 512;
    load.s1 = sf + ((r1 >> 7) * per_row + p.k0 * F::kAtoms) * 512;
    load.x = p.k0 * 128;
    load.y0 = (int)r0;
    load.y1 = (int)r1;
    load.left = p.k1 - p.k0;
  };
  auto load_weights = [&]() {
    const uint32_t st = base + ring.s * STB, bar = bar_w + 8 * ring.s;
    mbar_arrive_expect_tx(bar, w_bytes(KIND));
    tma_load_2d_once(st, load.map, load.x, load.y0, bar, once);
    tma_load_2d_once(st + TILE, load.map, load.x, load.y1, bar, once);
    bulk_load_once(st + off_sf, load.s0, SF, bar, once);
    bulk_load_once(st + off_sf + SF, load.s1, SF, bar, once);
    load.x += 128;
    load.s0 += SF;
    load.s1 += SF;
    ring.next(S);
    if (--load.left == 0) load_part();
  };
  if (warp == 0 && leader) {
    load_part();
    for (int s = 0; s < PRE && load.left; ++s) load_weights();
  }
  __syncwarp();
  cooperative_groups::this_grid().barrier_wait(std::move(met));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const uint32_t sf_cols = 3 * F::kAtoms * 4, sf_base = tmem + 4 * a.nb;
  bool ok = true;

  if (warp == 0) {
    if (leader) {
      while (load.left) {
        if (!mbar_wait(bar_empty + 8 * ring.s, ring.ph ^ 1u, a.status)) { ok = false; break; }
        load_weights();
      }
      if (!ok) ring.drain(bar_w, S, a.status);
    }
  } else if (warp == 10) {
    // ---------------------------------------------------------------- rows of each step
    if (leader) {
      fence_proxy_global();
      int ready = -1;                                    // the last group whose D was seen to be there
      while (ok && walk.next(p)) {
        const bool second = walk.phase;
        // the first product takes all tokens' rows, the second its group's
        const int nblk = second ? (g.rows[p.group] + 15) / 16 : a.nb / 16, blk = second ? g.block[p.group] : 0, nk = walk.cut().nk;
        if (second && p.group != ready) {
          ok = NV ? wait_count(grp_ready + p.group, g.rows[p.group], a.status)
                  : wait_count(grp_done + p.group, a.I / 128, a.status);
          if (!ok) break;
          fence_proxy_global();
          ready = p.group;
        }
        const void* map = second ? &maps.dq : &maps.xq;
        const uint8_t* sc = (second ? a.ds : a.xs) + ((size_t)blk * nk + p.k0) * RS;
        const uint32_t bytes = nblk * (2048 + RS);
        int x = p.k0 * 128;
        for (int kb = p.k0; kb < p.k1; ++kb) {
          if (!mbar_wait(bar_empty + 8 * ring.s, ring.ph ^ 1u, a.status)) { ok = false; break; }
          const uint32_t st = base + ring.s * STB, bar = bar_x + 8 * ring.s;
          mbar_arrive_expect_tx(bar, bytes);
#pragma unroll 1
          for (int j = 0; j < nblk; ++j) {
            tma_load_2d(st + off_x + j * 2048, map, x, (blk + j) * 16, bar);
            bulk_load(st + off_xs + j * RS, sc + (size_t)j * nk * RS, RS, bar);
          }
          x += 128;
          sc += RS;
          ring.next(S);
        }
      }
      if (!ok) ring.drain(bar_x, S, a.status);
    }
  } else if (warp == 1) {
    if (leader) {
      // -------------------------------------------------------------- MMA issue
      uint32_t j = 0;
      const uint64_t desc0 = sdesc_sw128(base);
      while (ok && walk.next(p)) {
        const uint32_t n = walk.phase ? (g.rows[p.group] + 15) / 16 * 16 : a.nb;
        const uint32_t idesc = idesc_block_scaled(F::kFmt, n, F::kUe8m0, 0, 128);
        const uint32_t ab = j & 1u;
        if (!mbar_wait(bar_acce + 8 * ab, ((j >> 1) & 1u) ^ 1u, a.status)) break;
        ++j;
        tc_fence_after();
        const uint32_t acc = tmem + ab * 2 * a.nb;
        for (int kb = p.k0; kb < p.k1; ++kb) {
          if (!mbar_wait(bar_sf + 8 * ring.s, ring.ph, a.status)) { ok = false; break; }
          tc_fence_after();
          // descriptors differ in their start address, in units of 16 bytes
          const uint64_t st = desc0 + (uint64_t)(ring.s * (uint32_t)STB >> 4);
          const uint32_t sfc = sf_base + ring.s * sf_cols, sfr = sfc + 2 * F::kAtoms * 4;
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint64_t bdesc = st + (uint32_t)(off_x + ks * 32) / 16;
            const uint32_t add = (kb > p.k0 || ks > 0) ? 1u : 0u;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const uint64_t adesc = st + (w * TILE + ks * 32) / 16;
              if (NV)
                mma_nvf4(acc + w * a.nb, adesc, bdesc, idesc, sfc + (w * F::kAtoms + ks) * 4, sfr + ks * 4, add);
              else
                mma_mxf8(acc + w * a.nb, adesc, bdesc, idesc | ((uint32_t)ks << 4) | ((uint32_t)ks << 29), sfc + w * 4, sfr, add);
            }
          }
          tc_commit(bar_empty + 8 * ring.s);
          ring.next(S);
        }
        if (ok) tc_commit(bar_accf + 8 * ab);
      }
    }
  } else if (warp >= 6) {
    // ---------------------------------------------------------------- scale tiles into TMEM
    const uint32_t tq = (uint32_t)((warp & 3) * 32) << 16;
    while (ok && walk.next(p)) {
      for (int kb = p.k0; kb < p.k1; ++kb) {
        ok = warp_agrees(mbar_wait(bar_w + 8 * ring.s, ring.ph, a.status) && mbar_wait(bar_x + 8 * ring.s, ring.ph, a.status));
        if (!ok) break;
        tc_fence_after();
        const uint8_t* st = gbase + ring.s * STB;
        const uint32_t col = sf_base + tq + ring.s * sf_cols;
#pragma unroll
        for (int i = 0; i < 2 * F::kAtoms; ++i)
          tmem_st_32x32b_x4(col + i * 4, *reinterpret_cast<const uint4*>(st + off_sf + i * 512 + lane * 16));
#pragma unroll
        for (int i = 0; i < F::kAtoms; ++i) {
          // row l in lane l % 32, word l / 32
          const uint8_t* x = st + off_xs + i * 64 + (lane & 15) * 4;
          uint4 v = make_uint4(0, 0, 0, 0);
          if ((lane >> 4) * 16 < a.nb) v.x = *reinterpret_cast<const uint32_t*>(x + (lane >> 4) * RS);
          if (32 + (lane >> 4) * 16 < a.nb) v.y = *reinterpret_cast<const uint32_t*>(x + (2 + (lane >> 4)) * RS);
          tmem_st_32x32b_x4(col + (2 * F::kAtoms + i) * 4, v);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_sf + 8 * ring.s);
        ring.next(S);
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3, f = q * 32 + lane;           // this thread's weight row of each tile
    const uint32_t tq = (uint32_t)(q * 32) << 16;
    const int et = tid - 64;                             // 0 .. 127
    const size_t part_n = (size_t)256 * a.nb;            // floats of a partial
    const int nk2 = a.I / F::kStep;
    if (NV) {
      for (int t = et; t < a.T; t += 128) s_xts[t] = __ldcg(a.xts + t);
      named_sync(1, 128);
    }
    uint32_t j = 0;
    for (int phase = 0; phase < PHASES && ok; ++phase) {
      if (phase) walk.enter(phase);
      const bool second = phase;
      while (walk.next_here(p)) {
        const int n = g.rows[p.group], start = g.start[p.group], row0 = g.block[p.group] * 16;
        const int tile = p.tile;
        const float wts = NV ? __ldg((second ? a.w2_ts : a.w1_ts) + g.expert[p.group]) : 1.0f;
        const uint32_t ab = j & 1u;
        if (!mbar_wait(bar_accf + 8 * ab, (j >> 1) & 1u, a.status)) s_fail = 1;
        ++j;
        if (et < n) {
          const int slot = g.slot[start + et];
          s_slot[et] = (uint16_t)slot;
          s_col[et] = (uint8_t)(second ? et : slot / a.k);         // the row's accumulator column
          if (!second) s_p[et] = s_prob[slot];
          if (NV) s_alpha[et] = __fmul_rn(second ? nvfp4_outer(__uint_as_float(__ldcg(a.amax + slot))) : s_xts[slot / a.k], wts);
        }
        named_sync(1, 128);
        if (s_fail) { ok = false; break; }
        tc_fence_after();
        const uint32_t acc = tmem + tq + ab * 2 * a.nb;
        const bool whole = p.task < 0;
        const int parts = whole ? 1 : walk.cut().parts;  // blocks task * parts ... share the task
        if (!whole) {
          float* mine = a.part + (size_t)(phase * MAX_CTAS + blockIdx.x) * part_n + f;
#pragma unroll 1
          for (int c = 0; c < n; c += 4) {
            uint32_t v0[4], v1[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t col = c + i < n ? s_col[c + i] : 0u;
              v0[i] = tmem_ld_32x32b_x1(acc + col);
              v1[i] = tmem_ld_32x32b_x1(acc + a.nb + col);
            }
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (c + i < n) {
                __stcg(mine + (c + i) * 128, __uint_as_float(v0[i]));
                __stcg(mine + (a.nb + c + i) * 128, __uint_as_float(v1[i]));
              }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_acce + 8 * ab);
          named_sync(1, 128);
          if (et == 0) s_flag = add_acq_rel(part_done + phase * MAX_CTAS + p.task, 1) == parts - 1;
          named_sync(1, 128);
          if (!s_flag) continue;
        }
#pragma unroll 1
        for (int c = 0; c < n; c += 4) {                 // four rows at a time
          float v0[4], v1[4];
          if (whole) {
            uint32_t u0[4], u1[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t col = c + i < n ? s_col[c + i] : 0u;
              u0[i] = tmem_ld_32x32b_x1(acc + col);
              u1[i] = tmem_ld_32x32b_x1(acc + a.nb + col);
            }
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v0[i] = __uint_as_float(u0[i]);
              v1[i] = __uint_as_float(u1[i]);
            }
            if (c + 4 >= n) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar_acce + 8 * ab);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v0[i] = v1[i] = 0.0f;
#pragma unroll 4
            for (int b = 0; b < parts; ++b) {
              const float* from = a.part + (size_t)(phase * MAX_CTAS + p.task * parts + b) * part_n + f;
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (c + i < n) {
                  v0[i] = __fadd_rn(v0[i], __ldcg(from + (c + i) * 128));
                  v1[i] = __fadd_rn(v1[i], __ldcg(from + (a.nb + c + i) * 128));
                }
            }
          }
          if (!second) {
            // D = bf16(silu(gate) * up * prob); rows past the last one are computed and not stored
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = c + i;
              const bool in = r < n;
              const int slot = s_slot[r];
              const float alpha = NV ? s_alpha[r] : 1.0f;
              const __nv_bfloat16 d =
                  __float2bfloat16_rn(swiglu_fwd(__fmul_rn(v0[i], alpha), __fmul_rn(v1[i], alpha), s_p[r]));
              const uint32_t bits = (uint32_t)(*reinterpret_cast<const uint16_t*>(&d)) & 0x7FFFu;
              const uint32_t top = __reduce_max_sync(0xffffffffu, bits > 0x7F80u ? 0u : bits);
              if (NV) {
                if (in) reinterpret_cast<__nv_bfloat16*>(a.d)[(size_t)slot * a.I + tile * 128 + f] = d;
                if (in && lane == 0 && top) atomicMax(a.amax + slot, top << 16);
              } else {
                // the warp's 32 features are one MXFP8 block
                const int e = mx_exponent(top << 16);
                const uint32_t code = cvt_e4m3x2(__fmul_rn(__bfloat162float(d), pow2_neg(e)), 0.0f);
                if (in) a.dq[(size_t)(row0 + r) * a.I + tile * 128 + f] = (uint8_t)code;
                if (in && lane == 0) a.ds[scale_at<KIND>(row0 + r, nk2, tile * 4 + q)] = (uint8_t)(e + 127);
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = c + i;
              const float alpha = NV ? s_alpha[r] : 1.0f;
              float* y = a.y + (size_t)s_slot[r] * a.H + tile * 256 + f;
              if (r < n) {
                __stcg(y, __fmul_rn(v0[i], alpha));
                __stcg(y + 128, __fmul_rn(v1[i], alpha));
              }
            }
          }
        }
        if (!second && !NV) fence_proxy_global();        // the codes are read by TMA
        named_sync(1, 128);
        if (et == 0) add_release(second ? tile_done + tile : grp_done + p.group, 1);
      }
      if (NV && !second && ok) {
        // D's rows go around the blocks, each quantised when its group is complete: by all four warps where
        // every block has one at most, else by a warp each
        const int rows = g.n ? g.start[g.n - 1] + g.rows[g.n - 1] : 0;
        const int team = rows <= (int)gridDim.x ? 128 : 32, B = (int)gridDim.x;
        auto there = [&](int r) { return wait_count(grp_done + g.group[r], a.I / 128, a.status); };
        auto quantise = [&](int r) {
          const int slot = g.slot[r];
          quantise_d_row(a, slot, g.row[slot], et & (team - 1), team);
          fence_proxy_global();
          if (team == 128) named_sync(1, 128);
          else __syncwarp();
          if ((et & (team - 1)) == 0) add_release(grp_ready + g.group[r], 1);
        };
        ok = team == 128 ? rows_as_one(EpilogueTeam{et}, (int)blockIdx.x, B, rows, there, quantise)
                         : rows_as_one(WarpTeam{lane}, (int)blockIdx.x + et / 32 * B, B * 4, rows, there, quantise);
        if (!ok) s_fail = 1;
        named_sync(1, 128);
        ok = !s_fail;
      }
    }
  }
  // ------------------------------------------------------------------ each token's sum, in slot order
  // 256 features of a token a warp, when every group has written them
  __syncwarp();
  __syncthreads();
  const int tiles = a.H / 256;
  for (int i = blockIdx.x + gridDim.x * warp; i < a.T * tiles && !s_fail; i += gridDim.x * (NT / 32)) {
    const int t = i / tiles, tile = i - t * tiles;
    if (!wait_as_one(WarpTeam{lane}, [&]() { return wait_count(tile_done + tile, g.n, a.status); })) break;
    float o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const float* y = a.y + (size_t)t * a.k * a.H + tile * 256 + lane * 8;
    for (int s0 = 0; s0 < a.k; s0 += 8) {
      float4 lo[8], hi[8];
#pragma unroll
      for (int s = 0; s < 8; ++s) {                    // a slot that does not count adds zero
        const bool in = s0 + s < a.k && g.row[t * a.k + (s0 + s < a.k ? s0 + s : 0)] != 0xFFFF;
        const float4* from = reinterpret_cast<const float4*>(y + (size_t)(s0 + s) * a.H);
        lo[s] = in ? __ldcg(from) : make_float4(0.f, 0.f, 0.f, 0.f);
        hi[s] = in ? __ldcg(from + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        o[0] = __fadd_rn(o[0], lo[s].x); o[1] = __fadd_rn(o[1], lo[s].y);
        o[2] = __fadd_rn(o[2], lo[s].z); o[3] = __fadd_rn(o[3], lo[s].w);
        o[4] = __fadd_rn(o[4], hi[s].x); o[5] = __fadd_rn(o[5], hi[s].y);
        o[6] = __fadd_rn(o[6], hi[s].z); o[7] = __fadd_rn(o[7], hi[s].w);
      }
    }
    uint32_t w[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * s], o[2 * s + 1]);
      w[s] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(a.out + (long long)t * a.ldo + tile * 256 + lane * 8) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

int group_rows(long long T) { return (int)(T >= 64 ? 64 : (T + 15) / 16 * 16); }

Layout layout(int kind, long long T, int k, long long E, long long H, long long I) {
  Layout l{};
  const bool nv = kind == MPM_KIND_NVFP4;
  const long long R = T * k, experts = R < E ? R : E;
  l.blocks = R / 16 + experts < R ? R / 16 + experts : R;    // ceil(n / 16) <= n and <= n / 16 + 1, summed
  const size_t rows = (size_t)l.blocks * 16, sb = nv ? 16 : 32;
  size_t at = 0;
  auto take = [&at](size_t bytes) { const size_t o = at; at = up256(at + bytes); return o; };
  const size_t tokens = group_rows(T);
  l.xq = take(tokens * (nv ? H / 2 : H));
  l.xs = take(tokens * (H / sb));
  l.xts = take(T * 4);
  l.d = take(nv ? (size_t)R * I * 2 : 0);
  l.amax = take(R * 4);
  l.dq = take(rows * (nv ? I / 2 : I));
  l.ds = take(rows * (I / sb));
  l.y = take((size_t)R * H * 4);
  l.part_bytes = (size_t)PHASES * MAX_CTAS * 256 * group_rows(T) * 4;
  l.part = take(l.part_bytes);
  l.count_ints = 2 * MAX_R + PHASES * MAX_CTAS + (size_t)(H / 256);
  l.count = take(l.count_ints * 4);
  l.total = at;
  return l;
}

}  // namespace few

template <int KIND>
static cudaError_t launch_few(const FewMaps& maps, FewArgs a, cudaStream_t st) {
  auto kern = few::moe_few_kernel<KIND>;
  static std::atomic<int> sms[64], fixed[64];            // by device: SMs, set last; static shared memory
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (sms[dev] == 0) {
    cudaFuncAttributes fa;
    err = cudaFuncGetAttributes(&fa, kern);
    if (err != cudaSuccess) return err;
    fixed[dev] = (int)fa.sharedSizeBytes;
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, few::SMEM_LIMIT - fixed[dev]);
    if (err != cudaSuccess) return err;
    int n = 0, coop = 0;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    cudaDeviceGetAttribute(&coop, cudaDevAttrCooperativeLaunch, dev);
    if (n < few::MAX_T || !coop) return cudaErrorNotSupported;       // a block a token at least
    sms[dev] = n < few::MAX_CTAS ? n : few::MAX_CTAS;
  }
  a.stage_bytes = few::stage_bytes(KIND, a.nb);
  const int room = few::SMEM_LIMIT - fixed[dev] - 1024;
  a.stages = room / a.stage_bytes < few::MAX_STAGES ? room / a.stage_bytes : few::MAX_STAGES;
  // accumulators: two buffers of two tiles; scales: three sets a stage
  const int sf_cols = 3 * few::Fmt<KIND>::kAtoms * 4;
  while (4 * a.nb + a.stages * sf_cols > (int)few::TMEM_COLS) --a.stages;
  if (a.stages < few::MIN_STAGES) return cudaErrorInvalidValue;
  void* args[] = {const_cast<FewMaps*>(&maps), &a};
  return cudaLaunchCooperativeKernel((const void*)kern, dim3(sms[dev]), dim3(few::NT), args,
                                     (size_t)(1024 + a.stages * a.stage_bytes), st);
}

cudaError_t launch_moe_few(int kind, const FewMaps& maps, const FewArgs& a, cudaStream_t st) {
  return kind == MPM_KIND_NVFP4 ? launch_few<MPM_KIND_NVFP4>(maps, a, st) : launch_few<MPM_KIND_MXFP8>(maps, a, st);
}

}  // namespace mpm
