// Expert segments, permutation gather and combine for sm_103a.
//
// "miniTE technical report", section 5.2: the routed rows of all experts sit
// in one contiguous buffer whose expert boundaries are offsets kept on the
// device; zero-token experts and the padding of each segment (to 128 rows, one
// MMA tile, 256, one CTA-pair tile, or 16-64 rows for the small-M kernel) are
// handled in the same path.  Section 5.3: the permute gathers each routed
// (token, slot) row; the combine sums a token's expert outputs.
//
// The counting sort is stable: rows of one expert appear in ascending flat
// index t*k + j.  Every step is integer work, so results are bit-identical
// run to run.
#include "moe.cuh"
#include "launch.cuh"

namespace mpm {

constexpr int kSegChunk = 512;    // flat (token, slot) pairs per chunk (one warp each)

// 1) per-chunk expert histogram: hist[chunk][e]
__global__ void __launch_bounds__(256) seg_hist_kernel(const int* ids, long long n, int E,
                                                      int* hist, int* st) {
  extern __shared__ int h[];
  for (int e = threadIdx.x; e < E; e += blockDim.x) h[e] = 0;
  __syncthreads();
  const long long base = (long long)blockIdx.x * kSegChunk;
  for (int i = threadIdx.x; i < kSegChunk; i += blockDim.x) {
    const long long f = base + i;
    if (f >= n) break;
    const int e = ids[f];
    if (e >= 0 && e < E) atomicAdd(&h[e], 1);
    else set_status(st, MPM_ERR_DEVICE_BOUNDS);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) hist[(long long)blockIdx.x * E + e] = h[e];
}

// 2a) one CTA per expert: exclusive prefix of the expert's column of the
//     histogram over the chunks (each thread sums a run of chunks, then a
//     block scan of the thread sums): base[chunk][e] relative to the
//     segment start, and the expert's total
__global__ void __launch_bounds__(256) seg_colscan_kernel(const int* __restrict__ hist, int nchunks,
                                                         int E, int* __restrict__ base,
                                                         int* __restrict__ totals) {
  __shared__ int warp_sum[8];
  const int e = blockIdx.x;
  const int per = (nchunks + 255) / 256;
  const int c0 = threadIdx.x * per;
  const int c1 = min(c0 + per, nchunks);
  int local = 0;
  for (int c = c0; c < c1; ++c) local += hist[(long long)c * E + e];
  // block exclusive scan of the 256 thread sums
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[w] = incl;
  __syncthreads();
  int woff = 0;
  for (int i = 0; i < w; ++i) woff += warp_sum[i];
  int run = woff + incl - local;                 // exclusive prefix of this thread's run
  for (int c = c0; c < c1; ++c) {
    const int v = hist[(long long)c * E + e];
    base[(long long)c * E + e] = run;
    run += v;
  }
  if (threadIdx.x == 255) totals[e] = woff + incl;
}

// 2b) one CTA: padded segment offsets from the expert totals (exclusive scan)
__global__ void __launch_bounds__(1024) seg_offsets_kernel(const int* __restrict__ totals, int E,
                                                          int pad, int* __restrict__ seg_offsets) {
  __shared__ int padded[1024];
  const int e = threadIdx.x;
  const int mine = (e < E) ? (totals[e] + pad - 1) / pad * pad : 0;
  padded[e] = mine;
  __syncthreads();
  // Hillis-Steele inclusive scan over padded sizes
  for (int o = 1; o < 1024; o <<= 1) {
    const int v = (e >= o) ? padded[e - o] : 0;
    __syncthreads();
    padded[e] += v;
    __syncthreads();
  }
  if (e < E) seg_offsets[e] = padded[e] - mine;
  if (e == E - 1) seg_offsets[E] = padded[e];
}

// 3) stable scatter: one warp walks its chunk in order, 32 pairs at a time
__global__ void __launch_bounds__(32) seg_scatter_kernel(const int* ids, const float* prob,
                                                        long long n, int E, const int* base,
                                                        const int* seg_offsets, int* perm,
                                                        int* inv_perm, float* row_prob) {
  extern __shared__ int cnt[];
  const int lane = threadIdx.x;
  for (int e = lane; e < E; e += 32) cnt[e] = base[(long long)blockIdx.x * E + e] + seg_offsets[e];
  __syncwarp();
  const long long c0 = (long long)blockIdx.x * kSegChunk;
  for (int s = 0; s < kSegChunk; s += 32) {
    const long long f = c0 + s + lane;
    int e = -1;
    if (f < n) {
      e = ids[f];
      if (e < 0 || e >= E) e = -1;
    }
    const unsigned grp = __match_any_sync(0xFFFFFFFFu, e);
    const unsigned lt = (1u << lane) - 1u;
    const int rank = __popc(grp & lt);
    int row = -1;
    if (e >= 0) row = cnt[e] + rank;
    __syncwarp();
    if (e >= 0 && (grp >> lane) == 1u) cnt[e] += __popc(grp);   // highest lane of group
    __syncwarp();
    if (f < n) {
      inv_perm[f] = row;
      if (row >= 0) {
        perm[row] = (int)f;
        row_prob[row] = prob[f];
      }
    }
    if (c0 + s + 32 >= n) break;
  }
}

// ---------------------------------------------------------------- one cooperative kernel
// The same four steps (histogram, per-expert column scan, padded offsets,
// stable scatter) in one persistent launch whose CTAs meet at two grid
// barriers: at these sizes the separate launches cost more than their work
// (about 46 us for any T).  The kernel is launched cooperatively, so every
// CTA is resident; a barrier wait is bounded and, past the limit, records
// MPM_ERR_DEVICE_TIMEOUT and leaves the kernel.  The results are those of the
// four kernels above, bit for bit: the same chunks, the same scans, the same
// per-chunk stable scatter.
struct SegFused {
  const int* ids; const float* prob;
  long long n; int E; int pad; int nchunks;
  int* hist; int* base; int* totals;
  int* seg_offsets; int* perm; int* inv_perm; float* row_prob; long long cap;
  unsigned* bar;            // [2]: arrival count, generation (zeroed by the launcher)
  int* st;
};

// grid-wide barrier: the last CTA to arrive resets the count and bumps the
// generation; the others wait for the generation to move (bounded)
MPM_DEV bool seg_grid_sync(unsigned* bar, int* st) {
  __syncthreads();
  __shared__ int ok;
  if (threadIdx.x == 0) {
    ok = 1;
    volatile unsigned* gen = bar + 1;
    const unsigned g0 = *gen;
    __threadfence();
    if (atomicAdd(bar, 1u) == gridDim.x - 1) {
      atomicExch(bar, 0u);
      __threadfence();
      atomicAdd(bar + 1, 1u);
    } else {
      long long n = 0;
      while (*gen == g0) {
        if (++n > (1ll << 26)) { set_status(st, MPM_ERR_DEVICE_TIMEOUT); ok = 0; break; }
        __nanosleep(32);
      }
    }
    __threadfence();
  }
  __syncthreads();
  return ok != 0;
}

__global__ void __launch_bounds__(256) seg_fused_kernel(const SegFused a) {
  extern __shared__ int sh[];                  // max(E, 8 E) ints
  const int E = a.E;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // phase 0: clear the permuted buffers, per-chunk histograms
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < a.cap;
       i += (long long)gridDim.x * blockDim.x) {
    a.perm[i] = -1;
    a.row_prob[i] = 0.0f;
  }
  for (int c = blockIdx.x; c < a.nchunks; c += gridDim.x) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) sh[e] = 0;
    __syncthreads();
    const long long base = (long long)c * kSegChunk;
    for (int i = threadIdx.x; i < kSegChunk; i += blockDim.x) {
      const long long f = base + i;
      if (f >= a.n) break;
      const int e = a.ids[f];
      if (e >= 0 && e < E) atomicAdd(&sh[e], 1);
      else set_status(a.st, MPM_ERR_DEVICE_BOUNDS);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) a.hist[(long long)c * E + e] = sh[e];
    __syncthreads();
  }
  if (!seg_grid_sync(a.bar, a.st)) return;
  // phase 1: per-expert exclusive scan over the chunks (as seg_colscan_kernel);
  // data other CTAs wrote before a barrier is read from L2 (__ldcg)
  for (int e = blockIdx.x; e < E; e += gridDim.x) {
    const int per = (a.nchunks + 255) / 256;
    const int c0 = threadIdx.x * per;
    const int c1 = min(c0 + per, a.nchunks);
    int local = 0;
    for (int c = c0; c < c1; ++c) local += __ldcg(a.hist + (long long)c * E + e);
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sh[warp] = incl;
    __syncthreads();
    int woff = 0;
    for (int i = 0; i < warp; ++i) woff += sh[i];
    int run = woff + incl - local;
    for (int c = c0; c < c1; ++c) {
      const int v = __ldcg(a.hist + (long long)c * E + e);
      a.base[(long long)c * E + e] = run;
      run += v;
    }
    if (threadIdx.x == 255) a.totals[e] = woff + incl;
    __syncthreads();
  }
  if (!seg_grid_sync(a.bar, a.st)) return;
  // phase 2: padded offsets, computed by every CTA from the totals (block
  // scan over E <= 1024 values: 4 per thread), written by CTA 0
  {
    int v[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = threadIdx.x * 4 + i;
      v[i] = e < E ? (__ldcg(a.totals + e) + a.pad - 1) / a.pad * a.pad : 0;
      sum += v[i];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == 31) sh[warp] = incl;
    __syncthreads();
    int woff = 0;
    for (int i = 0; i < warp; ++i) woff += sh[i];
    int run = woff + incl - sum;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = threadIdx.x * 4 + i;
      if (e < E) {
        sh[e] = run;                             // this CTA's copy of seg_offsets[e]
        if (blockIdx.x == 0) a.seg_offsets[e] = run;
      }
      run += v[i];
    }
    if (blockIdx.x == 0 && threadIdx.x == 255) a.seg_offsets[E] = run;
    __syncthreads();
  }
  // phase 3: stable scatter, one warp per chunk (as seg_scatter_kernel), the
  // warp's counters after the offsets in shared memory
  int* cnt = sh + E + warp * E;
  constexpr int kSteps = kSegChunk / 32;
  for (int c = blockIdx.x * 8 + warp; c < a.nchunks; c += gridDim.x * 8) {
    const long long c0 = (long long)c * kSegChunk;
    // the chunk's expert ids and router weights are loaded up front (all
    // in flight at once), so the ordered walk below waits on no load
    int ids_r[kSteps];
    float prob_r[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const long long f = c0 + s * 32 + lane;
      ids_r[s] = f < a.n ? a.ids[f] : -1;
      prob_r[s] = f < a.n ? a.prob[f] : 0.0f;
    }
    for (int e = lane; e < E; e += 32) cnt[e] = __ldcg(a.base + (long long)c * E + e) + sh[e];
    __syncwarp();
#pragma unroll
    for (int si = 0; si < kSteps; ++si) {
      const int s = si * 32;
      const long long f = c0 + s + lane;
      int e = -1;
      if (f < a.n) {
        e = ids_r[si];
        if (e < 0 || e >= E) e = -1;
      }
      const unsigned grp = __match_any_sync(0xFFFFFFFFu, e);
      const unsigned lt = (1u << lane) - 1u;
      const int rank = __popc(grp & lt);
      int row = -1;
      if (e >= 0) row = cnt[e] + rank;
      __syncwarp();
      if (e >= 0 && (grp >> lane) == 1u) cnt[e] += __popc(grp);
      __syncwarp();
      if (f < a.n) {
        a.inv_perm[f] = row;
        if (row >= 0) {
          a.perm[row] = (int)f;
          a.row_prob[row] = prob_r[si];
        }
      }
    }
    __syncwarp();
  }
}

// ---------------------------------------------------------------- gather
// dst[row] = src[perm[row] / k] (bf16 rows), zeros for padding rows
__global__ void __launch_bounds__(256) gather_bf16_kernel(const uint4* src, long long K8,
                                                         int k, const int* perm,
                                                         const int* seg_end, long long cap,
                                                         uint4* dst, float* amax_zero) {
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  long long rend = *seg_end;
  if (rend > cap) rend = cap;
  if (row >= rend) return;
  if (amax_zero && lane == 0) amax_zero[row] = 0.0f;
  const int f = perm[row];
  uint4* d = dst + row * K8;
  if (f < 0) {
    for (long long i = lane; i < K8; i += 32) d[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  const uint4* s = src + (long long)(f / k) * K8;
  for (long long i = lane; i < K8; i += 32) d[i] = __ldg(s + i);
}

// NVFP4 rows: codes (K/2 bytes), 128x4-tiled scales (K/16 columns) and the
// token scale move together.  One CTA per 128 destination rows (one row of
// scale tiles): each warp copies 16 rows of codes; each 512-byte scale tile of
// the destination is assembled by 128 threads, one 4-byte word (a row's four
// scales of the tile) each, and written as one contiguous 512-byte run.
__global__ void __launch_bounds__(256) gather_nvfp4_kernel(const uint4* __restrict__ src_q,
                                                          const uint8_t* __restrict__ src_s,
                                                          const float* __restrict__ src_ts, long long K,
                                                          int k, const int* __restrict__ perm,
                                                          const int* __restrict__ seg_end, long long cap,
                                                          uint4* __restrict__ dst_q,
                                                          uint8_t* __restrict__ dst_s,
                                                          float* __restrict__ dst_ts,
                                                          float* __restrict__ amax_zero) {
  __shared__ long long tok[128];                  // source token of each row, -1 for padding
  const long long rbase = (long long)blockIdx.x * 128;
  long long rend = *seg_end;
  if (rend > cap) rend = cap;
  if (rbase >= rend) return;
  const int nrows = (int)min(128LL, rend - rbase);
  if (threadIdx.x < 128) {
    const int i = threadIdx.x;
    long long t = -1;
    if (i < nrows) {
      const int f = perm[rbase + i];
      if (f >= 0) t = f / k;
      if (amax_zero) amax_zero[rbase + i] = 0.0f;
      dst_ts[rbase + i] = t >= 0 ? src_ts[t] : 0.0f;
    }
    tok[i] = t;
  }
  __syncthreads();
  const long long q16 = K / 32;                  // uint4 chunks of packed codes per row
  const long long cpad = K / 16;                 // scale columns (K % 64 == 0: no padding)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = warp; i < nrows; i += 8) {
    uint4* d = dst_q + (rbase + i) * q16;
    const long long t = tok[i];
    if (t < 0) {
#pragma unroll 4
      for (long long c = lane; c < q16; c += 32) d[c] = make_uint4(0, 0, 0, 0);
    } else {
      const uint4* sq = src_q + t * q16;
#pragma unroll 4
      for (long long c = lane; c < q16; c += 32) d[c] = __ldg(sq + c);
    }
  }
  // scale tiles: word w of a tile holds row (w % 4) * 32 + w / 4
  const long long ntiles = cpad / 4;
  const long long rt = rbase >> 7;
  const int w = threadIdx.x & 127;
  const int r = (w & 3) * 32 + (w >> 2);
  const long long t = tok[r];
#pragma unroll 4
  for (long long g = threadIdx.x >> 7; g < ntiles; g += 2) {
    if (r >= nrows) continue;
    uint32_t v = 0;
    if (t >= 0) v = *reinterpret_cast<const uint32_t*>(src_s + sf_offset(t, g * 4, cpad));
    reinterpret_cast<uint32_t*>(dst_s + (rt * ntiles + g) * 512)[w] = v;
  }
}

// MXFP8 rows: codes (K bytes) and 128x4-tiled E8M0 scales (K/32 columns).  Two
// kinds of blocks, since a row's codes are one run and its scales one word in
// each of K/128 tiles that it shares with 127 rows: the first code_blocks copy
// 2 KB of the codes of 16 rows each (two rows a warp, all eight 16-byte loads of
// a lane in flight together); the others write whole runs of up to 8 scale tiles
// of 128 rows, one word (a row's four scales of a tile) per thread and tile.
// Bound by the bytes, K (1 + 1/32) written a row and a token's row read once from
// DRAM (its k copies come from L2): 8192 tokens x 8 x 2048 take 31.0 us, 6.2 TB/s
// and 0.91 of the measured copy; 64 x 8 x 7168, 26 MB written in 16-row segments
// (mostly padding), 5.4 us, 4 by its bytes.  STREAM, for outputs that L2 cannot
// hold: codes stored to leave it first, so that the tokens' rows stay (33.5 us
// without; a smaller output is left there for the GEMM that reads it next).  Codes and scales of 128 rows in one
// block took 39.2 and 24 us: too few loads in flight, too few blocks for 64
// tokens.  Bulk copies through shared memory, a row a lane: 35.9 and 5.3 us.
constexpr int kGatherRows = 16, kGatherTiles = 8, kGatherChunk = 128;   // 16-byte words

template <bool STREAM>
__global__ void __launch_bounds__(256) gather_mxfp8_kernel(const uint4* __restrict__ src_q,
                                                          const uint8_t* __restrict__ src_s,
                                                          int T, long long K, int k,
                                                          const int* __restrict__ perm,
                                                          const int* __restrict__ seg_end,
                                                          long long cap, long long code_blocks,
                                                          uint4* __restrict__ dst_q,
                                                          uint8_t* __restrict__ dst_s, int* st) {
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x < code_blocks) {
    const int q16 = (int)(K / 16);               // 16-byte words of codes per row
    const unsigned row_blocks = (unsigned)((cap + kGatherRows - 1) / kGatherRows);
    const unsigned chunk = blockIdx.x / row_blocks;
    const long long r0 = (long long)(blockIdx.x - chunk * row_blocks) * kGatherRows + warp * 2;
    const int c0 = (int)chunk * kGatherChunk + lane;
    int f[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) f[i] = r0 + i < cap ? perm[r0 + i] : -1;
    const long long rend = min((long long)*seg_end, cap);
    uint4 v[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int t = f[i] >= 0 ? f[i] / k : -1;
      if (t >= T) {
        if (lane == 0 && r0 + i < rend) set_status(st, MPM_ERR_DEVICE_BOUNDS);
        t = -1;
      }
      const uint4* s = src_q + (long long)max(t, 0) * q16;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[i][j] = make_uint4(0, 0, 0, 0);
        if (t >= 0 && c0 + 32 * j < q16) v[i][j] = __ldg(s + c0 + 32 * j);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint4* d = dst_q + (r0 + i) * q16;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (r0 + i < rend && c0 + 32 * j < q16) {
          if (STREAM) __stcs(d + c0 + 32 * j, v[i][j]);
          else d[c0 + 32 * j] = v[i][j];
        }
    }
    return;
  }
  // word w of a tile holds row (w % 4) * 32 + w / 4
  const long long cpad = (K / 32 + 3) / 4 * 4, ntiles = cpad / 4;
  const long long groups = (ntiles + kGatherTiles - 1) / kGatherTiles;
  const long long b = blockIdx.x - code_blocks, rt = b / groups, g0 = (b - rt * groups) * kGatherTiles;
  const int w = threadIdx.x & 127;
  const long long row = rt * 128 + (w & 3) * 32 + (w >> 2);
  const int f = row < cap ? perm[row] : -1;
  if (row >= min((long long)*seg_end, cap)) return;
  int t = f >= 0 ? f / k : -1;
  if (t >= T) t = -1;                            // reported by the row's code block
  uint32_t v[kGatherTiles / 2];
#pragma unroll
  for (int j = 0; j < kGatherTiles / 2; ++j) {
    const long long g = g0 + (threadIdx.x >> 7) + 2 * j;
    v[j] = 0;
    if (t >= 0 && g < ntiles) v[j] = *reinterpret_cast<const uint32_t*>(src_s + sf_offset(t, g * 4, cpad));
  }
#pragma unroll
  for (int j = 0; j < kGatherTiles / 2; ++j) {
    const long long g = g0 + (threadIdx.x >> 7) + 2 * j;
    if (g < ntiles) reinterpret_cast<uint32_t*>(dst_s + (rt * ntiles + g) * 512)[w] = v[j];
  }
}

// ---------------------------------------------------------------- combine
// out[t] = sum_j y[inv[t*k + j]] in fp32, slot order, one rounding to bf16
__global__ void __launch_bounds__(128) combine_kernel(const uint4* y, const int* inv, long long T,
                                                     int k, long long H8, uint4* out) {
  const long long c = (long long)blockIdx.y * blockDim.x + threadIdx.x;
  const long long t = blockIdx.x;
  if (c >= H8) return;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  for (int j = 0; j < k; ++j) {
    const int r = inv[t * k + j];
    if (r < 0) continue;
    const uint4 v = __ldg(y + (long long)r * H8 + c);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[2 * i] = __fadd_rn(acc[2 * i], bf16lo(w[i]));
      acc[2 * i + 1] = __fadd_rn(acc[2 * i + 1], bf16hi(w[i]));
    }
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 b = __floats2bfloat162_rn(acc[2 * i], acc[2 * i + 1]);
    o[i] = *reinterpret_cast<uint32_t*>(&b);
  }
  out[t * H8 + c] = make_uint4(o[0], o[1], o[2], o[3]);
}

// ---------------------------------------------------------------- gradient of the routing weights
// out[t] = sum_j y[inv[t k + j]] and y of a slot is linear in its weight p (the
// FC1 epilogue multiplies D by p), so d out[t] / d p_j = y / p_j and
//   dprob[t, j] = <dout[t], y[inv[t k + j]]> / p_j.
// A slot without a row (inv < 0) and a weight of 0 get 0: a weight of 0 comes
// from a score of 0 (or a masked token), whose own gradient is 0.
//
// P warps share a slot's row (P = 1 up to 2048 columns, so that a lane takes at
// most 8 words of it), 8 / P slots a block: a block's slots are mostly one
// token's, whose dout row then comes from L1.  (One block per token, reading
// dout once, was slower, 75.6 against 49 us at 8192 x 8 x 2048: its barrier and
// its 80 registers left too little in flight.)  Bound by the bytes of y, 2 H a
// slot: that size takes 48.4 us, 6.3 TB/s and 0.92 of the measured copy; 257 x 6
// x 7168, read in about one round of loads, 6.7 us of which 3.8 are its bytes.
template <int P>
__global__ void __launch_bounds__(256) combine_dprob_kernel(const uint4* __restrict__ dout,
                                                           const uint4* __restrict__ y,
                                                           const int* __restrict__ inv,
                                                           const float* __restrict__ prob, int slots,
                                                           int k, int H8, long long cap, float* dprob,
                                                           int* st) {
  __shared__ float sh[8];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int f = blockIdx.x * (8 / P) + warp / P;
  const int r = f < slots ? inv[f] : -1;
  const float p = f < slots ? prob[f] : 0.0f;
  const bool live = r >= 0 && r < cap && p != 0.0f;
  if (f < slots && r >= cap && lane == 0) set_status(st, MPM_ERR_DEVICE_BOUNDS);
  float acc = 0.0f;
  if (live) {
    const uint4* a = dout + (long long)(f / k) * H8;
    const uint4* b = y + (long long)r * H8;
    constexpr int U = 2;                   // (4: 49.1, 8: 51.1 against 48.4 us at 8192 x 8 x 2048)
    for (int c0 = (warp % P) * 32 + lane; c0 < H8; c0 += U * P * 32) {
      uint4 u[U], v[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int c = c0 + i * P * 32;
        v[i] = u[i] = make_uint4(0, 0, 0, 0);
        if (c < H8) { v[i] = __ldcs(b + c); u[i] = __ldg(a + c); }
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const uint32_t uw[4] = {u[i].x, u[i].y, u[i].z, u[i].w}, vw[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc = __fmaf_rn(bf16lo(uw[j]), bf16lo(vw[j]), acc);
          acc = __fmaf_rn(bf16hi(uw[j]), bf16hi(vw[j]), acc);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc = __fadd_rn(acc, __shfl_xor_sync(0xffffffffu, acc, o));
  }
  if constexpr (P > 1) {
    if (lane == 0) sh[warp] = acc;
    __syncthreads();
    acc = 0.0f;
    for (int w = warp / P * P; w < warp / P * P + P; ++w) acc = __fadd_rn(acc, sh[w]);
  }
  if (lane == 0 && warp % P == 0 && f < slots) dprob[f] = live ? __fdiv_rn(acc, p) : 0.0f;
}

// ---------------------------------------------------------------- launchers
size_t segments_ws_bytes(long long T, int k, long long E) {
  const long long n = T * k;
  const long long nchunks = (n + kSegChunk - 1) / kSegChunk;
  // histograms, chunk bases, expert totals, the fused kernel's barrier words
  return (size_t)(2 * nchunks * E + E + 2) * sizeof(int);
}

// the cooperative form; cudaErrorNotSupported when the device cannot run it
static cudaError_t launch_segments_fused(const SegFused& a, cudaStream_t s) {
  static int ctas[64] = {0};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorNotSupported;
  const size_t smem = (size_t)9 * 1024 * sizeof(int);     // offsets + 8 warps' counters, E <= 1024
  if (ctas[dev] == 0) {
    int sms = 0, per = 0, coop = 0;
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    cudaDeviceGetAttribute(&coop, cudaDevAttrCooperativeLaunch, dev);
    err = cudaFuncSetAttribute(seg_fused_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)smem);
    if (err != cudaSuccess) return err;
    err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, seg_fused_kernel, 256, smem);
    if (err != cudaSuccess) return err;
    ctas[dev] = (coop && sms > 0 && per > 0) ? sms * (per < 2 ? per : 2) : -1;
  }
  if (ctas[dev] < 0) return cudaErrorNotSupported;
  // enough CTAs for the widest phase, no more than can be resident
  long long want = a.nchunks > a.E ? a.nchunks : a.E;
  if (want < 1) want = 1;
  const unsigned grid = (unsigned)(want < ctas[dev] ? want : ctas[dev]);
  SegFused arg = a;
  void* args[] = {&arg};
  return cudaLaunchCooperativeKernel((const void*)seg_fused_kernel, dim3(grid), dim3(256), args,
                                     smem, s);
}

cudaError_t launch_build_segments(const int* ids, const float* prob, long long T, int k,
                                  long long E, int pad, int* seg_offsets, int* perm,
                                  int* inv_perm, float* row_prob, long long cap, void* ws,
                                  int* st, cudaStream_t s) {
  const long long n = T * k;
  const int nchunks = (int)((n + kSegChunk - 1) / kSegChunk);
  int* hist = static_cast<int*>(ws);
  int* base = hist + (long long)nchunks * E;
  cudaError_t err;
  if (E <= 1024) {
    SegFused a{};
    a.ids = ids; a.prob = prob; a.n = n; a.E = (int)E; a.pad = pad; a.nchunks = nchunks;
    a.hist = hist; a.base = base; a.totals = base + (long long)nchunks * E;
    a.seg_offsets = seg_offsets; a.perm = perm; a.inv_perm = inv_perm; a.row_prob = row_prob;
    a.cap = cap;
    a.bar = reinterpret_cast<unsigned*>(a.totals + E);
    a.st = st;
    if ((err = cudaMemsetAsync(a.bar, 0, 2 * sizeof(unsigned), s)) != cudaSuccess) return err;
    err = launch_segments_fused(a, s);
    if (err != cudaErrorNotSupported) return err;
  }
  if ((err = cudaMemsetAsync(perm, 0xFF, (size_t)cap * sizeof(int), s)) != cudaSuccess) return err;
  if ((err = cudaMemsetAsync(row_prob, 0, (size_t)cap * sizeof(float), s)) != cudaSuccess) return err;
  seg_hist_kernel<<<nchunks, 128, (size_t)E * sizeof(int), s>>>(ids, n, (int)E, hist, st);
  if ((err = cudaGetLastError()) != cudaSuccess) return err;
  int* totals = base + (long long)nchunks * E;
  seg_colscan_kernel<<<(unsigned)E, 256, 0, s>>>(hist, nchunks, (int)E, base, totals);
  if ((err = cudaGetLastError()) != cudaSuccess) return err;
  seg_offsets_kernel<<<1, 1024, 0, s>>>(totals, (int)E, pad, seg_offsets);
  if ((err = cudaGetLastError()) != cudaSuccess) return err;
  seg_scatter_kernel<<<nchunks, 32, (size_t)E * sizeof(int), s>>>(ids, prob, n, (int)E, base,
                                                                  seg_offsets, perm, inv_perm,
                                                                  row_prob);
  return cudaGetLastError();
}

cudaError_t launch_gather(int what, const void* src, const uint8_t* src_s, const float* src_ts,
                          long long K, int k, const int* perm, const int* seg_end,
                          long long cap, void* dst, uint8_t* dst_s, float* dst_ts,
                          float* amax_zero, cudaStream_t s) {
  const unsigned grid = (unsigned)((cap + 7) / 8);
  if (what == MPM_GATHER_BF16) {
    gather_bf16_kernel<<<grid, 256, 0, s>>>(static_cast<const uint4*>(src), K / 8, k, perm,
                                            seg_end, cap, static_cast<uint4*>(dst), amax_zero);
  } else {
    gather_nvfp4_kernel<<<(unsigned)((cap + 127) / 128), 256, 0, s>>>(
        static_cast<const uint4*>(src), src_s, src_ts, K,
                                             k, perm, seg_end, cap, static_cast<uint4*>(dst),
                                             dst_s, dst_ts, amax_zero);
  }
  return cudaGetLastError();
}

cudaError_t launch_combine(const void* y, const int* inv, long long T, int k, long long H,
                           void* out, cudaStream_t s) {
  const long long H8 = H / 8;
  const dim3 grid((unsigned)T, (unsigned)((H8 + 127) / 128));
  combine_kernel<<<grid, 128, 0, s>>>(static_cast<const uint4*>(y), inv, T, k, H8,
                                      static_cast<uint4*>(out));
  return cudaGetLastError();
}

cudaError_t launch_gather_mxfp8(const uint8_t* q, const uint8_t* sc, long long T, long long K, int k,
                                const int* perm, const int* seg_end, long long cap, uint8_t* dst_q,
                                uint8_t* dst_s, int* status, cudaStream_t s) {
  const long long chunks = (K / 16 + kGatherChunk - 1) / kGatherChunk;
  const long long code_blocks = (cap + kGatherRows - 1) / kGatherRows * chunks;
  const long long ntiles = (K / 32 + 3) / 4, groups = (ntiles + kGatherTiles - 1) / kGatherTiles;
  const long long blocks = code_blocks + (cap + 127) / 128 * groups;
  if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const auto kernel = cap * K > (96ll << 20) ? gather_mxfp8_kernel<true> : gather_mxfp8_kernel<false>;
  return launch_serial(kernel, dim3((unsigned)blocks), dim3(256), 0, s,
                       reinterpret_cast<const uint4*>(q), sc, (int)T, K, k, perm, seg_end, cap,
                       code_blocks, reinterpret_cast<uint4*>(dst_q), dst_s, status);
}

cudaError_t launch_combine_dprob(const void* dout, const void* y, const int* inv, const float* prob,
                                 long long T, int k, long long H, long long cap, float* dprob,
                                 int* status, cudaStream_t s) {
  const int H8 = (int)(H / 8), slots = (int)(T * k);       // T k <= 2^30
  const int p = H8 <= 256 ? 1 : (H8 <= 512 ? 2 : (H8 <= 1024 ? 4 : 8));
  const auto kernel = p == 1 ? combine_dprob_kernel<1> : p == 2 ? combine_dprob_kernel<2>
                    : p == 4 ? combine_dprob_kernel<4> : combine_dprob_kernel<8>;
  return launch_serial(kernel, dim3((unsigned)((slots + 8 / p - 1) / (8 / p))), dim3(256), 0, s,
                       static_cast<const uint4*>(dout), static_cast<const uint4*>(y), inv, prob, slots, k,
                       H8, cap, dprob, status);
}

}  // namespace mpm
