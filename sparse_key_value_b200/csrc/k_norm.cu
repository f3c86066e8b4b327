// k_norm.cu -- the residual's addition and the root-mean-square norm in front
// of a memory layer, with its output in 16 (or 32) and in 8 bits, and its
// backward.
//
// Forward, per row: h = x + r rounded to the storage type (the value the rest
// of the network sees, so the backward differentiates the same one),
// rstd = (mean h^2 + eps)^-1/2, y = h rstd w.  The 8-bit copy is rounded from
// the fp32 y, not from its 16-bit rounding.
// Backward: n = h rstd, g = dy w, dx = rstd (g - n mean(g n)) + dsum,
// dweight = sum over rows of dy n.
//
// Both are bound by memory: every tensor is read or written once, a row stays
// in registers between its sum and its outputs.  A row belongs to WPR warps,
// each lane holding NU units of 8 columns; 16 consecutive lanes hold a
// quantisation group.
// Measured on one B200: forward of 16384 x 1024 bf16 with a residual, both
// outputs and the 8-bit copy 24 us (151 MB: 6.2 TB/s); backward of 8191 x 2048
// bf16 with a second gradient 27.1 us with the weight gradient's join (134 MB:
// 5.0 TB/s; the join and its launch take 3), from an 8-bit h 27.0 (118 MB: DRAM at
// 42 % of its peak; with four warps a scheduler, which decode what they read,
// instructions issue in 55 % of the cycles, and a fifth of a warp's wait is for
// its row's sum).
#include <type_traits>

#include "kernels.h"
#include "q8.cuh"

namespace pkm {

namespace {

constexpr int kNormThreads = 256;

constexpr int block_threads(int wpr) { return wpr * 32 > kNormThreads ? wpr * 32 : kNormThreads; }

// Sum over the row's WPR warps (consecutive ones, a named barrier of their
// own; `red` [2][warps], used in turn: the barrier of the next sum follows
// every read of this one).  Fixed order: the same bits every run.
template <int WPR, int WARPS = block_threads(WPR) / 32>
__device__ __forceinline__ float row_sum(float v, float* red, int turn) {
  v = warp_sum(v);
  if constexpr (WPR > 1) {
    const int warp = threadIdx.x >> 5;
    float* r = red + (turn & 1) * WARPS;
    if ((threadIdx.x & 31) == 0) r[warp] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / WPR), "n"(32 * WPR) : "memory");
    v = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) v += r[warp / WPR * WPR + w];
  }
  return v;
}

__device__ __forceinline__ void bulk_load(void* to, const void* from, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(smem_u32(to)), "l"(from), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

struct NormFwd {
  int64_t T;
  int d;
  float eps;
  pkm_q8 fmt;
  const void *x, *r, *w;
  void *sum, *y;
  uint8_t* y8;
  float *scales, *rstd;
};

template <pkm_dtype DT, int NU, int WPR>
__global__ void __launch_bounds__(block_threads(WPR)) norm_fwd_kernel(const NormFwd p) {
  using E = typename Elem<DT>::T;
  __shared__ float red[2 * block_threads(WPR) / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kRows = block_threads(WPR) / 32 / WPR;
  const int64_t row = (int64_t)blockIdx.x * kRows + warp / WPR;
  const bool live = row < p.T;
  const int col0 = ((warp % WPR) * 32 + lane) * kUnit;
  const int64_t base = row * p.d;
  float h[NU][8];
  float ss = 0.f;
  {
    Raw8<DT> x[NU], r[NU];
#pragma unroll
    for (int c = 0; c < NU; ++c) {
      const int col = col0 + c * (WPR * 32 * kUnit);
      x[c].zero();
      if (live && col < p.d) {
        x[c].load(static_cast<const E*>(p.x) + base + col);
        if (p.r) r[c].load(static_cast<const E*>(p.r) + base + col);
      }
    }
#pragma unroll
    for (int c = 0; c < NU; ++c) {
      x[c].unpack(h[c]);
      if (p.r && live && col0 + c * (WPR * 32 * kUnit) < p.d) {
        float f[8];
        r[c].unpack(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[c][e] += f[e];
        round8<DT>(h[c]);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < NU; ++c) {
    const int col = col0 + c * (WPR * 32 * kUnit);
    if (p.sum && live && col < p.d) store8<DT>(static_cast<E*>(p.sum) + base + col, h[c]);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(h[c][e], h[c][e], ss);
  }
  ss = row_sum<WPR>(ss, red, 0);
  const float rstd = 1.0f / sqrtf(ss / (float)p.d + p.eps);
  if (live && p.rstd && col0 == 0) p.rstd[row] = rstd;
  const int groups = q8_groups(p.d);
#pragma unroll
  for (int c = 0; c < NU; ++c) {
    const int col = col0 + c * (WPR * 32 * kUnit);
    const bool in = live && col < p.d;
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.f;
    if (p.w && in) load8<DT>(static_cast<const E*>(p.w) + col, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[c][e] = h[c][e] * rstd * w[e];
    if (p.y && in) store8<DT>(static_cast<E*>(p.y) + base + col, h[c]);
    if (p.y8) {
      if (!in) {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[c][e] = 0.f;
      }
      const float s = q8_scale(group_amax_bits(h[c]), p.fmt);
      if (in) {
        *reinterpret_cast<uint2*>(p.y8 + base + col) = q8_encode(h[c], q8_inverse(s), p.fmt);
        if (lane % kGroupLanes == 0) p.scales[row * groups + col / kQ8Group] = s;
      }
    }
  }
}

struct NormBwd {
  int64_t T;
  int d;
  pkm_q8 fmt;  // PKM_Q8_NONE: h in the storage type
  const void *dy, *h, *w, *dsum;
  const float *scales, *rstd;
  void* dx;
  float* part;  // [blocks, d] weight-gradient partials, or null
};

// Blocks of the backward per SM.
constexpr int bwd_per_sm(int wpr) { return block_threads(wpr) <= 256 ? 3 : 1; }

// DY: type of dy; DT: type of h (when not 8-bit), weight, dsum and dx.  A
// row's dy, h and dsum wait packed in registers, all loaded up front: the
// blocks of an SM then keep about 75 KB of loads in flight.
template <pkm_dtype DT, pkm_dtype DY, int NU, int WPR>
__global__ void __launch_bounds__(block_threads(WPR), bwd_per_sm(WPR))
    norm_bwd_kernel(const NormBwd p) {
  using E = typename Elem<DT>::T;
  using Ey = typename Elem<DY>::T;
  constexpr int kWarps = block_threads(WPR) / 32;
  constexpr int kTeams = kWarps / WPR;  // rows in flight per block
  __shared__ float red[2 * kWarps];
  int turn = 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int team = warp / WPR;
  const int col0 = ((warp % WPR) * 32 + lane) * kUnit;
  const int groups = q8_groups(p.d);
  pdl_launch_dependents();
  pdl_wait();
  float dw[NU][8];
#pragma unroll
  for (int c = 0; c < NU; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[c][e] = 0.f;
  // every team of the block makes the same number of rounds (row_sum syncs)
  for (int64_t r0 = (int64_t)blockIdx.x * kTeams; r0 < p.T; r0 += (int64_t)gridDim.x * kTeams) {
    const int64_t row = r0 + team;
    const bool live = row < p.T;
    const int64_t base = row * p.d;
    const float rstd = live ? p.rstd[row] : 0.f;
    Raw8<DY> dy[NU];
    Raw8<DT> h[NU], ds[NU];
    float hs[NU];  // 8-bit h: its scale (the bytes wait in h)
#pragma unroll
    for (int c = 0; c < NU; ++c) {
      const int col = col0 + c * (WPR * 32 * kUnit);
      dy[c].zero();
      h[c].zero();
      ds[c].zero();
      hs[c] = 0.f;
      if (live && col < p.d) {
        dy[c].load(static_cast<const Ey*>(p.dy) + base + col);
        if (p.fmt == PKM_Q8_NONE) {
          h[c].load(static_cast<const E*>(p.h) + base + col);
        } else {
          const uint2 q =
              *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.h) + base + col);
          h[c].v[0].x = q.x;
          h[c].v[0].y = q.y;
          hs[c] = p.scales[row * groups + col / kQ8Group];
        }
        if (p.dsum) ds[c].load(static_cast<const E*>(p.dsum) + base + col);
      }
    }
    auto unpack = [&](int c, float* g, float* n) {  // g = dy w, n = h rstd
      if (p.fmt == PKM_Q8_NONE)
        h[c].unpack(n);
      else
        q8_decode(make_uint2(h[c].v[0].x, h[c].v[0].y), hs[c], p.fmt, n);
      dy[c].unpack(g);
      const int col = col0 + c * (WPR * 32 * kUnit);
#pragma unroll
      for (int e = 0; e < 8; ++e) n[e] *= rstd;
      return col;
    };
    auto weigh = [&](int col, float* g) {
      if (p.w && col < p.d) {
        float w[8];
        load8<DT>(static_cast<const E*>(p.w) + col, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] *= w[e];
      }
    };
    float dot = 0.f;
#pragma unroll
    for (int c = 0; c < NU; ++c) {
      float g[8], n[8];
      const int col = unpack(c, g, n);
#pragma unroll
      for (int e = 0; e < 8; ++e) dw[c][e] = fmaf(g[e], n[e], dw[c][e]);
      weigh(col, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) dot = fmaf(g[e], n[e], dot);
    }
    const float mean = row_sum<WPR>(dot, red, turn++) / (float)p.d;
#pragma unroll
    for (int c = 0; c < NU; ++c) {
      float g[8], n[8], o[8];
      const int col = unpack(c, g, n);
      if (!(live && col < p.d)) continue;
      weigh(col, g);
      ds[c].unpack(o);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] += rstd * (g[e] - n[e] * mean);
      store8<DT>(static_cast<E*>(p.dx) + base + col, o);
    }
  }
  if (!p.part) return;
  // the block's teams in order, then one partial row per block
  __shared__ float acc[kTeams > 1 ? kTeams - 1 : 1][NU * WPR * 32 * kUnit];
  if (team > 0) {
#pragma unroll
    for (int c = 0; c < NU; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        acc[team - 1][col0 + c * (WPR * 32 * kUnit) + e] = dw[c][e];
  }
  __syncthreads();
  if (team == 0) {
#pragma unroll
    for (int c = 0; c < NU; ++c) {
      const int col = col0 + c * (WPR * 32 * kUnit);
      if (col >= p.d) continue;
#pragma unroll
      for (int t = 1; t < kTeams; ++t)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[c][e] += acc[t - 1][col + e];
      store8<PKM_F32>(p.part + (int64_t)blockIdx.x * p.d + col, dw[c]);
    }
  }
}

// The backward of long batches: a row's tensors come by bulk
// copies into a ring of shared memory, so that up to 200 KB per SM are on their
// way while rows are summed and written; registers hold a row only while it is
// worked on.  One block per SM, kRingWarps / WPR teams of a row each, a ring of
// up to kRingStages rows per team; the team's leader refills a place after the
// row's sum, whose barrier follows the team's last read of it.
// Against the rows straight into registers (bf16, second gradient, us): 8191 x
// 2048 27.1 and 30.7, 4096 x 4096 27.2 and 34.8, 2048 x 8192 27.6 and 38.4, 30000
// x 512 26.6 and 29.9; 40000 x 256 20.6 and 21.1, 100000 x 64 39.1 and 38.9;
// int8 h: 8191 x 2048 27.0 and 30.8, 4096 x 4096 27.0 and 34.7.  20 warps took
// 28.9 at the first (12 rounds of rows for 11.1), 12 with a deeper ring 27.1 but
// 38.4 at the third.
constexpr int kRingWarps = 16, kRingStages = 4;
constexpr int kRingBytes = 200 * 1024;
constexpr int ring_teams(int wpr) { return kRingWarps / wpr; }

template <pkm_dtype DT, pkm_dtype DY, int NU, int WPR, bool Q8>
__global__ void __launch_bounds__(32 * WPR * ring_teams(WPR), 1)
    norm_bwd_ring_kernel(const NormBwd p, int stages, int32_t* status) {
  using E = typename Elem<DT>::T;
  using Ey = typename Elem<DY>::T;
  constexpr int kTeams = ring_teams(WPR), kWarps = WPR * kTeams;
  extern __shared__ __align__(128) unsigned char ring_raw[];
  __shared__ __align__(8) uint64_t full[kTeams][kRingStages];
  __shared__ float red[2 * kWarps];
  __shared__ volatile int abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int team = warp / WPR;
  const int col0 = ((warp % WPR) * 32 + lane) * kUnit;
  const bool leads = threadIdx.x == team * WPR * 32;
  const int d = p.d;
  const uint32_t ny = (uint32_t)d * sizeof(Ey), ns = p.dsum ? (uint32_t)d * sizeof(E) : 0;
  const uint32_t nh = Q8 ? (uint32_t)d : (uint32_t)d * sizeof(E);
  const uint32_t row_bytes = ny + nh + ns;
  unsigned char* ring = ring_raw + (size_t)team * stages * row_bytes;
  if (threadIdx.x == 0) {
    for (int t = 0; t < kTeams; ++t)
      for (int i = 0; i < kRingStages; ++i) mbar_init(&full[t][i], 1);
    abort = 0;
    fence_barrier_init();
  }
  __syncthreads();
  pdl_launch_dependents();
  pdl_wait();
  const int64_t step = (int64_t)gridDim.x * kTeams;
  const int64_t row0 = (int64_t)blockIdx.x * kTeams + team;
  auto copy = [&](int64_t row, int place) {  // the leader's
    unsigned char* to = ring + (size_t)place * row_bytes;
    uint64_t* bar = &full[team][place];
    mbar_arrive_expect_tx(bar, row_bytes);
    bulk_load(to, static_cast<const Ey*>(p.dy) + row * d, ny, bar);
    bulk_load(to + ny, static_cast<const uint8_t*>(p.h) + row * nh, nh, bar);
    if (ns) bulk_load(to + ny + nh, static_cast<const E*>(p.dsum) + row * d, ns, bar);
  };
  if (leads)
    for (int i = 0; i < stages && row0 + i * step < p.T; ++i) copy(row0 + i * step, i);
  Raw8<DT> w[NU];
#pragma unroll
  for (int c = 0; c < NU; ++c) {
    const int col = col0 + c * (WPR * 32 * kUnit);
    if (p.w && col < d) w[c].load(static_cast<const E*>(p.w) + col);
  }
  float dw[NU][8];
#pragma unroll
  for (int c = 0; c < NU; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[c][e] = 0.f;
  // a row's rstd, with 8-bit h its scales too, are read a turn ahead
  float rstd = row0 < p.T ? p.rstd[row0] : 0.f;
  const int groups = q8_groups(d);
  auto scale_of = [&](int64_t row, int c) {
    const int col = col0 + c * (WPR * 32 * kUnit);
    return Q8 && row < p.T && col < d ? p.scales[row * groups + col / kQ8Group] : 0.f;
  };
  float next[NU];
#pragma unroll
  for (int c = 0; c < NU; ++c) next[c] = scale_of(row0, c);
  int place = 0, turn = 0;
  uint32_t parity = 0;
  bool ok = true;
  for (int64_t row = row0; row < p.T; row += step) {
    const float rs = rstd;
    if (row + step < p.T) rstd = p.rstd[row + step];
    float hs[NU];
#pragma unroll
    for (int c = 0; c < NU; ++c) {
      hs[c] = next[c];
      next[c] = scale_of(row + step, c);
    }
    ok = ok && mbar_wait_or_abort(&full[team][place], parity, &abort, status);
    const unsigned char* at = ring + (size_t)place * row_bytes;
    Raw8<DY> dy[NU];
    Raw8<DT> h[NU], ds[NU];
#pragma unroll
    for (int c = 0; c < NU; ++c) {
      const int col = col0 + c * (WPR * 32 * kUnit);
      dy[c].zero();
      h[c].zero();
      ds[c].zero();
      if (col < d) {
        dy[c].load(reinterpret_cast<const Ey*>(at) + col);
        if constexpr (Q8) {
          const uint2 q = *reinterpret_cast<const uint2*>(at + ny + col);
          h[c].v[0].x = q.x;
          h[c].v[0].y = q.y;
        } else {
          h[c].load(reinterpret_cast<const E*>(at + ny) + col);
        }
        if (ns) ds[c].load(reinterpret_cast<const E*>(at + ny + nh) + col);
      }
    }
    float hv[Q8 ? NU : 1][8];  // 8-bit h as numbers: decoded once, used twice
    if constexpr (Q8) {
#pragma unroll
      for (int c = 0; c < NU; ++c)
        q8_decode(make_uint2(h[c].v[0].x, h[c].v[0].y), hs[c], p.fmt, hv[c]);
    }
    auto value = [&](int c, float* n) {
      if constexpr (Q8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) n[e] = hv[c][e];
      } else {
        h[c].unpack(n);
      }
    };
    auto weigh = [&](int c, float* g) {
      if (p.w && col0 + c * (WPR * 32 * kUnit) < d) {
        float f[8];
        w[c].unpack(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] *= f[e];
      }
    };
    float dot = 0.f;
#pragma unroll
    for (int c = 0; c < NU; ++c) {
      float g[8], n[8];
      value(c, n);
      dy[c].unpack(g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n[e] *= rs;
        dw[c][e] = fmaf(g[e], n[e], dw[c][e]);
      }
      weigh(c, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) dot = fmaf(g[e], n[e], dot);
    }
    const float mean = row_sum<WPR, kWarps>(dot, red, turn++) / (float)d;
    if constexpr (WPR == 1) __syncwarp();
    if (leads && ok && row + stages * step < p.T) copy(row + stages * step, place);
#pragma unroll
    for (int c = 0; c < NU; ++c) {
      const int col = col0 + c * (WPR * 32 * kUnit);
      float g[8], n[8], o[8];
      value(c, n);
      dy[c].unpack(g);
      weigh(c, g);
      ds[c].unpack(o);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] += rs * (g[e] - n[e] * rs * mean);
      if (ok && col < d) store8<DT>(static_cast<E*>(p.dx) + row * d + col, o);
    }
    if (++place == stages) {
      place = 0;
      parity ^= 1;
    }
  }
  // a team that gave up lets the copies that it was told about land
  if (leads && !ok)
    for (int i = 0; i < stages; ++i)
      for (unsigned long long k = 0; k < kSpinLimit; ++k)
        if (mbar_try_wait(&full[team][i], i < place ? parity ^ 1 : parity)) break;
  if (!p.part) return;
  __syncthreads();  // the ring is free: the teams' sums in order, one row per block
  float* acc = reinterpret_cast<float*>(ring_raw);
  constexpr int kCols = NU * WPR * 32 * kUnit;
  if (team > 0) {
#pragma unroll
    for (int c = 0; c < NU; ++c) {
      const int col = col0 + c * (WPR * 32 * kUnit);
      store8<PKM_F32>(acc + (team - 1) * kCols + col, dw[c]);
    }
  }
  __syncthreads();
  if (team == 0) {
#pragma unroll
    for (int c = 0; c < NU; ++c) {
      const int col = col0 + c * (WPR * 32 * kUnit);
      if (col >= d) continue;
#pragma unroll 4
      for (int t = 1; t < kTeams; ++t)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[c][e] += acc[(t - 1) * kCols + col + e];
      store8<PKM_F32>(p.part + (int64_t)blockIdx.x * d + col, dw[c]);
    }
  }
}

// dweight[c] = sum over blocks of part[block][c]: 32 columns per block, 16
// row strides of several loads in flight, joined in order
constexpr int kDwStrips = 16;
__global__ void __launch_bounds__(32 * kDwStrips) norm_dw_kernel(const float* __restrict__ part,
                                                                 int blocks, int d,
                                                                 float* __restrict__ dw) {
  __shared__ float s[kDwStrips][32];
  const int lane = threadIdx.x & 31, col = blockIdx.x * 32 + lane, r = threadIdx.x >> 5;
  float v = 0.f;
  pdl_wait();
  if (col < d) {
#pragma unroll 8
    for (int b = r; b < blocks; b += kDwStrips) v += part[(int64_t)b * d + col];
  }
  s[r][lane] = v;
  __syncthreads();
  if (r == 0 && col < d) {
    for (int k = 1; k < kDwStrips; ++k) v += s[k][lane];
    dw[col] = v;
  }
}

constexpr int kMaxD = 16384;
constexpr int kSMs = 148;

int rows_per_block(int wpr) { return wpr >= 8 ? 1 : 8 / wpr; }

template <int N>
using Int = std::integral_constant<int, N>;

// Units per lane and warps per row: as few warps as hold the row with UMAX
// units a lane.  The forward holds four (no barrier up to 1024 columns).  The
// backward, with three tensors and the weight gradient in registers, holds
// two of bf16 and one of fp32: three blocks per SM then have more rows in
// flight than two with four units (8191 x 2048 bf16, without the ring: 30.9 us,
// two blocks of two units 34.0, two of four 34.8).
template <int UMAX, typename F>
cudaError_t norm_shape(int d, F&& f) {
  if (d <= 256) return f(Int<1>{}, Int<1>{});
  if constexpr (UMAX == 4) {
    if (d <= 512) return f(Int<2>{}, Int<1>{});
    if (d <= 1024) return f(Int<4>{}, Int<1>{});
    if (d <= 2048) return f(Int<4>{}, Int<2>{});
    if (d <= 4096) return f(Int<4>{}, Int<4>{});
    if (d <= 8192) return f(Int<4>{}, Int<8>{});
    return f(Int<4>{}, Int<16>{});
  } else if constexpr (UMAX == 2) {
    if (d <= 512) return f(Int<2>{}, Int<1>{});
    if (d <= 1024) return f(Int<2>{}, Int<2>{});
    if (d <= 2048) return f(Int<2>{}, Int<4>{});
    if (d <= 4096) return f(Int<2>{}, Int<8>{});
    if (d <= 8192) return f(Int<2>{}, Int<16>{});
    return f(Int<2>{}, Int<32>{});
  } else {
    if (d <= 512) return f(Int<1>{}, Int<2>{});
    if (d <= 1024) return f(Int<1>{}, Int<4>{});
    if (d <= 2048) return f(Int<1>{}, Int<8>{});
    if (d <= 4096) return f(Int<1>{}, Int<16>{});
    if (d <= 8192) return f(Int<1>{}, Int<32>{});
    return f(Int<2>{}, Int<32>{});
  }
}

// The rows that a team's ring holds, or 0 where the backward takes its rows
// straight into registers: 8-bit h in rows of odd multiples of 8 bytes, short rows
// and those of more warps than the ring's block has, batches of fewer than kRingRows rows
// per team (the other path spreads those over more blocks; at 1500 and 740 x 2048
// both end before the call's host side does).
constexpr int kRingRows = 4;
struct NormPlan {
  int stages, blocks;
};
NormPlan bwd_plan(int64_t T, int d, bool f32, pkm_q8 fmt, int row_bytes) {
  NormPlan plan{0, 1};
  const auto f = [&](auto, auto wpr) {
    constexpr int WPR = decltype(wpr)::value;
    if constexpr (WPR <= kRingWarps) {
      constexpr int kTeams = ring_teams(WPR);
      int stages = kRingBytes / (kTeams * row_bytes);
      if (stages > kRingStages) stages = kRingStages;
      if ((fmt == PKM_Q8_NONE || d % 16 == 0) && d > 256 && stages >= 2 && T >= (int64_t)kSMs * kTeams * kRingRows) {
        plan = NormPlan{stages, kSMs};
        return cudaSuccess;
      }
    }
    const int rows = rows_per_block(WPR);
    const int64_t b = (T + rows - 1) / rows, most = kSMs * bwd_per_sm(WPR);
    plan.blocks = (int)(b < most ? b : most);
    return cudaSuccess;
  };
  f32 ? norm_shape<1>(d, f) : norm_shape<2>(d, f);
  return plan;
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool need16(const void* p) { return p && al16(p); }

template <pkm_dtype DT>
cudaError_t fwd_launch(const NormFwd& p, cudaStream_t st) {
  return norm_shape<4>(p.d, [&](auto nu, auto wpr) {
    constexpr int NU = decltype(nu)::value, WPR = decltype(wpr)::value;
    const int rows = rows_per_block(WPR);
    note_launch();
    return launch_maybe_pdl(true, norm_fwd_kernel<DT, NU, WPR>,
                            dim3((unsigned)((p.T + rows - 1) / rows)), dim3(block_threads(WPR)), 0,
                            st, p);
  });
}

int row_bytes(int d, pkm_dtype dt, pkm_dtype dy, pkm_q8 fmt, bool dsum) {
  const int b = dt == PKM_F32 ? 4 : 2, y = dy == PKM_F32 ? 4 : 2;
  return d * (y + (fmt == PKM_Q8_NONE ? b : 1) + (dsum ? b : 0));
}

template <pkm_dtype DT, pkm_dtype DY>
cudaError_t bwd_launch(const NormBwd& p, float* dweight, int32_t* status, cudaStream_t st) {
  constexpr bool f32 = DT == PKM_F32 || DY == PKM_F32;
  const int bytes = row_bytes(p.d, DT, DY, p.fmt, p.dsum != nullptr);
  const NormPlan plan = bwd_plan(p.T, p.d, f32, p.fmt, bytes);
  const int blocks = plan.blocks;
  const cudaError_t e = norm_shape<f32 ? 1 : 2>(p.d, [&](auto nu, auto wpr) {
    constexpr int NU = decltype(nu)::value, WPR = decltype(wpr)::value;
    note_launch();
    if constexpr (WPR <= kRingWarps) {
      if (plan.stages) {
        constexpr int kTeams = ring_teams(WPR);
        const size_t ring = (size_t)kTeams * plan.stages * bytes;
        const size_t sums = (size_t)(kTeams - 1) * NU * WPR * 32 * kUnit * 4;
        const size_t smem = ring > sums ? ring : sums;
        auto kern = p.fmt == PKM_Q8_NONE ? norm_bwd_ring_kernel<DT, DY, NU, WPR, false>
                                         : norm_bwd_ring_kernel<DT, DY, NU, WPR, true>;
        const cudaError_t set = cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
        if (set != cudaSuccess) return set;
        return launch_maybe_pdl(true, kern, dim3(blocks), dim3(32 * WPR * kTeams), smem, st, p,
                                plan.stages, status);
      }
    }
    return launch_maybe_pdl(true, norm_bwd_kernel<DT, DY, NU, WPR>, dim3(blocks),
                            dim3(block_threads(WPR)), 0, st, p);
  });
  if (e != cudaSuccess || !dweight) return e;
  note_launch();
  return launch_maybe_pdl(true, norm_dw_kernel, dim3((p.d + 31) / 32), dim3(32 * kDwStrips), 0, st,
                          p.part, blocks, p.d, dweight);
}

pkm_status fwd_validate(const pkm_norm_args* a) {
  if (!a || a->T < 0 || a->d < 8 || a->d % 8 || !(a->eps >= 0.f) ||
      (a->dtype != PKM_F32 && a->dtype != PKM_BF16) ||
      (a->fmt != PKM_Q8_NONE && a->fmt != PKM_Q8_E4M3 && a->fmt != PKM_Q8_INT8))
    return PKM_ERR_INVALID_ARG;
  if (a->d > kMaxD || a->T > (int64_t(1) << 31) - 64) return PKM_ERR_UNSUPPORTED;
  if (a->T == 0) return PKM_OK;
  if (!need16(a->x) || !al16(a->residual) || !al16(a->weight) || !al16(a->sum) || !al16(a->y) ||
      !al16(a->y8) || !al16(a->rstd))
    return PKM_ERR_INVALID_ARG;
  if ((a->y8 != nullptr) != (a->fmt != PKM_Q8_NONE)) return PKM_ERR_INVALID_ARG;
  if (a->y8 && !need16(a->scales)) return PKM_ERR_INVALID_ARG;
  if (!a->y && !a->y8) return PKM_ERR_INVALID_ARG;
  return PKM_OK;
}

size_t bwd_bytes(const pkm_norm_bwd_args* a) {
  if (a->T <= 0 || a->d < 8 || a->d > kMaxD) return 0;
  const bool f32 = a->dtype == PKM_F32 || a->dy_dtype == PKM_F32;
  // of the register path, whose blocks are the more: the same for every fmt and dsum
  return (size_t)bwd_plan(a->T, a->d, f32, PKM_Q8_NONE, kRingBytes).blocks * (size_t)a->d * 4;
}

pkm_status bwd_validate(const pkm_norm_bwd_args* a) {
  if (!a || a->T < 0 || a->d < 8 || a->d % 8 || (a->dtype != PKM_F32 && a->dtype != PKM_BF16) ||
      (a->dy_dtype != PKM_F32 && a->dy_dtype != PKM_BF16) ||
      (a->fmt != PKM_Q8_NONE && a->fmt != PKM_Q8_E4M3 && a->fmt != PKM_Q8_INT8))
    return PKM_ERR_INVALID_ARG;
  if (a->d > kMaxD || a->T > (int64_t(1) << 31) - 64) return PKM_ERR_UNSUPPORTED;
  if (!al16(a->dweight)) return PKM_ERR_INVALID_ARG;
  if (a->T == 0) return PKM_OK;
  if (!need16(a->dy) || !need16(a->sum) || !need16(a->rstd) || !need16(a->dx) ||
      !al16(a->weight) || !al16(a->dsum))
    return PKM_ERR_INVALID_ARG;
  if (a->fmt != PKM_Q8_NONE && !need16(a->scales)) return PKM_ERR_INVALID_ARG;
  if (a->dweight && (!need16(a->workspace) || a->workspace_bytes < bwd_bytes(a)))
    return PKM_ERR_WORKSPACE;
  return PKM_OK;
}

}  // namespace
}  // namespace pkm

using namespace pkm;

extern "C" {

PKM_API pkm_status pkm_add_rmsnorm_forward(const pkm_norm_args* a, pkm_stream_t stream) {
  const pkm_status s = fwd_validate(a);
  if (s != PKM_OK || a->T == 0) return s;
  const NormFwd p{a->T,   a->d, a->eps, a->fmt, a->x, a->residual, a->weight, a->sum,
                  a->y,   static_cast<uint8_t*>(a->y8), a->scales, a->rstd};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      a->dtype == PKM_BF16 ? fwd_launch<PKM_BF16>(p, st) : fwd_launch<PKM_F32>(p, st);
  return e == cudaSuccess ? PKM_OK : PKM_ERR_CUDA;
}

PKM_API size_t pkm_add_rmsnorm_backward_workspace_size(const pkm_norm_bwd_args* a) {
  return a ? bwd_bytes(a) : 0;
}

PKM_API pkm_status pkm_add_rmsnorm_backward(const pkm_norm_bwd_args* a, pkm_stream_t stream) {
  const pkm_status s = bwd_validate(a);
  if (s != PKM_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (a->T == 0)
    return a->dweight && cudaMemsetAsync(a->dweight, 0, sizeof(float) * (size_t)a->d, st) !=
                             cudaSuccess
               ? PKM_ERR_CUDA
               : PKM_OK;
  const NormBwd p{a->T, a->d,      a->fmt,  a->dy, a->sum, a->weight, a->dsum,
                  a->scales, a->rstd, a->dx,
                  a->dweight ? static_cast<float*>(a->workspace) : nullptr};
  int32_t* status = status_ptr();
  if (!status) return PKM_ERR_CUDA;
  cudaError_t e;
  if (a->dtype == PKM_BF16)
    e = a->dy_dtype == PKM_BF16 ? bwd_launch<PKM_BF16, PKM_BF16>(p, a->dweight, status, st)
                                : bwd_launch<PKM_BF16, PKM_F32>(p, a->dweight, status, st);
  else
    e = a->dy_dtype == PKM_BF16 ? bwd_launch<PKM_F32, PKM_BF16>(p, a->dweight, status, st)
                                : bwd_launch<PKM_F32, PKM_F32>(p, a->dweight, status, st);
  return e == cudaSuccess ? PKM_OK : PKM_ERR_CUDA;
}

}  // extern "C"
