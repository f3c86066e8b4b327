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
// bf16 with a second gradient 30.9 us with the weight gradient's join (134 MB:
// 4.3 TB/s; the main kernel 24 us, held back by the row's sum between its loads
// and its stores).  A backward with its loads by asynchronous copies into
// shared memory took 45 us where the packed registers took 38.
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
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* red, int turn) {
  v = warp_sum(v);
  if constexpr (WPR > 1) {
    const int warp = threadIdx.x >> 5;
    float* r = red + (turn & 1) * (block_threads(WPR) / 32);
    if ((threadIdx.x & 31) == 0) r[warp] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / WPR), "n"(32 * WPR) : "memory");
    v = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) v += r[warp / WPR * WPR + w];
  }
  return v;
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
// flight than two with four units (8191 x 2048 bf16: 30.9 us, two blocks of two
// units 34.0, two of four 34.8).
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

// Blocks of the backward (each writes a partial weight gradient): what the SMs
// hold at a time, at most one per group of rows.
int bwd_blocks(int64_t T, int d, bool f32) {
  int rows = 1, most = kSMs;
  const auto f = [&](auto, auto wpr) {
    constexpr int WPR = decltype(wpr)::value;
    rows = rows_per_block(WPR);
    most = kSMs * bwd_per_sm(WPR);
    return cudaSuccess;
  };
  f32 ? norm_shape<1>(d, f) : norm_shape<2>(d, f);
  const int64_t b = (T + rows - 1) / rows;
  return (int)(b < most ? b : most);
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

template <pkm_dtype DT, pkm_dtype DY>
cudaError_t bwd_launch(const NormBwd& p, float* dweight, cudaStream_t st) {
  constexpr bool f32 = DT == PKM_F32 || DY == PKM_F32;
  const int blocks = bwd_blocks(p.T, p.d, f32);
  const cudaError_t e = norm_shape<f32 ? 1 : 2>(p.d, [&](auto nu, auto wpr) {
    constexpr int NU = decltype(nu)::value, WPR = decltype(wpr)::value;
    note_launch();
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
  return (size_t)bwd_blocks(a->T, a->d, f32) * (size_t)a->d * 4;
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
  cudaError_t e;
  if (a->dtype == PKM_BF16)
    e = a->dy_dtype == PKM_BF16 ? bwd_launch<PKM_BF16, PKM_BF16>(p, a->dweight, st)
                                : bwd_launch<PKM_BF16, PKM_F32>(p, a->dweight, st);
  else
    e = a->dy_dtype == PKM_BF16 ? bwd_launch<PKM_F32, PKM_BF16>(p, a->dweight, st)
                                : bwd_launch<PKM_F32, PKM_F32>(p, a->dweight, st);
  return e == cudaSuccess ? PKM_OK : PKM_ERR_CUDA;
}

}  // extern "C"
