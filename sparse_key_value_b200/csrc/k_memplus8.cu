// k_memplus8.cu -- the Memory+ backward from activations kept in 8 bits
// ("Memory Layers at Scale" digest, "Memory+ 블록": out = (y ⊙ silu(x W1)) W2).
//
//   a = x W1, dz = dout W2^T, g = silu(a):
//   dy = dz g, da = dz y silu'(a), z = y g, dx = da W1^T, dW1 = x^T da,
//   dW2 = z^T dout
//
// x is read back to bf16 (exact: 8 significant bits) for the tensor cores; y
// is decoded where it is used.  One launch computes a and dz of the same tile,
// each in its own accumulator, and its epilogue writes dy, da and z: neither a
// nor dz nor an elementwise pass touches HBM.  (Two launches of 512-column
// tiles with dz in fp32 between them measured 39 + 40 us at best, against 62 at
// 16384 x 1024 x 1024, and 67 MB of workspace.)  da and z are rounded to bf16
// once, the operand type of the three products that follow; those run in one
// launch, the weight gradients (few tiles, a long contraction over the tokens)
// cut into slices that are summed in order.
// Bound by the tensor cores for long batches (10 T d_model d_v operations),
// by launches for short ones.  Measured on one B200: 16384 x 1024 x 1024 181-184
// us back to back (0.94 PFLOP/s; the power cap holds the SMs at 1451 MHz then),
// alone and at full clock: reading x back 8.5, a and dz 62 (operands from L2: 64
// bytes per SM and cycle where each accumulator has 256 columns, the tensor pipe
// busy half the time; 11 for writing dy, da and z), the three products 63 (1.6
// PFLOP/s), the slices' sum 7.  1000 x 640 x 520: 32 us, four dependent launches,
// the longest (a and dz, 256 x 256 a pair of SMs) on 12 pairs of 74.
#include <math.h>

#include "gemm_pair.cuh"
#include "kernels.h"
#include "q8.cuh"

namespace pkm {

namespace {

// a and dz in TMEM, y from memory -> dy, da, z, 32 columns at a time through
// the warp's staging rows.  A lane takes its 128 columns of a into registers
// while dz is still being worked on, so that a of the next tile can follow; the
// columns move down one place a turn, which keeps the loop short and its
// registers fixed (against a and dz read together, on one box: 16384 x 1024 x
// 1024 184 -> 180 us in all, the launch alone 76 -> 66 from cold caches; unrolled
// four times 181, and 1000 x 640 x 520 34 us for 32, the longer code's first
// pass).  Two sets of staging rows: with one, and five ring stages, the short
// batch took 33 us.  The lane's bytes of y for the next columns are loaded while
// these are worked on, the tile's first before its products are done; a warp's
// columns lie in one quantisation group, so a lane has one scale.
struct Memplus8Gate {
  CUtensorMap dy_map, da_map, z_map;
  int64_t T;
  int dv;
  pkm_q8 fmt;
  const uint8_t* y8;
  const float* y_scales;

  static constexpr int kWarps = 8, kCols = 128, kStages = 4, kWarpBytes = 6 * kStageBytesPerWarp;
  static constexpr int kSharedBytes = 0, kBarArrivals = 1;
  static constexpr bool kDual = true;
  struct State {
    uint32_t a[kCols / 32][32];
    uint2 y[4];
    float scale;
    int half;  // of the staging rows, used in turn
  };

  __device__ __forceinline__ void fetch(State& s, int64_t m, int col) const {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (m < T && col + 8 * u < dv)
        s.y[u] = *reinterpret_cast<const uint2*>(y8 + m * dv + col + 8 * u);
  }
  __device__ __forceinline__ void setup(State&, const EpiWarp&) const {}
  __device__ __forceinline__ void begin(State& s, const EpiWarp& w, int, int64_t row0, int n0,
                                        int) const {
    const int c0 = n0 + w.part * kCols;
    const int64_t m = row0 + w.lane;
    if (m >= T || c0 >= dv) return;
    s.scale = y_scales[m * q8_groups(dv) + c0 / kQ8Group];
    fetch(s, m, c0);
  }
  __device__ __forceinline__ void abandon(State&, const EpiWarp&) const {}

  // the lane's row of a, from buffer 0
  template <class Release>
  __device__ __forceinline__ void first(State& s, const EpiWarp& w, int64_t row0, int n0,
                                        uint32_t tmem, Release release) const {
    const int c0 = n0 + w.part * kCols;
    if (row0 < T && c0 < dv) {  // the whole warp
      __syncwarp();             // the loads are warp-aligned
#pragma unroll
      for (int q = 0; q < kCols / 32; ++q)
        if (q == 0 || c0 + q * 32 < dv) tmem_ld_32x32b_x32(tmem + q * 32, s.a[q]);
      __syncwarp();
      tmem_ld_wait();
    }
    release();
  }

  template <class Release>
  __device__ __forceinline__ void tile(State& s, const EpiWarp& w, int, int64_t row0, int n0, int,
                                       uint32_t tmem, Release release) const {
    const int c0 = n0 + w.part * kCols;
    if (row0 >= T || c0 >= dv) {  // the whole warp
      release();
      return;
    }
#pragma unroll 1
    for (int q = 0; q < kCols / 32; ++q) {
      const int col = c0 + q * 32;
      const bool last = q + 1 == kCols / 32 || col + 32 >= dv;
      const uint32_t* a = s.a[0];
      uint32_t d[32];
      __syncwarp();
      tmem_ld_32x32b_x32(tmem + q * 32, d);
      uint2 yq[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) yq[u] = s.y[u];
      if (!last) fetch(s, row0 + w.lane, col + 32);
      __syncwarp();
      tmem_ld_wait();
      if (last) release();
      stage_free<1>(w.lane);  // the stores of the turn before last
      unsigned char* const stage = w.stage + s.half * 3 * kStageBytesPerWarp;
      s.half ^= 1;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float y[8], o[3][8];
        q8_decode(yq[u], s.scale, fmt, y);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {  // two columns an instruction
          const float2 av = make_float2(__uint_as_float(a[8 * u + e]),
                                        __uint_as_float(a[8 * u + e + 1]));
          const float2 dz = make_float2(__uint_as_float(d[8 * u + e]),
                                        __uint_as_float(d[8 * u + e + 1]));
          const float2 yv = make_float2(y[e], y[e + 1]);
          const float2 one = make_float2(1.f, 1.f), neg = make_float2(-1.f, -1.f);
          const float2 t = __fmul2_rn(av, make_float2(-kLog2e, -kLog2e));
          const float2 den = __fadd2_rn(make_float2(ex2(t.x), ex2(t.y)), one);
          const float2 sg = make_float2(rcp(den.x), rcp(den.y));
          const float2 g = __fmul2_rn(av, sg);
          // slope = sg + g (1 - sg)
          const float2 slope = __ffma2_rn(g, __ffma2_rn(sg, neg, one), sg);
          const float2 o0 = __fmul2_rn(dz, g), o2 = __fmul2_rn(yv, g);
          const float2 o1 = __fmul2_rn(__fmul2_rn(dz, yv), slope);
          o[0][e] = o0.x, o[0][e + 1] = o0.y;
          o[1][e] = o1.x, o[1][e + 1] = o1.y;
          o[2][e] = o2.x, o[2][e + 1] = o2.y;
        }
#pragma unroll
        for (int k = 0; k < 3; ++k)
          *reinterpret_cast<uint4*>(stage64_at(stage + k * kStageBytesPerWarp, w.lane, u)) =
              pack16<PKM_BF16>(o[k]);
      }
      stage_ready();
      if (w.lane == 0) {
        tma_store_3d(&dy_map, stage, col, (int)row0, 0);
        tma_store_3d(&da_map, stage + kStageBytesPerWarp, col, (int)row0, 0);
        tma_store_3d(&z_map, stage + 2 * kStageBytesPerWarp, col, (int)row0, 0);
        bulk_commit();
      }
      __syncwarp();
      if (last) break;
#pragma unroll
      for (int k = 0; k + 1 < kCols / 32; ++k)
#pragma unroll
        for (int e = 0; e < 32; ++e) s.a[k][e] = s.a[k + 1][e];
    }
  }
};

// Problems 0 and 1: slices of dW1 and dW2 (fp32).  Problem 2: dx.
struct Memplus8Grads {
  CUtensorMap map[3];
  StoreOut out[3];

  static constexpr int kWarps = 16, kCols = 64, kStages = 4, kSharedBytes = 0;
  static constexpr int kWarpBytes = kStageBytesPerWarp;
  static constexpr int kBarArrivals = 1;
  static constexpr bool kDual = false;
  struct State {};
  __device__ __forceinline__ void setup(State&, const EpiWarp&) const {}
  __device__ __forceinline__ void begin(State&, const EpiWarp&, int, int64_t, int, int) const {}
  __device__ __forceinline__ void abandon(State&, const EpiWarp&) const {}
  template <class Release>
  __device__ __forceinline__ void tile(State&, const EpiWarp& w, int prob, int64_t row0, int n0,
                                       int z, uint32_t tmem, Release release) const {
    store_tile(out[prob], &map[prob], w, row0, n0, z, tmem, release);
  }
};

bool need16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t rup(size_t x) { return (x + 255) / 256 * 256; }

struct Mp8Layout {
  size_t xb, da, z, w1, w2, total;
  int nz;
  PairPlan plan;
};

// The weight gradients have few tiles and a long contraction over the tokens:
// cut into slices of at least four k-blocks (a unit of the plan takes as long
// as 2 MB of the slices' traffic).
PairPlan grads_plan(int64_t T, int dm, int dv) {
  const auto tiles = [](int64_t m, int64_t n, int tn) {
    return (m + 255) / 256 * ((n + tn - 1) / tn);
  };
  return pair_plan([&](int tn) { return tiles(dm, dv, tn) + tiles(dv, dm, tn); },
                   (T + gp::kKB - 1) / gp::kKB, 64, 4, 2.0 * dm * dv * 8 / (2 << 20),
                   [&](int tn) { return tiles(T, dm, tn); }, (dv + gp::kKB - 1) / gp::kKB);
}

Mp8Layout mp8_layout(const pkm_memplus_bwd8_args* g) {
  Mp8Layout L{};
  const size_t T = (size_t)g->T, dm = (size_t)g->d_model, dv = (size_t)g->d_v;
  size_t off = 0;
  auto take = [&](size_t b) {
    const size_t o = off;
    off += rup(b);
    return o;
  };
  L.plan = grads_plan(g->T, g->d_model, g->d_v);
  L.nz = L.plan.nz;
  L.xb = take(T * dm * 2);
  L.da = take(T * dv * 2);
  L.z = take(T * dv * 2);
  const bool direct = L.nz == 1 && g->grad_dtype == PKM_F32;
  L.w1 = direct ? 0 : take((size_t)L.nz * dm * dv * 4);
  L.w2 = direct ? 0 : take((size_t)L.nz * dm * dv * 4);
  L.total = off;
  return L;
}

pkm_status mp8_sizes(const pkm_memplus_bwd8_args* g) {
  if (!g || g->T < 0 || g->d_model < 8 || g->d_model % 8 || g->d_v < 8 || g->d_v % 8 ||
      (g->fmt != PKM_Q8_E4M3 && g->fmt != PKM_Q8_INT8) ||
      (g->grad_dtype != PKM_F32 && g->grad_dtype != PKM_BF16))
    return PKM_ERR_INVALID_ARG;
  // tile counts and the 8-bit load's grid stay in 31 bits
  if (g->T > (int64_t(1) << 28) || g->d_model > 65536 || g->d_v > 65536 ||
      g->T * q8_groups(g->d_model) >= (int64_t(1) << 34))
    return PKM_ERR_UNSUPPORTED;
  return PKM_OK;
}

pkm_status mp8_validate(const pkm_memplus_bwd8_args* g, Mp8Layout* L) {
  const pkm_status s = mp8_sizes(g);
  if (s != PKM_OK) return s;
  if (!need16(g->dW1) || !need16(g->dW2)) return PKM_ERR_INVALID_ARG;
  if (g->T == 0) return PKM_OK;
  const void* need[] = {g->x8,       g->x_scales, g->W1, g->W2, g->y8,
                        g->y_scales, g->dout,     g->dy, g->dx};
  for (const void* p : need)
    if (!need16(p)) return PKM_ERR_INVALID_ARG;
  *L = mp8_layout(g);
  if (!need16(g->workspace) || g->workspace_bytes < L->total)
    return PKM_ERR_WORKSPACE;
  return PKM_OK;
}

#define PKM_TRY(expr)                 \
  do {                                \
    const cudaError_t e_ = (expr);    \
    if (e_ != cudaSuccess) return e_; \
    note_launch();                    \
  } while (0)

cudaError_t memplus8_backward(const pkm_memplus_bwd8_args* g, const Mp8Layout& L, int32_t* status,
                              cudaStream_t st) {
  char* ws = static_cast<char*>(g->workspace);
  const int64_t T = g->T;
  const int dm = g->d_model, dv = g->d_v;
  auto* xb = reinterpret_cast<__nv_bfloat16*>(ws + L.xb);
  auto* da = reinterpret_cast<__nv_bfloat16*>(ws + L.da);
  auto* z = reinterpret_cast<__nv_bfloat16*>(ws + L.z);
  cudaError_t e = launch_act8_load(g->x8, g->x_scales, T, dm, g->fmt, xb, PKM_BF16, st);
  if (e != cudaSuccess) return e;
  {  // a = x W1 and dz = dout W2^T, and everything elementwise
    PairMaps<2> m;
    if (!pair_map(&m.a[0], xb, T, dm, dm, false) || !pair_map(&m.b[0], g->W1, dv, dm, dv, true) ||
        !pair_map(&m.a[1], g->dout, T, dm, dm, false) ||
        !pair_map(&m.b[1], g->W2, dv, dm, dm, false))
      return cudaErrorInvalidValue;
    const PairProbs<2> p{{pair_prob(T, dv, dm, false, true, 1, 1, gp::kN),
                          pair_prob(T, dv, dm, false, false, 1, 1, gp::kN)}, 2, {}};
    Memplus8Gate epi{{}, {}, {}, T, dv, g->fmt, static_cast<const uint8_t*>(g->y8), g->y_scales};
    if (!pair_out_map(&epi.dy_map, g->dy, dv, T, 1, dv, PKM_BF16) ||
        !pair_out_map(&epi.da_map, da, dv, T, 1, dv, PKM_BF16) ||
        !pair_out_map(&epi.z_map, z, dv, T, 1, dv, PKM_BF16))
      return cudaErrorInvalidValue;
    PKM_TRY((launch_pair_gemm<2>(m, p, epi, status, st)));
  }
  const bool gb = g->grad_dtype == PKM_BF16;
  const bool direct = L.nz == 1 && !gb;
  float* w1 = direct ? static_cast<float*>(g->dW1) : reinterpret_cast<float*>(ws + L.w1);
  float* w2 = direct ? static_cast<float*>(g->dW2) : reinterpret_cast<float*>(ws + L.w2);
  {  // dW1 = x^T da, dW2 = z^T dout, dx = da W1^T
    PairMaps<3> m;
    if (!pair_map(&m.a[0], xb, dm, (int)T, dm, true) ||
        !pair_map(&m.b[0], da, dv, (int)T, dv, true) ||
        !pair_map(&m.a[1], z, dv, (int)T, dv, true) ||
        !pair_map(&m.b[1], g->dout, dm, (int)T, dm, true) ||
        !pair_map(&m.a[2], da, T, dv, dv, false) || !pair_map(&m.b[2], g->W1, dm, dv, dv, false))
      return cudaErrorInvalidValue;
    const PairProbs<3> p{{pair_prob(dm, dv, (int)T, true, true, L.nz, 1, L.plan.tile0),
                          pair_prob(dv, dm, (int)T, true, true, L.nz, 1, L.plan.tile0),
                          pair_prob(T, dm, dv, false, false, 1, 1, L.plan.tile1)}, 2, {}};
    Memplus8Grads epi{{}, {{dm, dv, 0, 0}, {dv, dm, 0, 0}, {T, dm, gb, 0}}};
    if (!pair_out_map(&epi.map[0], w1, dv, dm, L.nz, dv, PKM_F32) ||
        !pair_out_map(&epi.map[1], w2, dm, dv, L.nz, dm, PKM_F32) ||
        !pair_out_map(&epi.map[2], g->dx, dm, T, 1, dm, g->grad_dtype))
      return cudaErrorInvalidValue;
    PKM_TRY((launch_pair_gemm<3>(m, p, epi, status, st)));
  }
  if (direct) return cudaSuccess;
  PKM_TRY(launch_slice_sum(w1, L.nz, (int64_t)dm * dv, g->dW1, g->grad_dtype, st, w2, g->dW2));
  return cudaSuccess;
}

}  // namespace
}  // namespace pkm

using namespace pkm;

extern "C" {

PKM_API size_t pkm_memplus_backward_act8_workspace_size(const pkm_memplus_bwd8_args* g) {
  return mp8_sizes(g) == PKM_OK ? mp8_layout(g).total : 0;
}

PKM_API pkm_status pkm_memplus_backward_act8(const pkm_memplus_bwd8_args* g,
                                             pkm_stream_t stream) {
  Mp8Layout L{};
  const pkm_status s = mp8_validate(g, &L);
  if (s != PKM_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (g->T == 0) {
    const size_t b = (size_t)g->d_model * g->d_v * (g->grad_dtype == PKM_F32 ? 4 : 2);
    return cudaMemsetAsync(g->dW1, 0, b, st) == cudaSuccess &&
                   cudaMemsetAsync(g->dW2, 0, b, st) == cudaSuccess
               ? PKM_OK
               : PKM_ERR_CUDA;
  }
  int32_t* status = status_ptr();
  if (!status) return PKM_ERR_CUDA;
  return memplus8_backward(g, L, status, st) == cudaSuccess ? PKM_OK : PKM_ERR_CUDA;
}

}  // extern "C"
