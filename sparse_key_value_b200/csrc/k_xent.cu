// k_xent.cu -- softmax cross entropy of an output layer over a large
// vocabulary, without keeping the logits, and its gradients.
//
//   logit[t, v] = <x[t], W[v]>,  lse[t] = log sum_v exp(logit[t, v]),
//   loss[t] = lse[t] - logit[t, target[t]]          (0 where there is none)
//   d[t, v] = (exp(logit[t, v] - lse[t]) - [v = target[t]]) dloss[t]
//   dx = d W,  dW = d^T x
//
// Forward: the logits live in TMEM only.  Each tile's epilogue reduces its
// columns to a running maximum and sum per row, a small kernel joins the tiles'
// partials.  Base 2 throughout: with s = logit log2(e), a term is 2^(s - max)
// -- one multiply-add and one ex2 -- and the rounding of log2(e) scales every
// term alike (1.3e-8 of the logit).
// Backward: d for a piece of the vocabulary (recomputed logits, rounded to
// bf16 once: the operand type of the products that read it, half a step of
// each d), then both products in one launch; dx is summed over the pieces in
// fp32, in piece order.  d is held over s = max |dloss| and the products are
// multiplied by s in fp32: with equal weights the large terms are then near
// -1, which bf16 holds, where all of -1 / n may sit on the same worst
// rounding (2.6e-3 of dW's norm against 1.7e-3).
// Bound by the tensor cores: 2 T V d operations forward, 6 T V d backward.
// Measured on one B200 at 8192 x 32768 x 1024: forward 395-420 us (1.31-1.39
// PFLOP/s; the library's product of the same sizes, which writes the logits and
// reads none back, 442-466), 340 us alone on a cool GPU; backward 1.27-1.32 ms
// (1.25-1.30 PFLOP/s).  At 16384 x 131072 x 1024 3.27 ms (the library's product
// 3.66) and 10.3 ms.  Back to back both run into the power cap (SMs at 1425 and
// 1294 MHz), which holds plain products at 1.40-1.42.  Short
// batches: 37 x 50021 x 512 20.4 us for the 51 MB of W, its gradients 62 us (W
// read twice, dW written, 256 rows of a tile for 37 tokens).
#include <math.h>

#include "gemm_pair.cuh"
#include "kernels.h"

namespace pkm {

namespace {

constexpr float kLn2 = 0.6931471805599453f;

struct MaxSum {  // of terms 2^s: the maximum and the sum of 2^(s - maximum)
  float mx, sum;
  __device__ __forceinline__ void join(float qm, float qs) {
    const float nm = fmaxf(mx, qm);
    const float ref = nm == -INFINITY ? 0.f : nm;  // all -inf so far: every term is 0
    sum = sum * ex2(mx - ref) + qs * ex2(qm - ref);
    mx = nm;
  }
};

// Row maximum and sum of a tile -> part[tile column][row], and the target's
// logit.  A lane carries its row over the tile's two buffers; the four warps of
// a row quarter join theirs through shared memory.
struct XentStats {
  int64_t T;
  int V, tile_n;
  const int32_t* target;
  float2* part;  // [tiles_n][T]
  float* picked;

  static constexpr int kWarps = 16, kCols = 64, kStages = 4, kWarpBytes = 0;
  static constexpr int kSharedBytes = 2 * 4 * 128 * sizeof(float2), kBarArrivals = 4;
  static constexpr bool kDual = false;
  struct State {
    int target;
    MaxSum v;
    uint32_t turn;  // tiles so far
  };
  __device__ __forceinline__ void setup(State&, const EpiWarp&) const {}
  __device__ __forceinline__ void begin(State& s, const EpiWarp& w, int, int64_t row0, int n0,
                                        int) const {
    if (n0 % tile_n) return;  // the tile's second buffer
    s.target = row0 + w.lane < T ? target[row0 + w.lane] : -1;
    s.v = MaxSum{-INFINITY, 0.f};
  }
  __device__ __forceinline__ void abandon(State&, const EpiWarp&) const {}

  __device__ __forceinline__ void columns(State& st, int64_t m, int col, uint32_t* r) const {
    if (col + 32 > V) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (col + j >= V) r[j] = 0xff800000u;  // -inf: no such column
    }
    float top[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) top[j] = __uint_as_float(r[j]);
#pragma unroll
    for (int j = 4; j < 32; ++j) top[j & 3] = fmaxf(top[j & 3], __uint_as_float(r[j]));
    const float all = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    const float nm = fmaxf(st.v.mx, all * kLog2e);
    const float ref = nm == -INFINITY ? 0.f : nm;
    // two columns an instruction where it is not the exponential
    const float2 l2 = make_float2(kLog2e, kLog2e), minus = make_float2(-ref, -ref);
    float2 s[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float2 x = __ffma2_rn(
          make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), l2, minus);
      s[(j >> 1) & 1] = __fadd2_rn(s[(j >> 1) & 1], make_float2(ex2(x.x), ex2(x.y)));
    }
    st.v.sum = fmaf(st.v.sum, ex2(st.v.mx - ref), (s[0].x + s[0].y) + (s[1].x + s[1].y));
    st.v.mx = nm;
    const uint32_t at = (uint32_t)st.target - (uint32_t)col;
    if (at < 32u) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (at == j) picked[m] = __uint_as_float(r[j]);
    }
  }

  template <class Release>
  __device__ __forceinline__ void tile(State& st, const EpiWarp& w, int, int64_t row0, int n0,
                                       int, uint32_t tmem, Release release) const {
    const int64_t m = row0 + w.lane;
    const int c0 = n0 + w.part * kCols;
    if (row0 < T && c0 < V) {
      uint32_t r[64];
      tmem_ld_32x32b_x32(tmem, r);
      tmem_ld_32x32b_x32(tmem + 32, r + 32);
      tmem_ld_wait();
      release();
      columns(st, m, c0, r);
      if (c0 + 32 < V) columns(st, m, c0 + 32, r + 32);
    } else {
      release();
    }
    if (n0 % tile_n + gp::kN < tile_n && n0 + gp::kN < V) return;  // the second buffer follows
    __syncwarp();
    // Two sets of slots, each with a barrier per row quarter, in turn.  A warp
    // hands TMEM back before it comes here, so a faster one may already be here
    // with the next tile, but no further: the products of the tile after that
    // need the buffer of the next one back from every warp, which each gives
    // only after it has arrived (the joining warp: after it has read) for this
    // one.  So a phase counts the four arrivals of one tile, and a slot is
    // written again only after it was read.  (On one barrier a fast warp's
    // second arrival would count for a slow warp's first.)
    const int set = st.turn & 1;
    const uint32_t parity = (st.turn >> 1) & 1;
    ++st.turn;
    float2* slot = reinterpret_cast<float2*>(w.shared) + set * 4 * 128;
    slot[w.part * 128 + w.quarter * 32 + w.lane] = make_float2(st.v.mx, st.v.sum);
    __syncwarp();
    uint64_t* bar = &w.bars[set][w.quarter];
    if (w.lane == 0) mbar_arrive(bar);
    if (w.part != 0) return;
    if (mbar_wait_or_abort(bar, parity, w.abort, w.status) && m < T) {
      for (int k = 1; k < 4; ++k) {
        const float2 q = slot[k * 128 + w.quarter * 32 + w.lane];
        st.v.join(q.x, q.y);
      }
      part[(int64_t)(n0 / tile_n) * T + m] = make_float2(st.v.mx, st.v.sum);
    }
    __syncwarp();
  }
};

// lse and loss from the partials: 8 rows per block, 64 strips of partials (a
// warp reads 8 rows of 4 strips), joined over the warp, then over the warps.
constexpr int kJoinRows = 8, kJoinThreads = 512;

__global__ void __launch_bounds__(kJoinThreads) xent_join_kernel(
    const float2* __restrict__ part, int slots, int64_t T, int V,
    const int32_t* __restrict__ target, int32_t ignore, const float* __restrict__ picked,
    float* __restrict__ loss, float* __restrict__ lse, int32_t* status) {
  __shared__ float2 sm[kJoinThreads / 32][kJoinRows];
  constexpr int kStrips = kJoinThreads / kJoinRows, kAtOnce = 4;
  pdl_launch_dependents();
  pdl_wait();
  const int in = threadIdx.x % kJoinRows, strip = threadIdx.x / kJoinRows;
  const int64_t m = (int64_t)blockIdx.x * kJoinRows + in;
  MaxSum v{-INFINITY, 0.f};
  for (int s0 = strip; s0 < slots && m < T; s0 += kAtOnce * kStrips) {
    float2 q[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int s = s0 + u * kStrips;
      q[u] = s < slots ? part[(int64_t)s * T + m] : make_float2(-INFINITY, 0.f);
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) v.join(q[u].x, q[u].y);
  }
#pragma unroll
  for (int o = kJoinRows; o < 32; o <<= 1) {
    const float qm = __shfl_xor_sync(0xffffffffu, v.mx, o);
    const float qs = __shfl_xor_sync(0xffffffffu, v.sum, o);
    v.join(qm, qs);
  }
  if ((threadIdx.x & 31) < kJoinRows) sm[threadIdx.x >> 5][in] = make_float2(v.mx, v.sum);
  __syncthreads();
  if (threadIdx.x >= kJoinRows || m >= T) return;
  for (int k = 1; k < kJoinThreads / 32; ++k) v.join(sm[k][in].x, sm[k][in].y);
  const float l = (v.mx + log2f(v.sum)) * kLn2;
  lse[m] = l;
  const int32_t t = target[m];
  const bool counted = t != ignore && t >= 0 && t < V;
  if (!counted && t != ignore) set_status(status, PKM_ERR_DEVICE);
  loss[m] = counted ? l - picked[m] : 0.f;
}

// d of one vocabulary piece, bf16
struct XentDelta {
  CUtensorMap out;  // [T][Vp]
  int64_t T;
  int Vp, v0, V;    // piece columns, first column, vocabulary
  const int32_t* target;
  int32_t ignore;
  const float *lse, *dloss;
  float* scale;  // max |dloss| over the counted positions (1 if 0 or infinite): out

  static constexpr int kWarps = 16, kCols = 64, kStages = 4, kSharedBytes = 64;
  static constexpr int kWarpBytes = kStageBytesPerWarp;
  static constexpr int kBarArrivals = 1;
  static constexpr bool kDual = false;
  struct State {
    int target;
    float g, l2, scale;
    bool counted;
  };
  // Every CTA finds the same maximum while its first products run.
  __device__ __forceinline__ void setup(State& s, const EpiWarp& w) const {
    const int warp = w.part * 4 + w.quarter;
    float m = 0.f;
#pragma unroll 4
    for (int64_t t = warp * 32 + w.lane; t < T; t += 32 * kWarps) {
      const int32_t k = target[t];
      if (k != ignore && k >= 0 && k < V) m = fmaxf(m, fabsf(dloss[t]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float* all = reinterpret_cast<float*>(w.shared);
    if (w.lane == 0) all[warp] = m;
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
#pragma unroll
    for (int k = 0; k < kWarps; ++k) m = fmaxf(m, all[k]);
    s.scale = m > 0.f && m < INFINITY ? m : 1.f;
    if (blockIdx.x == 0 && warp == 0 && w.lane == 0) *scale = s.scale;
  }
  __device__ __forceinline__ void begin(State& s, const EpiWarp& w, int, int64_t row0, int n0,
                                        int) const {
    const int64_t m = row0 + w.lane;
    s.target = m < T ? target[m] : ignore;
    s.counted = s.target != ignore && s.target >= 0 && s.target < V;
    s.g = s.counted ? dloss[m] / s.scale : 0.f;
    s.l2 = s.counted ? lse[m] * kLog2e : 0.f;
  }
  __device__ __forceinline__ void abandon(State&, const EpiWarp&) const {}

  __device__ __forceinline__ void columns(const State& s, const EpiWarp& w, int64_t row0, int col,
                                          const uint32_t* r) const {
    float p[32];
    const float2 l2 = make_float2(kLog2e, kLog2e), minus = make_float2(-s.l2, -s.l2);
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float2 x = __ffma2_rn(
          make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), l2, minus);
      p[j] = ex2(x.x);
      p[j + 1] = ex2(x.y);
    }
    const uint32_t at = (uint32_t)s.target - (uint32_t)(v0 + col);
    if (at < 32u) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (at == j) p[j] -= 1.f;
    }
    uint32_t o[16];
    const float2 g = make_float2(s.g, s.g);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float2 v = __fmul2_rn(make_float2(p[2 * j], p[2 * j + 1]), g);
      o[j] = s.counted ? pack_bf16x2(v.x, v.y) : 0u;
    }
    uint4 v4[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v4[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
    stage_out(&out, w, col, row0, 0, v4, false);
  }

  template <class Release>
  __device__ __forceinline__ void tile(State& s, const EpiWarp& w, int, int64_t row0, int n0, int,
                                       uint32_t tmem, Release release) const {
    const int c0 = n0 + w.part * kCols;
    if (row0 >= T || c0 >= Vp) {  // the whole warp
      release();
      return;
    }
    uint32_t r[64];
    tmem_ld_32x32b_x32(tmem, r);
    tmem_ld_32x32b_x32(tmem + 32, r + 32);
    tmem_ld_wait();
    release();
    columns(s, w, row0, c0, r);
    if (c0 + 32 < Vp) columns(s, w, row0, c0 + 32, r + 32);
  }
};

// Problem 0: dx partials, fp32 (overwritten or added to), one [T, d] slice per
// z.  Problem 1: rows of dW.
struct XentGrads {
  CUtensorMap map[2];
  StoreOut out[2];
  const float* scale;

  static constexpr int kWarps = 16, kCols = 64, kStages = 4, kSharedBytes = 0;
  static constexpr int kWarpBytes = kStageBytesPerWarp;
  static constexpr int kBarArrivals = 1;
  static constexpr bool kDual = false;
  struct State {
    float scale;
  };
  __device__ __forceinline__ void setup(State& s, const EpiWarp&) const { s.scale = *scale; }
  __device__ __forceinline__ void begin(State&, const EpiWarp&, int, int64_t, int, int) const {}
  __device__ __forceinline__ void abandon(State&, const EpiWarp&) const {}
  template <class Release>
  __device__ __forceinline__ void tile(State& s, const EpiWarp& w, int prob, int64_t row0, int n0,
                                       int z, uint32_t tmem, Release release) const {
    store_tile(out[prob], &map[prob], w, row0, n0, z, tmem, release, s.scale);
  }
};

// ------------------------------------------------------------ host side

bool need16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool need4(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
size_t rup(size_t x) { return (x + 255) / 256 * 256; }

// The most that a piece's d may take.  Fewer pieces mean fewer launches and
// fewer read-modify-writes of dx: 64, 128, 256 and 512 MiB took 1480, 1377, 1358
// and 1314 us at 8192 x 32768 x 1024 and 14.1, 11.5, 10.8 and 10.5 ms at 16384 x
// 131072 x 1024 (a piece in L2 saves less than that).
constexpr int64_t kPieceBytes = int64_t(512) << 20;
constexpr int kMinPiece = 1024;
constexpr int kMaxSlices = 64;  // of dx

struct XentLayout {  // of the backward
  int piece, ld, nz, tile_dx, tile_dw;
  size_t delta, scale, dx, total;
};

PairProb fwd_prob(const pkm_xent_args* a) {
  return pair_prob(a->T, a->V, a->d, false, false, 1, 8);
}

XentLayout xent_layout(const pkm_xent_args* a) {
  XentLayout L{};
  const size_t T = (size_t)a->T;
  // Columns of a piece and slices of dx: at least as many pieces as keep d
  // within kPieceBytes, of the next few counts the plan whose longest pairs of
  // SMs have least to do.  A slice costs its sums' traffic (a unit of the
  // plans takes as long as 2 MB of it).
  const int64_t V = a->V, Tt = a->T > 0 ? a->T : 1;
  int64_t most = kPieceBytes / 2 / Tt / gp::kTileN * gp::kTileN;
  if (most < kMinPiece) most = kMinPiece;
  const int64_t fewest = (V + most - 1) / most;
  const auto tiles = [](int64_t m, int64_t n, int tn) {
    return (m + 255) / 256 * ((n + tn - 1) / tn);
  };
  double best = -1;
  // (a short batch's products take less time than weighing more plans)
  for (int64_t n = fewest; n <= fewest + (Tt >= 1024 && V >= 8 * kMinPiece ? 3 : 0); ++n) {
    int64_t piece = ((V + n - 1) / n + gp::kTileN - 1) / gp::kTileN * gp::kTileN;
    if (piece > V) piece = V;
    const int64_t pieces = (V + piece - 1) / piece;
    const int tn = pair_tile_n(Tt, (int)piece, a->d, 1);
    const int64_t delta = (tiles(Tt, piece, tn) + kPlanPairs - 1) / kPlanPairs *
                          pair_len((a->d + 63) / 64, tn);
    const PairPlan plan = pair_plan(
        [&](int tn) { return tiles(Tt, a->d, tn); }, (piece + 63) / 64, kMaxSlices, 8,
        (double)Tt * a->d * 8 / (2 << 20), [&](int tn) { return tiles(piece, a->d, tn); },
        (Tt + 63) / 64);
    const double cost = (double)pieces * (delta + plan.cost + 8);  // two launches a piece
    if (best < 0 || cost < best) {
      best = cost;
      L.piece = (int)piece;
      L.nz = plan.nz;
      L.tile_dx = plan.tile0;
      L.tile_dw = plan.tile1;
    }
  }
  L.ld = (L.piece + 63) / 64 * 64;
  L.delta = 0;
  L.scale = rup((size_t)a->T * (size_t)L.ld * 2);
  L.dx = L.scale + 256;
  const bool direct = L.nz == 1 && a->grad_dtype == PKM_F32;
  L.total = L.dx + (direct ? 0 : rup((size_t)L.nz * (size_t)a->T * (size_t)a->d * 4));
  return L;
}

pkm_status xent_sizes(const pkm_xent_args* a) {
  if (!a || a->T < 0 || a->V < 1 || a->d < 8 || a->d % 8) return PKM_ERR_INVALID_ARG;
  if (a->dtype != PKM_BF16)
    return a->dtype == PKM_F32 ? PKM_ERR_UNSUPPORTED : PKM_ERR_INVALID_ARG;
  if (a->grad_dtype != PKM_F32 && a->grad_dtype != PKM_BF16) return PKM_ERR_INVALID_ARG;
  // tile counts and tensor-map coordinates stay in 31 bits
  if (a->T > (int64_t(1) << 30) || a->V > (1 << 30) || a->d > 65536 ||
      ((a->T + 255) / 256) * (((int64_t)a->V + 255) / 256) >= (int64_t(1) << 30))
    return PKM_ERR_UNSUPPORTED;
  return PKM_OK;
}

size_t fwd_bytes(const pkm_xent_args* a, size_t* picked) {
  const size_t at = rup((size_t)fwd_prob(a).tiles_n * (size_t)a->T * sizeof(float2));
  if (picked) *picked = at;
  return at + rup((size_t)a->T * 4);
}

pkm_status xent_validate(const pkm_xent_args* a, XentLayout* L) {  // L: of the backward
  const bool backward = L != nullptr;
  const pkm_status s = xent_sizes(a);
  if (s != PKM_OK) return s;
  if (backward && !need16(a->dW)) return PKM_ERR_INVALID_ARG;
  if (a->T == 0) return PKM_OK;
  if (!need16(a->x) || !need16(a->W) || !need4(a->targets) || !need16(a->lse))
    return PKM_ERR_INVALID_ARG;
  if (!backward && !need16(a->loss)) return PKM_ERR_INVALID_ARG;
  if (backward && (!need16(a->dloss) || !need16(a->dx))) return PKM_ERR_INVALID_ARG;
  if (backward) *L = xent_layout(a);
  if (!need16(a->workspace) ||
      a->workspace_bytes < (backward ? L->total : fwd_bytes(a, nullptr)))
    return PKM_ERR_WORKSPACE;
  return PKM_OK;
}

#define PKM_TRY(expr)                         \
  do {                                        \
    const cudaError_t e_ = (expr);            \
    if (e_ != cudaSuccess) return e_;         \
    note_launch();                            \
  } while (0)

cudaError_t xent_forward(const pkm_xent_args* a, int32_t* status, cudaStream_t st) {
  char* ws = static_cast<char*>(a->workspace);
  size_t picked_at = 0;
  fwd_bytes(a, &picked_at);
  auto* part = reinterpret_cast<float2*>(ws);
  auto* picked = reinterpret_cast<float*>(ws + picked_at);
  PairMaps<1> maps;
  if (!pair_map(&maps.a[0], a->x, a->T, a->d, a->d, false) ||
      !pair_map(&maps.b[0], a->W, a->V, a->d, a->d, false))
    return cudaErrorInvalidValue;
  const PairProbs<1> p{{fwd_prob(a)}, 1, {}};
  const XentStats epi{a->T, a->V, p.p[0].tile_n, a->targets, part, picked};
  PKM_TRY((launch_pair_gemm<1>(maps, p, epi, status, st)));
  PKM_TRY(launch_maybe_pdl(true, xent_join_kernel,
                           dim3((unsigned)((a->T + kJoinRows - 1) / kJoinRows)),
                           dim3(kJoinThreads), 0, st, part, p.p[0].tiles_n, a->T, a->V, a->targets,
                           a->ignore_index, picked, a->loss, a->lse, status));
  return cudaSuccess;
}

cudaError_t xent_backward(const pkm_xent_args* a, const XentLayout& L, int32_t* status,
                          cudaStream_t st) {
  char* ws = static_cast<char*>(a->workspace);
  auto* delta = reinterpret_cast<__nv_bfloat16*>(ws + L.delta);
  auto* scale = reinterpret_cast<float*>(ws + L.scale);
  const bool direct = L.nz == 1 && a->grad_dtype == PKM_F32;
  float* dx = direct ? static_cast<float*>(a->dx) : reinterpret_cast<float*>(ws + L.dx);
  const bool gb = a->grad_dtype == PKM_BF16;
  for (int v0 = 0; v0 < a->V; v0 += L.piece) {
    const int Vp = a->V - v0 < L.piece ? a->V - v0 : L.piece;
    const char* Wp = static_cast<const char*>(a->W) + (size_t)v0 * a->d * 2;
    PairMaps<1> m1;
    if (!pair_map(&m1.a[0], a->x, a->T, a->d, a->d, false) ||
        !pair_map(&m1.b[0], Wp, Vp, a->d, a->d, false))
      return cudaErrorInvalidValue;
    const PairProbs<1> p{{pair_prob(a->T, Vp, a->d, false, false, 1, 8)}, 1, {}};
    XentDelta de{{}, a->T, Vp, v0, a->V, a->targets, a->ignore_index, a->lse, a->dloss,
                 scale};
    if (!pair_out_map(&de.out, delta, Vp, a->T, 1, L.ld, PKM_BF16)) return cudaErrorInvalidValue;
    PKM_TRY((launch_pair_gemm<1>(m1, p, de, status, st)));
    PairMaps<2> m2;
    if (!pair_map(&m2.a[0], delta, a->T, Vp, L.ld, false) ||
        !pair_map(&m2.b[0], Wp, a->d, Vp, a->d, true) ||
        !pair_map(&m2.a[1], delta, Vp, (int)a->T, L.ld, true) ||
        !pair_map(&m2.b[1], a->x, a->d, (int)a->T, a->d, true))
      return cudaErrorInvalidValue;
    // a shorter last piece may fill fewer slices: the others keep their sums
    const PairProbs<2> q{{pair_prob(a->T, a->d, Vp, false, true, L.nz, 1, L.tile_dx),
                          pair_prob(Vp, a->d, (int)a->T, true, true, 1, 1, L.tile_dw)}, 1, {}};
    XentGrads ge{{}, {{a->T, a->d, 0, v0 > 0}, {Vp, a->d, gb, 0}}, scale};
    if (!pair_out_map(&ge.map[0], dx, a->d, a->T, L.nz, a->d, PKM_F32) ||
        !pair_out_map(&ge.map[1], static_cast<char*>(a->dW) + (size_t)v0 * a->d * (gb ? 2 : 4),
                      a->d, Vp, 1, a->d, a->grad_dtype))
      return cudaErrorInvalidValue;
    PKM_TRY((launch_pair_gemm<2>(m2, q, ge, status, st)));
  }
  if (direct) return cudaSuccess;
  PKM_TRY(launch_slice_sum(dx, L.nz, a->T * a->d, a->dx, a->grad_dtype, st));
  return cudaSuccess;
}

}  // namespace
}  // namespace pkm

using namespace pkm;

extern "C" {

PKM_API size_t pkm_linear_xent_forward_workspace_size(const pkm_xent_args* a) {
  return xent_sizes(a) == PKM_OK ? fwd_bytes(a, nullptr) : 0;
}

PKM_API size_t pkm_linear_xent_backward_workspace_size(const pkm_xent_args* a) {
  return xent_sizes(a) == PKM_OK ? xent_layout(a).total : 0;
}

PKM_API pkm_status pkm_linear_xent_forward(const pkm_xent_args* a, pkm_stream_t stream) {
  const pkm_status s = xent_validate(a, nullptr);
  if (s != PKM_OK || a->T == 0) return s;
  int32_t* status = status_ptr();
  if (!status) return PKM_ERR_CUDA;
  return xent_forward(a, status, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PKM_OK
             : PKM_ERR_CUDA;
}

PKM_API pkm_status pkm_linear_xent_backward(const pkm_xent_args* a, pkm_stream_t stream) {
  XentLayout L{};
  const pkm_status s = xent_validate(a, &L);
  if (s != PKM_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (a->T == 0)
    return cudaMemsetAsync(a->dW, 0, (size_t)a->V * a->d * (a->grad_dtype == PKM_F32 ? 4 : 2),
                           st) == cudaSuccess
               ? PKM_OK
               : PKM_ERR_CUDA;
  int32_t* status = status_ptr();
  if (!status) return PKM_ERR_CUDA;
  return xent_backward(a, L, status, st) == cudaSuccess ? PKM_OK : PKM_ERR_CUDA;
}

}  // extern "C"
