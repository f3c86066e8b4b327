// gemm_pair.cuh -- persistent bf16 GEMMs on pairs of SMs with an epilogue of
// the caller's (loss statistics, softmax gradients, activation gradients).
//
//   acc[M, N] = A[M, K] B[N, K]^T, fp32 accumulation, 256 x 256 tiles per pair
//
// through tcgen05.mma.cta_group::2: each CTA of a cluster of two loads its own
// 128 rows of A and its own half of B (a ring of up to 6 stages of 32 KiB), one
// instruction multiplies both, each CTA's epilogue reads its 128 rows from
// TMEM while the next tile's products fill the other accumulator.  A or B may
// be held K-major ([M][K]) or MN-major ([K][M]); one launch takes up to three
// problems, so that the tiles of several products fill the GPU together.
//
//   warp 0      TMA producer of this CTA's halves
//   warp 1      TMEM; in the leader, the MMA issuer
//   warps 2-9   epilogue: warp w reads TMEM lanes 32 (w % 4) .. + 31 (rows) of
//               column half (w - 2) / 4.  Two warps per lane quarter: with
//               one, the exponentials of a 256-column tile outlast the
//               products of a short K.
// Spin-waits are bounded as in the library's other pipelined kernels: on a
// timeout the status word is set, the roles stop issuing, the leader waits for
// every copy it was told about and the pair meets before TMEM is freed.
#pragma once

#include "common.cuh"
#include "tc_pair.cuh"
#include "tmap.h"

namespace pkm {

namespace gp {
constexpr int kM = 128, kN = 256, kNh = kN / 2, kKB = 64, kMaxStages = 6, kAcc = 2, kBox = 64;
constexpr int kABytes = kM * kKB * 2, kBBytes = kNh * kKB * 2;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
// ring, staging of the epilogue warps, control words; the first kilobyte
// aligns the ring (the swizzle goes by the address)
template <class E>
constexpr size_t smem_bytes() {
  return 1024 + (size_t)E::kStages * kStageBytes + (size_t)kEpiWarps * E::kWarpBytes + 256;
}
}  // namespace gp

struct PairProb {
  int64_t M;
  int N, K;
  int tiles_m, tiles_n, nz, kb_per;  // nz slices of kb_per k-blocks
  int amn, bmn;                      // operand held MN-major
  int group_m;                       // tile rows walked together (operand reuse in L2)
};

template <int NP>
struct PairMaps {
  CUtensorMap a[NP], b[NP];
};

// Which item a pair takes in its iter-th turn.  The launch's problems form two
// lists: the items of the first go round the pairs; the pairs that then have
// one item less take `extra` items of the second list each to even that out,
// then the second list goes round as well.
struct PairSched {
  int n0, n1, extra;
};

template <int NP>
struct PairProbs {
  PairProb p[NP];
  int first;  // problems of the first list (the rest are the second)
  PairSched sched;
};

struct PairItem {
  int prob, idx;  // prob < 0: no more
};

template <int NP>
__device__ __forceinline__ PairItem pair_item(const PairProbs<NP>& q, int pair, int pairs,
                                              int iter) {
  const PairSched& s = q.sched;
  const int r = s.n0 % pairs;
  const int mine = s.n0 / pairs + (pair < r);
  int idx, prob, end;
  if (iter < mine) {
    idx = pair + iter * pairs;
    prob = 0;
    end = q.first;
  } else {
    const int j = iter - mine;
    if (pair >= r && j < s.extra)
      idx = j * (pairs - r) + pair - r;
    else
      idx = s.extra * (pairs - r) + (pair >= r ? j - s.extra : j) * pairs + pair;
    if (idx >= s.n1) return PairItem{-1, 0};
    prob = q.first;
    end = NP;
  }
  if (NP > 1)
    for (; prob + 1 < end; ++prob) {
      const int n = q.p[prob].tiles_m * q.p[prob].tiles_n * q.p[prob].nz;
      if (idx < n) break;
      idx -= n;
    }
  return PairItem{prob, idx};
}

struct PairTile {
  int64_t m0;
  int n0, z;
};

__device__ __forceinline__ PairTile pair_tile(const PairProb& p, int idx) {
  const int per = p.tiles_m * p.tiles_n;
  const int z = idx / per, rem = idx - z * per;
  const int g = rem / (p.group_m * p.tiles_n);
  const int in = rem - g * (p.group_m * p.tiles_n);
  const int gs = min(p.group_m, p.tiles_m - g * p.group_m);
  const int n = in / gs;
  return PairTile{(int64_t)(g * p.group_m + in - n * gs) * (2 * gp::kM), n * gp::kN, z};
}

struct PairCtl {
  uint64_t full[gp::kMaxStages];   // leader: both CTAs' copies of a stage landed
  uint64_t empty[gp::kMaxStages];  // each CTA: the MMAs are done with a stage
  uint64_t accf[gp::kAcc];         // each CTA: an accumulator is ready
  uint64_t acce[gp::kAcc];         // leader: both epilogues drained an accumulator
  uint64_t epi[gp::kEpiWarps];     // an epilogue warp's own copies
  uint64_t drain;
  uint32_t tmem;
  volatile int abort;
};

// ---- staging: an epilogue warp's 32 rows in shared memory, in the swizzled
// layout of a tensor copy, so that a lane writes its own row's 16-byte pieces
// without bank conflicts and the copy writes whole lines.  (Row-per-lane
// stores to global memory touch 32 lines an instruction: for a 128 x 256 fp32
// tile that alone took as long as the products of K = 1024.)

// 32 fp32 columns, rows of 128 bytes
__device__ __forceinline__ void stage_f32(unsigned char* buf, int lane, const uint32_t* r) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<uint4*>(buf + lane * 128 + ((j ^ (lane & 7)) << 4)) =
        make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
}
// columns 32 h .. + 31 of 64 bf16 columns, rows of 128 bytes
__device__ __forceinline__ void stage_bf16(unsigned char* buf, int lane, int h,
                                           const uint32_t* w) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(buf + lane * 128 + (((4 * h + j) ^ (lane & 7)) << 4)) =
        make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}
// piece j (of 4) of 32 bf16 columns, rows of 64 bytes
__device__ __forceinline__ unsigned char* stage64_at(unsigned char* buf, int lane, int j) {
  return buf + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4);
}

__device__ __forceinline__ void tma_store_3d(const void* map, const void* smem, int c0, int c1,
                                             int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];"
      ::"l"(map), "r"(smem_u32(smem)), "r"(c0), "r"(c1), "r"(c2) : "memory");
}
__device__ __forceinline__ void tma_add_3d(const void* map, const void* smem, int c0, int c1,
                                           int c2) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.bulk_group [%0, {%2, %3, %4}], [%1];"
      ::"l"(map), "r"(smem_u32(smem)), "r"(c0), "r"(c1), "r"(c2) : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// this thread's tensor stores have read their shared memory
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// The warp's staging buffer may be written again (lane 0 issues the stores).
__device__ __forceinline__ void stage_free(int lane) {
  if (lane == 0) bulk_wait_read();
  __syncwarp();
}
// The warp's writes are visible to the copy that lane 0 issues next.
__device__ __forceinline__ void stage_ready() {
  fence_async_smem();
  __syncwarp();
}

struct EpiWarp {
  int lane, half;         // half: columns 128 half .. + 127 of the tile
  unsigned char* stage;   // E::kWarpBytes of shared memory, 1024-byte aligned
  uint64_t* bar;          // a barrier of the warp's own, one arrival
  volatile int* abort;
  int32_t* status;
};

// E: a trivially copyable epilogue with
//   kStages, kWarpBytes   ring stages; staging bytes per epilogue warp
//   struct State          a warp's state over its tiles, zero-initialised
//   begin(State&, w, prob, row0, n0, z)        before the accumulator is ready
//   tile(State&, w, prob, row0, n0, z, tmem)   by a whole warp: rows row0 + lane,
//       columns n0 + 128 half .. + 127 at TMEM address `tmem` (lane quarter
//       and column included)
//   abandon(State&, w)    after an abort: lets copies in flight land
// The accumulator itself -> the problem's output map: fp32 (stored or added
// to; slice z is the map's third coordinate) or bf16.
struct StoreOut {
  int64_t rows;
  int cols;
  int bf16, add;
};

__device__ __forceinline__ void store_tile(const StoreOut& o, const CUtensorMap* map,
                                           const EpiWarp& w, int64_t row0, int n0, int z,
                                           uint32_t tmem) {
  if (row0 >= o.rows) return;  // the whole warp
  const int c0 = n0 + w.half * gp::kNh;
  const int step = o.bf16 ? 64 : 32;
  for (int q = 0; q < gp::kNh; q += step) {
    if (c0 + q >= o.cols) break;
    stage_free(w.lane);
#pragma unroll 1
    for (int h = 0; h < step / 32; ++h) {
      uint32_t r[32];
      tmem_ld_32x32b_x32(tmem + q + 32 * h, r);
      tmem_ld_wait();
      if (o.bf16) {
        uint32_t p[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
          p[j] = pack_bf16x2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
        stage_bf16(w.stage, w.lane, h, p);
      } else {
        stage_f32(w.stage, w.lane, r);
      }
    }
    stage_ready();
    if (w.lane == 0) {
      if (o.add)
        tma_add_3d(map, w.stage, c0 + q, (int)row0, z);
      else
        tma_store_3d(map, w.stage, c0 + q, (int)row0, z);
      bulk_commit();
    }
    __syncwarp();
  }
}

template <int NP, class E>
__global__ void __launch_bounds__(gp::kThreads, 1)
    pair_gemm_kernel(const __grid_constant__ PairMaps<NP> maps,
                     const __grid_constant__ PairProbs<NP> probs, const __grid_constant__ E epi,
                     int32_t* status) {
  using namespace gp;
  constexpr int kStages = E::kStages;
  static_assert(kStages <= kMaxStages && E::kWarpBytes % 1024 == 0, "shared memory layout");
  static_assert(sizeof(PairCtl) <= 256 && smem_bytes<E>() <= 227 * 1024, "shared memory size");
  extern __shared__ unsigned char smem_raw[];
  unsigned char* stages = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* staging = stages + kStages * kStageBytes;
  PairCtl* ctl = reinterpret_cast<PairCtl*>(staging + kEpiWarps * E::kWarpBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&ctl->full[s], 1);   // the leader's producer registers both CTAs' bytes
      mbar_init(&ctl->empty[s], 1);  // the leader's commit
    }
    for (int b = 0; b < kAcc; ++b) {
      mbar_init(&ctl->accf[b], 1);
      mbar_init(&ctl->acce[b], 2 * kEpiWarps);
    }
    for (int w = 0; w < kEpiWarps; ++w) mbar_init(&ctl->epi[w], 1);
    mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < NP; ++i) {
      prefetch_tmap(&maps.a[i]);
      prefetch_tmap(&maps.b[i]);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(&ctl->tmem, kAcc * kN);
    tmem_relinquish_pair();
  }
  __syncwarp();  // the cluster barrier is warp-aligned: reconverge first
  tc_fence_before();
  cluster_sync_all();  // both CTAs' barriers and TMEM exist before any remote use
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    if (lane == 0) {
      uint32_t issued_mask = 0, issued_par = 0;
      bool ok = true;
      int stage = 0;
      uint32_t phase = 0;
      for (int iter = 0; ok; ++iter) {
        const PairItem it = pair_item(probs, pair, pairs, iter);
        if (it.prob < 0) break;
        const PairProb& p = probs.p[it.prob];
        const CUtensorMap* ta = &maps.a[it.prob];
        const CUtensorMap* tb = &maps.b[it.prob];
        const PairTile tc = pair_tile(p, it.idx);
        const int am = (int)(tc.m0 + (int64_t)rank * kM);  // this CTA's rows
        const int bn = tc.n0 + (int)rank * kNh;            // this CTA's half of the columns
        const int kb0 = tc.z * p.kb_per;
        const int kb1 = min(kb0 + p.kb_per, (p.K + kKB - 1) / kKB);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait_or_abort(&ctl->empty[stage], phase ^ 1, &ctl->abort, status)) {
            ok = false;
            break;
          }
          unsigned char* sa = stages + stage * kStageBytes;
          unsigned char* sb = sa + kABytes;
          const int kc = kb * kKB;
          const uint32_t bar = map_to(&ctl->full[stage], 0);
          // the leader registers the bytes of both CTAs' copies; a copy of
          // the partner's that lands first only takes the count below zero
          if (leader) mbar_arrive_expect_tx(&ctl->full[stage], 2 * kStageBytes);
          if (p.amn) {
#pragma unroll
            for (int j = 0; j < kM / kBox; ++j)
              tma_load_2d_pair(sa + j * kBox * 128, ta, bar, am + j * kBox, kc);
          } else {
            tma_load_2d_pair(sa, ta, bar, kc, am);
          }
          if (p.bmn) {
#pragma unroll
            for (int j = 0; j < kNh / kBox; ++j)
              tma_load_2d_pair(sb + j * kBox * 128, tb, bar, bn + j * kBox, kc);
          } else {
            tma_load_2d_pair(sb, tb, bar, kc, bn);
          }
          issued_mask |= 1u << stage;
          issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // on an abort the leader lets every copy it was told about land
      if (!ok && leader) {
        for (int s = 0; s < kStages; ++s)
          if (issued_mask & (1u << s))
            for (unsigned long long i = 0; i < kSpinLimit; ++i)
              if (mbar_try_wait(&ctl->full[s], (issued_par >> s) & 1)) break;
      }
    }
  } else if (warp == 1) {
    // ----------------------------------------------- MMA issuer (leader)
    if (lane == 0 && leader) {
      bool ok = true;
      int stage = 0;
      uint32_t phase = 0;
      for (int iter = 0; ok; ++iter) {
        const PairItem it = pair_item(probs, pair, pairs, iter);
        if (it.prob < 0) break;
        const PairProb& p = probs.p[it.prob];
        const uint32_t idesc = idesc_bf16_f32(2 * kM, kN) | (p.amn ? (1u << 15) : 0u) |
                               (p.bmn ? (1u << 16) : 0u);
        // one 16-deep step inside a k-block: 32 bytes along a K-major row,
        // 16 lines of 128 bytes of an MN-major tile
        const uint32_t astep = p.amn ? 2048 >> 4 : 32 >> 4, bstep = p.bmn ? 2048 >> 4 : 32 >> 4;
        const PairTile tc = pair_tile(p, it.idx);
        const int kb0 = tc.z * p.kb_per;
        const int nkb = min(p.kb_per, (p.K + kKB - 1) / kKB - kb0);
        const int buf = iter & 1;
        // both epilogues have drained this accumulator's previous tile
        if (!mbar_wait_or_abort(&ctl->acce[buf], ((iter >> 1) & 1) ^ 1, &ctl->abort, status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t dt = tmem + (uint32_t)(buf * kN);
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait_or_abort(&ctl->full[stage], phase, &ctl->abort, status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(stages + stage * kStageBytes);
          const uint32_t sb = sa + kABytes;
          const uint64_t ad = p.amn ? smem_desc_mn128(sa) : smem_desc_k128(sa);
          const uint64_t bd = p.bmn ? smem_desc_mn128(sb) : smem_desc_k128(sb);
#pragma unroll
          for (int kk = 0; kk < kKB / 16; ++kk)
            tc_mma_f16_pair(dt, ad + kk * astep, bd + kk * bstep, idesc, (kb | kk) != 0);
          tc_commit_pair_both(&ctl->empty[stage]);  // both CTAs may refill the stage
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (ok) tc_commit_pair_both(&ctl->accf[buf]);
      }
      // every MMA issued must complete before either CTA frees TMEM or exits
      tc_commit_pair_local(&ctl->drain);
      for (unsigned long long i = 0; i < kSpinLimit; ++i)
        if (mbar_try_wait(&ctl->drain, 0)) break;
    }
  } else {
    // ----------------------------------------------------------- epilogue
    const int quarter = warp & 3;
    const EpiWarp w{lane, (warp - 2) >> 2, staging + (warp - 2) * E::kWarpBytes,
                    &ctl->epi[warp - 2], &ctl->abort, status};
    typename E::State state{};
    for (int iter = 0;; ++iter) {
      const PairItem it = pair_item(probs, pair, pairs, iter);
      if (it.prob < 0) break;
      const PairTile tc = pair_tile(probs.p[it.prob], it.idx);
      const int64_t row0 = tc.m0 + (int64_t)rank * kM + quarter * 32;
      const int buf = iter & 1;
      epi.begin(state, w, it.prob, row0, tc.n0, tc.z);
      const bool got =
          mbar_wait_or_abort(&ctl->accf[buf], (iter >> 1) & 1, &ctl->abort, status);
      if (!__all_sync(0xffffffffu, got)) {
        epi.abandon(state, w);
        break;
      }
      tc_fence_after();
      epi.tile(state, w, it.prob, row0, tc.n0, tc.z,
               tmem + ((uint32_t)(quarter * 32) << 16) + buf * kN + w.half * kNh);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) remote_arrive(map_to(&ctl->acce[buf], 0));
    }
    if (E::kWarpBytes > 0) stage_free(lane);  // no store reads shared memory any more
  }

  // both CTAs finished: the leader's MMAs no longer read either CTA's shared
  // memory or write either CTA's TMEM
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, kAcc * kN);
}

// out = the sum of nz slices of 8 n8 fp32 values, in slice order
template <pkm_dtype GT>
__global__ void __launch_bounds__(256) slice_sum_kernel(const float* __restrict__ part, int nz,
                                                        int64_t n8,
                                                        typename Elem<GT>::T* __restrict__ out) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8;
       i += (int64_t)gridDim.x * 256) {
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    for (int z = 0; z < nz; ++z)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 v = reinterpret_cast<const float4*>(part)[((int64_t)z * n8 + i) * 2 + h];
        acc[4 * h] += v.x;
        acc[4 * h + 1] += v.y;
        acc[4 * h + 2] += v.z;
        acc[4 * h + 3] += v.w;
      }
    constexpr int V = Elem<GT>::kVec;
#pragma unroll
    for (int h = 0; h < 8 / V; ++h)
      reinterpret_cast<uint4*>(out)[(8 / V) * i + h] = pack16<GT>(acc + V * h);
  }
}

// -------------------------------------------------------------- host side

inline cudaError_t launch_slice_sum(const float* part, int nz, int64_t n, void* out, pkm_dtype dt,
                                    cudaStream_t st) {
  const int64_t n8 = n / 8, blocks = (n8 + 255) / 256;
  const unsigned grid = (unsigned)(blocks < 148 * 8 ? blocks : 148 * 8);
  if (dt == PKM_BF16)
    slice_sum_kernel<PKM_BF16>
        <<<grid, 256, 0, st>>>(part, nz, n8, static_cast<__nv_bfloat16*>(out));
  else
    slice_sum_kernel<PKM_F32><<<grid, 256, 0, st>>>(part, nz, n8, static_cast<float*>(out));
  return cudaGetLastError();
}

// Tensor map of an operand with `rows` rows (M or N) and depth K, `ld`
// elements from row to row: [rows][K], or [K][rows] when mn.
inline bool pair_map(CUtensorMap* m, const void* base, int64_t rows, int K, int64_t ld, bool mn) {
  const uint64_t dims[2] = {mn ? (uint64_t)rows : (uint64_t)K, mn ? (uint64_t)K : (uint64_t)rows};
  const uint64_t strides[1] = {(uint64_t)ld * 2};
  const uint32_t box[2] = {(uint32_t)gp::kBox, mn ? (uint32_t)gp::kKB : (uint32_t)gp::kM};
  return make_tmap_bf16(m, base, 2, dims, strides, box);
}

// Tensor map of an output (or fp32 input) of an epilogue: [slices][rows][cols]
// with `ld` elements from row to row; boxes of 32 rows and 128 bytes (64 with
// half) of columns.
inline bool pair_out_map(CUtensorMap* m, const void* base, int64_t cols, int64_t rows,
                         int64_t slices, int64_t ld, pkm_dtype dt, bool half = false) {
  auto enc = tmap_encoder();
  if (!enc) return false;
  const int b = dt == PKM_F32 ? 4 : 2;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)slices};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * b, (cuuint64_t)(ld * rows) * b};
  const cuuint32_t box[3] = {(cuuint32_t)((half ? 64 : 128) / b), 32, 1}, one[3] = {1, 1, 1};
  return enc(m, dt == PKM_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
             3, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             half ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline PairProb pair_prob(int64_t M, int N, int K, bool amn, bool bmn, int nz = 1,
                          int group_m = 1) {
  const int kb = (K + gp::kKB - 1) / gp::kKB;
  const int per = kb > nz ? (kb + nz - 1) / nz : 1;  // every slice gets at least one k-block
  PairProb p{};
  p.M = M;
  p.N = N;
  p.K = K;
  p.tiles_m = (int)((M + 2 * gp::kM - 1) / (2 * gp::kM));
  p.tiles_n = (N + gp::kN - 1) / gp::kN;
  p.kb_per = per;
  p.nz = (kb + per - 1) / per;
  p.amn = amn;
  p.bmn = bmn;
  p.group_m = group_m;
  return p;
}
inline int64_t pair_items(const PairProb& p) { return (int64_t)p.tiles_m * p.tiles_n * p.nz; }

// Pairs that can be resident at once on the current device (0: none).  Cached
// per kernel and device.
template <int NP, class E>
int pair_slots() {
  static int cached[64] = {0};  // 0: not asked yet (racing first calls store the same number)
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (cached[dev]) return cached[dev];
  auto kern = pair_gemm_kernel<NP, E>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)gp::smem_bytes<E>()) != cudaSuccess)
    return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(gp::kThreads, 1, 1);
  cfg.dynamicSmemBytes = gp::smem_bytes<E>();
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  return cached[dev] = n;
}

// `probs`: its first `first` problems make the first list.
template <int NP, class E>
cudaError_t launch_pair_gemm(const PairMaps<NP>& maps, PairProbs<NP> probs, const E& epi,
                             int32_t* status, cudaStream_t stream) {
  const int slots = pair_slots<NP, E>();
  if (slots < 1) return cudaErrorNotSupported;
  int64_t n0 = 0, n1 = 0;
  for (int i = 0; i < NP; ++i) (i < probs.first ? n0 : n1) += pair_items(probs.p[i]);
  if (n0 + n1 >= (int64_t(1) << 30)) return cudaErrorInvalidValue;
  const int pairs = (int)(n0 + n1 < slots ? n0 + n1 : slots);
  probs.sched = PairSched{(int)n0, (int)n1, 0};
  if (n1 > 0 && n0 % pairs) {
    const int a = probs.p[0].kb_per, b = probs.p[probs.first].kb_per;
    probs.sched.extra = (a + b / 2) / b;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * pairs), 1, 1);
  cfg.blockDim = dim3(gp::kThreads, 1, 1);
  cfg.dynamicSmemBytes = gp::smem_bytes<E>();
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pair_gemm_kernel<NP, E>, maps, probs, epi, status);
}

}  // namespace pkm
