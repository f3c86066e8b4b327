// gemm_pair.cuh -- persistent bf16 GEMMs on pairs of SMs with an epilogue of
// the caller's (loss statistics, softmax gradients, activation gradients).
//
//   acc[M, N] = A[M, K] B[N, K]^T, fp32 accumulation, 256 x 512 tiles per pair
//
// through tcgen05.mma.cta_group::2: each CTA of a cluster of two loads its own
// 128 rows of A and its own half of B (a ring of stages of 48 KiB), one
// instruction multiplies both CTAs' operands for 256 columns, two instructions
// a step cover the tile.  Why 512 columns: 256 take 64 bytes of operands per SM
// and cycle at the full MMA rate, about what L2 delivers; 512 take 48.  The
// accumulators then fill TMEM (two buffers of 256 columns), so a tile's
// products cannot start before the last tile's first buffer is read: the
// products of the first buffer run ahead by up to a ring while the epilogue
// reads the second.  Problems with few tiles take 256 columns a tile, to
// spread over the SMs.
// A or B may be held K-major ([M][K]) or MN-major ([K][M]); one launch takes up
// to three problems, so that the tiles of several products fill the GPU
// together.  A dual epilogue takes two products over the same tile at once,
// 256 columns of each, one per buffer; it takes the first into registers while
// the second is worked on, so that the next tile's first can follow at once.
//
//   warp 0      TMA producer of this CTA's halves
//   warp 1      TMEM; in the leader, the MMA issuer
//   the others  E::kWarps epilogue warps: warp w reads TMEM lanes 32 (w % 4) ..
//               + 31 (rows) of columns E::kCols ((w - 2) / 4) .. of a buffer.
//               Eight or sixteen: an epilogue is a chain of latencies (TMEM,
//               exponentials, staging) that only other warps cover.
// Spin-waits are bounded as in the library's other pipelined kernels: on a
// timeout the status word is set, the roles stop issuing, the leader waits for
// every copy it was told about and the pair meets before TMEM is freed.
#pragma once

#include "common.cuh"
#include "kernels.h"
#include "tc_pair.cuh"
#include "tmap.h"

namespace pkm {

namespace gp {
constexpr int kM = 128;             // rows per CTA (the pair covers 256)
constexpr int kN = 256;             // columns of an instruction and a buffer
constexpr int kNh = kN / 2;         // of them, loaded by each CTA
constexpr int kBufs = 2;            // buffers: columns of a tile / kN
constexpr int kTileN = kBufs * kN;
constexpr int kKB = 64, kMaxStages = 6, kMaxWarps = 16, kBox = 64;
constexpr int kABytes = kM * kKB * 2, kBBytes = kNh * kKB * 2;
template <class E>
constexpr int stage_bytes() {
  return kABytes + (E::kDual ? 1 : kBufs) * kBBytes;
}
// Warps before the epilogue's.  A dual epilogue holds a buffer in registers: its
// two warpgroups take over registers of the first (40 + 2 * 232 = 3 * 168, what
// the block is launched with), which its roles then have for themselves.
template <class E>
constexpr int lead_warps() {
  return E::kDual ? 4 : 2;
}
constexpr int kLeadRegs = 40, kDualRegs = 232;
template <class E>
constexpr int threads() {
  return 32 * (lead_warps<E>() + E::kWarps);
}
// ring, staging of the epilogue warps, what they share, control words; the
// first kilobyte aligns the ring (the swizzle goes by the address)
template <class E>
constexpr size_t smem_bytes() {
  return 1024 + (size_t)E::kStages * stage_bytes<E>() + (size_t)E::kWarps * E::kWarpBytes +
         E::kSharedBytes + 512;
}
}  // namespace gp

struct PairProb {
  int64_t M;
  int N, K;
  int tile_n;                        // columns of a tile: 512, or 256
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
    else  // the remainder falls to the pairs from r on first
      idx = s.extra * (pairs - r) + (pair >= r ? j - s.extra : j) * pairs +
            (pair >= r ? pair - r : pair + pairs - r);
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
  return PairTile{(int64_t)(g * p.group_m + in - n * gs) * (2 * gp::kM), n * p.tile_n, z};
}

// Buffers that a tile's products fill at a time.
template <class E>
__device__ __forceinline__ int pair_bufs(const PairProb& p, const PairTile& t) {
  return !E::kDual && p.tile_n > gp::kN && t.n0 + gp::kN < p.N ? 2 : 1;
}

// The product that the producer and the MMA issuer work on in a turn: an item,
// or with a dual epilogue each item of problem 0 and the same one of problem 1.
template <class E, int NP>
__device__ __forceinline__ PairItem pair_turn(const PairProbs<NP>& q, int pair, int pairs,
                                              int iter) {
  PairItem it = pair_item(q, pair, pairs, E::kDual ? iter >> 1 : iter);
  if (E::kDual && it.prob >= 0) it.prob = iter & 1;
  return it;
}

struct PairCtl {
  uint64_t full[gp::kMaxStages];   // leader: both CTAs' copies of a stage landed
  uint64_t empty[gp::kMaxStages];  // each CTA: the MMAs are done with a stage
  uint64_t accf[gp::kBufs];        // each CTA: a buffer is ready
  uint64_t acce[gp::kBufs];        // leader: both epilogues drained a buffer
  uint64_t epi[2][4];              // the epilogue warps' own, two per row quarter
  uint64_t drain;
  uint32_t tmem;
  volatile int abort;
};

// Registers a thread, for a whole warpgroup
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// 2^x and 1 / x, as the hardware approximates them (2^-22 and 2^-23 relative;
// subnormals flushed)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// ---- staging: an epilogue warp's 32 rows in shared memory, in the swizzled
// layout of a tensor copy, so that a lane writes its own row's 16-byte pieces
// without bank conflicts and the copy writes whole lines.  (Row-per-lane
// stores to global memory touch 32 lines an instruction: for a 128 x 256 fp32
// tile that alone took as long as the products of K = 1024.)
//
// Piece j (of four, 16 bytes) of the lane's row: 32 bf16 or 16 fp32 columns,
// rows of 64 bytes, 2 KiB a warp
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
// this thread's writes to shared memory are visible to tensor copies issued after it
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// The warp's staging buffer may be written again (lane 0 issues the stores):
// all but the last BEHIND groups of stores have read theirs.
template <int BEHIND = 0>
__device__ __forceinline__ void stage_free(int lane) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(BEHIND) : "memory");
  __syncwarp();
}
// The warp's writes are visible to the copy that lane 0 issues next.
__device__ __forceinline__ void stage_ready() {
  fence_async_smem();
  __syncwarp();
}

// one look at a barrier's phase, without waiting
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Arrive on a barrier of either CTA without a cluster-scope release: nothing but
// "TMEM has been read" is passed on, which tcgen05.wait::ld and the fence
// before it have settled.  (With the cluster-scope release the epilogue waited
// about 2000 cycles for its earlier global writes at every buffer.)
__device__ __forceinline__ void remote_arrive_local_scope(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

// One lane of the (converged) warp.  The producer and the MMA issuer run their
// loops as whole warps and only issue through this lane: their addresses and
// descriptors are then warp-uniform values.  With the loops inside
// `if (lane == 0)` the issuer spent 1.4 cycles for every cycle of the products
// it issued (K = 4096: 66 % of the MMA rate).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(p));
  return p != 0;
}
// mbar_wait_or_abort by a whole warp, with one answer
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          int32_t* status) {
  for (unsigned long long i = 0; i < kSpinLimit; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if ((i & 255) == 255 && __any_sync(0xffffffffu, *abort != 0)) return false;
  }
  *abort = 1;
  set_status(status, PKM_ERR_TIMEOUT);
  return false;
}

struct EpiWarp {
  int lane, quarter, part;  // rows 32 quarter .. + 31, columns kCols part .. of a buffer
  unsigned char* stage;     // E::kWarpBytes of shared memory, 1024-byte aligned
  unsigned char* shared;    // E::kSharedBytes for all epilogue warps
  uint64_t (*bars)[4];      // two barriers per row quarter
  volatile int* abort;
  int32_t* status;
};

// E: a trivially copyable epilogue with
//   kWarps, kCols         8 warps of 128 columns, or 16 of 64
//   kStages, kWarpBytes, kSharedBytes   ring stages; shared memory per warp, for all
//   kBarArrivals          arrivals of the epilogue warps' own barriers (EpiWarp::bars)
//   kDual                 two products over the same tile (see above)
//   struct State          a warp's state over its tiles, zero-initialised
//   setup(State&, w)      once, by all epilogue warps, before the first tile; they
//                         may meet at named barrier 1 there
//   begin(State&, w, prob, row0, n0, z)        before the buffer is ready
//   tile(State&, w, prob, row0, n0, z, tmem, release)   by a whole warp: rows
//       row0 + lane, columns n0 + kCols part .. at TMEM address `tmem` (lane
//       quarter and column included; a dual epilogue finds the second product
//       256 columns further); n0 is the buffer's first column.  It calls
//       release() once, as soon as it has read TMEM: sixteen warps hold a
//       buffer in registers, and the next products start then and not after
//       the epilogue.
//   abandon(State&, w)    after an abort: lets copies in flight land
// The accumulator itself -> the problem's output map: fp32 (stored or added
// to; slice z is the map's third coordinate) or bf16.
struct StoreOut {
  int64_t rows;
  int cols;
  int bf16, add;
};

constexpr int kStageRowBytes = 64, kStageBytesPerWarp = 32 * kStageRowBytes;

// Four 16-byte pieces of the lane's row -> columns `col` .. of the map's rows
// row0 .. + 31 of slice z.
__device__ __forceinline__ void stage_out(const CUtensorMap* map, const EpiWarp& w, int col,
                                          int64_t row0, int z, const uint4* v, bool add) {
  stage_free(w.lane);
#pragma unroll
  for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(stage64_at(w.stage, w.lane, j)) = v[j];
  stage_ready();
  if (w.lane == 0) {
    if (add)
      tma_add_3d(map, w.stage, col, (int)row0, z);
    else
      tma_store_3d(map, w.stage, col, (int)row0, z);
    bulk_commit();
  }
  __syncwarp();
}

template <class Release>
__device__ __forceinline__ void store_tile(const StoreOut& o, const CUtensorMap* map,
                                           const EpiWarp& w, int64_t row0, int n0, int z,
                                           uint32_t tmem, Release release, float scale = 1.f) {
  const int c0 = n0 + w.part * 64;
  if (row0 >= o.rows || c0 >= o.cols) {  // the whole warp
    release();
    return;
  }
  uint32_t r[64];
  tmem_ld_32x32b_x32(tmem, r);
  tmem_ld_32x32b_x32(tmem + 32, r + 32);
  tmem_ld_wait();
  release();
#pragma unroll
  for (int j = 0; j < 64; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * scale);
  if (o.bf16) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (c0 + 32 * h >= o.cols) break;
      uint4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t* q = r + 32 * h + 8 * j;
        v[j] = make_uint4(pack_bf16x2(__uint_as_float(q[0]), __uint_as_float(q[1])),
                          pack_bf16x2(__uint_as_float(q[2]), __uint_as_float(q[3])),
                          pack_bf16x2(__uint_as_float(q[4]), __uint_as_float(q[5])),
                          pack_bf16x2(__uint_as_float(q[6]), __uint_as_float(q[7])));
      }
      stage_out(map, w, c0 + 32 * h, row0, z, v, o.add);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      if (c0 + 16 * h >= o.cols) break;
      uint4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t* q = r + 16 * h + 4 * j;
        v[j] = make_uint4(q[0], q[1], q[2], q[3]);
      }
      stage_out(map, w, c0 + 16 * h, row0, z, v, o.add);
    }
  }
}

template <int NP, class E>
__global__ void __launch_bounds__(gp::threads<E>(), 1)
    pair_gemm_kernel(const __grid_constant__ PairMaps<NP> maps,
                     const __grid_constant__ PairProbs<NP> probs, const __grid_constant__ E epi,
                     int32_t* status) {
  using namespace gp;
  constexpr int kStages = E::kStages, kStageBytes = stage_bytes<E>(), kEpiWarps = E::kWarps;
  static_assert(kStages <= kMaxStages && E::kWarpBytes % 1024 == 0 && E::kSharedBytes % 16 == 0,
                "shared memory layout");
  static_assert(sizeof(PairCtl) <= 512 && smem_bytes<E>() <= 227 * 1024, "shared memory size");
  static_assert(kEpiWarps * E::kCols == 4 * kN && kEpiWarps <= kMaxWarps, "columns per warp");
  pdl_launch_dependents();
  extern __shared__ unsigned char smem_raw[];
  unsigned char* stages = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* staging = stages + kStages * kStageBytes;
  unsigned char* shared = staging + kEpiWarps * E::kWarpBytes;
  PairCtl* ctl = reinterpret_cast<PairCtl*>(shared + E::kSharedBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&ctl->full[s], 1);   // the leader's producer registers both CTAs' bytes
      mbar_init(&ctl->empty[s], 1);  // the leader's commit
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(&ctl->accf[b], 1);
      mbar_init(&ctl->acce[b], 2 * kEpiWarps);
    }
    for (int q = 0; q < 8; ++q) mbar_init(&ctl->epi[q >> 2][q & 3], E::kBarArrivals);
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
    tmem_alloc_pair(&ctl->tmem, kTileN);
    tmem_relinquish_pair();
  }
  __syncwarp();  // the cluster barrier is warp-aligned: reconverge first
  tc_fence_before();
  cluster_sync_all();  // both CTAs' barriers and TMEM exist before any remote use
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  pdl_wait();  // operands and outputs belong to the kernel before until here

  constexpr int kLead = gp::lead_warps<E>();
  if (warp < kLead) {
    if constexpr (E::kDual) reg_dec<kLeadRegs>();
    if (warp == 0) {
      // ------------------------------------------------------ TMA producer
      const bool issue = elect_one();
      uint32_t issued_mask = 0, issued_par = 0;
      bool ok = true;
      int stage = 0;
      uint32_t phase = 0;
      for (int iter = 0; ok; ++iter) {
        const PairItem it = pair_turn<E>(probs, pair, pairs, iter);
        if (it.prob < 0) break;
        const PairProb& p = probs.p[it.prob];
        const CUtensorMap* ta = &maps.a[it.prob];
        const CUtensorMap* tb = &maps.b[it.prob];
        const PairTile tc = pair_tile(p, it.idx);
        const int am = (int)(tc.m0 + (int64_t)rank * kM);  // this CTA's rows
        const int bn = tc.n0 + (int)rank * kNh;  // this CTA's half of a buffer's columns
        const int bufs = pair_bufs<E>(p, tc);
        const bool amn = p.amn, bmn = p.bmn;
        const int kb0 = tc.z * p.kb_per;
        const int kb1 = min(kb0 + p.kb_per, (p.K + kKB - 1) / kKB);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!warp_wait(&ctl->empty[stage], phase ^ 1, &ctl->abort, status)) {
            ok = false;
            break;
          }
          if (issue) {
            unsigned char* sa = stages + stage * kStageBytes;
            const int kc = kb * kKB;
            const uint32_t bar = map_to(&ctl->full[stage], 0);
            // the leader registers the bytes of both CTAs' copies; a copy of
            // the partner's that lands first only takes the count below zero
            if (leader) mbar_arrive_expect_tx(&ctl->full[stage], 2 * (kABytes + bufs * kBBytes));
            if (amn) {
  #pragma unroll
              for (int j = 0; j < kM / kBox; ++j)
                tma_load_2d_pair(sa + j * kBox * 128, ta, bar, am + j * kBox, kc);
            } else {
              tma_load_2d_pair(sa, ta, bar, kc, am);
            }
            for (int u = 0; u < bufs; ++u) {
              unsigned char* sb = sa + kABytes + u * kBBytes;
              const int n = bn + u * kN;
              if (bmn) {
  #pragma unroll
                for (int j = 0; j < kNh / kBox; ++j)
                  tma_load_2d_pair(sb + j * kBox * 128, tb, bar, n + j * kBox, kc);
              } else {
                tma_load_2d_pair(sb, tb, bar, kc, n);
              }
            }
          }
          __syncwarp();
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
    } else if (warp == 1) {
      // ----------------------------------------------- MMA issuer (leader)
      if (leader) {
        const bool issue = elect_one();
        bool ok = true;
        int stage = 0;
        uint32_t phase = 0;
        uint32_t used0 = 0, used1 = 0;  // times each buffer was filled
        for (int iter = 0; ok; ++iter) {
          const PairItem it = pair_turn<E>(probs, pair, pairs, iter);
          if (it.prob < 0) break;
          const PairProb& p = probs.p[it.prob];
          const bool amn = p.amn, bmn = p.bmn;
          const uint32_t idesc = idesc_bf16_f32(2 * kM, kN) | (amn ? (1u << 15) : 0u) |
                                 (bmn ? (1u << 16) : 0u);
          // one 16-deep step inside a k-block: 32 bytes along a K-major row,
          // 16 lines of 128 bytes of an MN-major tile
          const uint32_t astep = amn ? 2048 >> 4 : 32 >> 4, bstep = bmn ? 2048 >> 4 : 32 >> 4;
          const PairTile tc = pair_tile(p, it.idx);
          const int kb0 = tc.z * p.kb_per;
          const int nkb = min(p.kb_per, (p.K + kKB - 1) / kKB - kb0);
          const bool wide = pair_bufs<E>(p, tc) > 1;
          const int b0 = E::kDual ? it.prob : 0;  // the (first) buffer
          auto products = [&](int st, int u, bool first) {  // k-block in stage st, buffer u
            const uint32_t sa = smem_u32(stages + st * kStageBytes);
            const uint32_t sb = sa + kABytes + (E::kDual ? 0 : u) * kBBytes;
            const uint64_t ad = amn ? smem_desc_mn128(sa) : smem_desc_k128(sa);
            const uint64_t bd = bmn ? smem_desc_mn128(sb) : smem_desc_k128(sb);
  #pragma unroll
            for (int kk = 0; kk < kKB / 16; ++kk)
              tc_mma_f16_pair(tmem + (uint32_t)(u * kN), ad + kk * astep, bd + kk * bstep, idesc,
                              !(first && kk == 0));
          };
          // both epilogues have drained the buffer's last tile
          const uint32_t n_used = E::kDual && b0 ? used1 : used0;
          if (!warp_wait(&ctl->acce[b0], (n_used & 1) ^ 1, &ctl->abort, status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          int back = 0, back_stage = stage;  // k-blocks the second buffer has had, its next stage
          bool open = !wide;                 // the second buffer may be written
          for (int kb = 0; kb < nkb; ++kb) {
            if (!warp_wait(&ctl->full[stage], phase, &ctl->abort, status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (issue) {
              products(stage, b0, kb == 0);
              if (kb == nkb - 1) tc_commit_pair_both(&ctl->accf[b0]);
              if (!wide) tc_commit_pair_both(&ctl->empty[stage]);  // both CTAs may refill the stage
            }
            __syncwarp();
            if (wide) {
              if (!open) {
                // wait only when the ring is full or the tile's last k-block is in
                const uint32_t par = (used1 & 1) ^ 1;
                if (kb + 1 - back == kStages || kb == nkb - 1) {
                  if (!warp_wait(&ctl->acce[1], par, &ctl->abort, status)) {
                    ok = false;
                    break;
                  }
                  open = true;
                } else {
                  open = __all_sync(0xffffffffu, mbar_test_wait(&ctl->acce[1], par));
                }
                if (open) tc_fence_after();
              }
              if (open)
                for (; back <= kb; ++back) {
                  if (issue) {
                    products(back_stage, 1, back == 0);
                    tc_commit_pair_both(&ctl->empty[back_stage]);
                  }
                  __syncwarp();
                  if (++back_stage == kStages) back_stage = 0;
                }
            }
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
          if (!ok) break;
          if (b0)
            ++used1;
          else
            ++used0;
          if (wide) {
            if (issue) tc_commit_pair_both(&ctl->accf[1]);
            __syncwarp();
            ++used1;
          }
        }
        // every MMA issued must complete before either CTA frees TMEM or exits
        if (issue) tc_commit_pair_local(&ctl->drain);
        __syncwarp();
        for (unsigned long long i = 0; i < kSpinLimit; ++i)
          if (mbar_try_wait(&ctl->drain, 0)) break;
      }
    }
  } else {
    // ----------------------------------------------------------- epilogue
    if constexpr (E::kDual) reg_inc<kDualRegs>();
    const int quarter = warp & 3, part = (warp - kLead) >> 2;
    const EpiWarp w{lane, quarter, part, staging + (warp - kLead) * E::kWarpBytes, shared,
                    ctl->epi, &ctl->abort, status};
    const uint32_t mine = tmem + ((uint32_t)(quarter * 32) << 16) + part * E::kCols;
    typename E::State state{};
    epi.setup(state, w);
    uint32_t used[kBufs] = {0, 0};
    bool ok = true;
    for (int iter = 0; ok; ++iter) {
      const PairItem it = pair_item(probs, pair, pairs, iter);
      if (it.prob < 0) break;
      const PairProb& p = probs.p[it.prob];
      const PairTile tc = pair_tile(p, it.idx);
      const int64_t row0 = tc.m0 + (int64_t)rank * kM + quarter * 32;
      const int bufs = pair_bufs<E>(p, tc);
#pragma unroll
      for (int u = 0; u < kBufs; ++u) {
        if (u >= bufs) break;
        const int n0 = tc.n0 + u * kN;
        epi.begin(state, w, it.prob, row0, n0, tc.z);
        bool got = mbar_wait_or_abort(&ctl->accf[u], used[u] & 1, &ctl->abort, status);
        const auto release = [&](int b) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) remote_arrive_local_scope(map_to(&ctl->acce[b], 0));
          __syncwarp();
        };
        if constexpr (E::kDual) {
          if (__all_sync(0xffffffffu, got)) {
            tc_fence_after();
            epi.first(state, w, row0, n0, mine, [&] { release(0); });
            got = mbar_wait_or_abort(&ctl->accf[1], used[u] & 1, &ctl->abort, status);
          } else {
            got = false;
          }
        }
        if (!__all_sync(0xffffffffu, got)) {
          epi.abandon(state, w);
          ok = false;
          break;
        }
        ++used[u];
        tc_fence_after();
        epi.tile(state, w, it.prob, row0, n0, tc.z, mine + (E::kDual ? 1 : u) * kN,
                 [&] { release(E::kDual ? 1 : u); });
      }
    }
    if (E::kWarpBytes > 0) stage_free(lane);  // no store reads shared memory any more
  }

  // both CTAs finished: the leader's MMAs no longer read either CTA's shared
  // memory or write either CTA's TMEM
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, kTileN);
}

// out = the sum of nz slices of 8 n8 fp32 values, in slice order; the second
// half of the grid (y = 1) does the same for part2 and out2.
template <pkm_dtype GT>
__global__ void __launch_bounds__(256) slice_sum_kernel(const float* __restrict__ part, int nz,
                                                        int64_t n8,
                                                        typename Elem<GT>::T* __restrict__ out,
                                                        const float* __restrict__ part2,
                                                        typename Elem<GT>::T* __restrict__ out2) {
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.y) {
    part = part2;
    out = out2;
  }
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8;
       i += (int64_t)gridDim.x * 256) {
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll 4
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
                                    cudaStream_t st, const float* part2 = nullptr,
                                    void* out2 = nullptr) {
  const int64_t n8 = n / 8, blocks = (n8 + 255) / 256;
  const dim3 grid((unsigned)(blocks < 148 * 8 ? blocks : 148 * 8), part2 ? 2 : 1);
  return dt == PKM_BF16
             ? launch_maybe_pdl(true, slice_sum_kernel<PKM_BF16>, grid, dim3(256), 0, st, part, nz,
                                n8, static_cast<__nv_bfloat16*>(out), part2,
                                static_cast<__nv_bfloat16*>(out2))
             : launch_maybe_pdl(true, slice_sum_kernel<PKM_F32>, grid, dim3(256), 0, st, part, nz,
                                n8, static_cast<float*>(out), part2, static_cast<float*>(out2));
}

// Tensor map of an operand with `rows` rows (M or N) and depth K, `ld`
// elements from row to row: [rows][K], or [K][rows] when mn.
inline bool pair_map(CUtensorMap* m, const void* base, int64_t rows, int K, int64_t ld, bool mn) {
  const uint64_t dims[2] = {mn ? (uint64_t)rows : (uint64_t)K, mn ? (uint64_t)K : (uint64_t)rows};
  const uint64_t strides[1] = {(uint64_t)ld * 2};
  const uint32_t box[2] = {(uint32_t)gp::kBox, mn ? (uint32_t)gp::kKB : (uint32_t)gp::kM};
  return make_tmap_bf16(m, base, 2, dims, strides, box);
}

// Tensor map of an epilogue's output: [slices][rows][cols] with `ld` elements
// from row to row; boxes of 32 rows and 64 bytes of columns.
inline bool pair_out_map(CUtensorMap* m, const void* base, int64_t cols, int64_t rows,
                         int64_t slices, int64_t ld, pkm_dtype dt) {
  auto enc = tmap_encoder();
  if (!enc) return false;
  const int b = dt == PKM_F32 ? 4 : 2;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)slices};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * b, (cuuint64_t)(ld * rows) * b};
  const cuuint32_t box[3] = {(cuuint32_t)(kStageRowBytes / b), 32, 1}, one[3] = {1, 1, 1};
  return enc(m, dt == PKM_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
             3, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pairs of SMs that the host's plans count on (148 SMs).
constexpr int kPlanPairs = 74;

// A problem's item in units of one 256-column k-block: its products, and about
// six such steps of the epilogue that nothing covers.
inline int64_t pair_len(int64_t kb, int tile_n) { return kb * (tile_n / gp::kN) + 6; }

// Columns of a tile of a launch's only problem, 512 or 256: those whose longest
// pair of SMs has less to do.  Measured as the loss (us, 512 and 256 columns):
// 8192 x 32768 x 1024 413 and 426, 256 x 32768 x 1024 22.9 and 24.6, but 37 x
// 50021 x 512 23.3 and 21.0 (98 tiles of 512 on 74 pairs are two rounds, 196 of
// 256 three of half the length).
inline int pair_tile_n(int64_t M, int N, int K, int64_t nz) {
  const int64_t rows = (M + 2 * gp::kM - 1) / (2 * gp::kM) * nz;
  const int64_t kb = ((K + gp::kKB - 1) / gp::kKB + nz - 1) / nz;
  const auto span = [&](int tn) {
    return (rows * ((N + tn - 1) / tn) + kPlanPairs - 1) / kPlanPairs * pair_len(kb, tn);
  };
  return span(gp::kN) < span(gp::kTileN) ? gp::kN : gp::kTileN;
}

inline PairProb pair_prob(int64_t M, int N, int K, bool amn, bool bmn, int nz = 1,
                          int group_m = 1, int tile_n = 0) {
  const int kb = (K + gp::kKB - 1) / gp::kKB;
  const int per = kb > nz ? (kb + nz - 1) / nz : 1;  // every slice gets at least one k-block
  PairProb p{};
  p.M = M;
  p.N = N;
  p.K = K;
  p.tiles_m = (int)((M + 2 * gp::kM - 1) / (2 * gp::kM));
  p.tile_n = tile_n ? tile_n : pair_tile_n(M, N, K, nz);
  p.tiles_n = (N + p.tile_n - 1) / p.tile_n;
  p.kb_per = per;
  p.nz = (kb + per - 1) / per;
  p.amn = amn;
  p.bmn = bmn;
  p.group_m = group_m;
  return p;
}
inline int64_t pair_items(const PairProb& p) { return (int64_t)p.tiles_m * p.tiles_n * p.nz; }

// The longest pair's work when n0 items of len0 and n1 of len1 are dealt out
// as pair_item does; *extra receives the best evening-out.
inline int64_t pair_span(int64_t n0, int64_t len0, int64_t n1, int64_t len1, int pairs,
                         int* extra = nullptr) {
  const int64_t r = n0 % pairs, lo = n0 / pairs;
  int64_t best = -1;
  const int64_t near = r && n1 ? len0 / len1 : 0;  // about what evens a long item out
  for (int64_t x = near > 1 ? near - 1 : 0; x <= near + (r && n1); ++x) {
    const int64_t early = x * (pairs - r) < n1 ? x * (pairs - r) : n1, rest = n1 - early;
    const int64_t each = rest / pairs, more = rest % pairs;  // `more` pairs, from r on, take one more
    const int64_t lo_span =
        lo * len0 + ((early + pairs - r - 1) / (pairs - r) + each + (more > 0)) * len1;
    const int64_t hi_span = r ? (lo + 1) * len0 + (each + (more > pairs - r)) * len1 : 0;
    const int64_t span = lo_span > hi_span ? lo_span : hi_span;
    if (best < 0 || span < best) {
      best = span;
      if (extra) *extra = (int)x;
    }
  }
  return best;
}

// How a launch of two lists is cut: the first list's `kb0` k-blocks into nz
// slices (at most max_nz, of at least min_kb), tiles of 256 or 512 columns.
// items0/1(tile_n): tiles of a list; slice_cost: what a slice adds, in units.
struct PairPlan {
  int nz = 1, tile0 = gp::kTileN, tile1 = gp::kTileN;
  int64_t cost = -1;
};
template <class F0, class F1>
inline PairPlan pair_plan(F0 items0, int64_t kb0, int max_nz, int min_kb, double slice_cost,
                          F1 items1, int64_t kb1) {
  PairPlan best;
  for (int64_t nz = 1; nz <= max_nz && (nz == 1 || nz * min_kb <= kb0);
       nz += nz < 8 ? 1 : nz < 16 ? 2 : 8) {
    const int64_t per = kb0 > nz ? (kb0 + nz - 1) / nz : 1, z = kb0 > 0 ? (kb0 + per - 1) / per : 1;
    if (z != nz) continue;  // the same cut as a smaller number
    for (int t = 0; t < 4; ++t) {
      const int t0 = t & 1 ? gp::kN : gp::kTileN, t1 = t & 2 ? gp::kN : gp::kTileN;
      const int64_t cost =
          pair_span(items0(t0) * z, pair_len(per, t0), items1(t1), pair_len(kb1, t1), kPlanPairs) +
          (int64_t)(slice_cost * z);
      if (best.cost < 0 || cost < best.cost) best = PairPlan{(int)z, t0, t1, cost};
    }
  }
  return best;
}

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
  cfg.blockDim = dim3(gp::threads<E>(), 1, 1);
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
  if (E::kDual)
    n0 = pair_items(probs.p[0]);
  else
    for (int i = 0; i < NP; ++i) (i < probs.first ? n0 : n1) += pair_items(probs.p[i]);
  if (n0 + n1 >= (int64_t(1) << 30)) return cudaErrorInvalidValue;
  const int pairs = (int)(n0 + n1 < slots ? n0 + n1 : slots);
  probs.sched = PairSched{(int)n0, (int)n1, 0};
  if (n1 > 0)
    pair_span(n0, pair_len(probs.p[0].kb_per, probs.p[0].tile_n), n1,
              pair_len(probs.p[probs.first].kb_per, probs.p[probs.first].tile_n), pairs,
              &probs.sched.extra);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * pairs), 1, 1);
  cfg.blockDim = dim3(gp::threads<E>(), 1, 1);
  cfg.dynamicSmemBytes = gp::smem_bytes<E>();
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, pair_gemm_kernel<NP, E>, maps, probs, epi, status);
}

}  // namespace pkm
