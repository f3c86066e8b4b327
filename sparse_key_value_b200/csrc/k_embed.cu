// k_embed.cu -- the token embedding with a scale, and its gradient by sorted
// tokens.
//
// Forward: out[t] = scale * table[ids[t]], one rounding.  Bound by memory:
// the distinct rows and the output.
//
// Backward: grad[r] = scale * sum of dout[t] over the tokens t with ids[t] = r,
// every row of the table's gradient written.  Launches:
//   1. embed_sort_kernel: one cluster sorts the tokens by id (stable radix
//      sort, counts and tokens exchanged through distributed shared memory) and
//      marks the rows that occur in a bitmap;
//      embed_zero_kernel: meanwhile zeroes the first rows of the gradient on
//      the other SMs (started early by programmatic dependent launch).
//   2. embed_sum_kernel: the sorted list is cut into chunks of kChunk entries,
//      one block sums a chunk's parts in order; the blocks after those zero the
//      other rows that no token reads.
//   3. embed_join_kernel: the parts of an id that covers three chunks or more,
//      joined in chunk order (up to kJoinMost tokens by the sums' own blocks).
// Lists of at most kRankMost tokens are sorted by counting, for each token, the
// tokens before it in the sorted list (embed_rank_kernel): one pass without
// barriers between blocks, and the filling blocks look into the list itself
// instead of a bitmap.
// Lists of more than kSortMost tokens go through the library's multi-block
// radix sort.
// No atomics on values: the same bits every run, and a frequent id spreads
// over many blocks (a short list's over the warps of a block).
// Measured on one B200: forward of 16384 x 1024 bf16 9.2 us (48 MB distinct:
// 5.2 TB/s, the rest in L2); gradient of those tokens over 131072 x 1024 fp32
// 99.7 us, bound by the write of its 537 MB (5.7 TB/s with reading dout, over all
// launches: the sort's 17 us go beside the first 112 MiB of zeros); 65536 tokens
// 170 us and 131072 tokens 254, bound by the sort, which eight SMs do through
// global memory; added to an existing gradient, where no zeros hide the sort,
// 16384 tokens 40 us and 65536 110; 509 tokens over 32003 x 520 fp32 17.5 us and
// 512 over 8192 x 512 12.7, two dependent launches.
#include "kernels.h"
#include "q8.cuh"
#include "tc_pair.cuh"

namespace pkm {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 16;   // sorted tokens per block
constexpr int kAhead = 8;    // rows of dout in flight per thread
// Tokens sorted by counting, at most (counting is quadratic).  The whole
// gradient, by counting and by the cluster: over 32768 x 1024 fp32 512 tokens
// 24.6 and 28.4 us, 1024 27.2 and 29.6, 1536 35.3 and 29.3, 2048 32.6 and 30.0,
// 4096 46.7 and 31.8; over 8192 x 512 512 12.7 and 16.9, 1024 16.7 and 17.7, 2048
// 20.7 and 18.4; added to 131072 x 1024 512 11.4 and 18.0, 1024 16.8 and 19.9,
// 1536 24.9 and 20.2, 2048 18.7 and 20.5.  Up to kJoinMost counting is ahead
// everywhere; from there to this limit the cluster mostly is, by 2 to 6 us.
constexpr int kRankMost = 2048;
// Tokens whose long ids' parts are joined by the sums' own blocks, at most.  The
// gradient with the join's launch and without: 100 tokens over 8192 x 512 13.5
// and 11.4 us, 512 13.7 and 12.7, 1024 over 32768 x 1024 31.6 and 27.2; 2048 32.6
// and 35.2.  Where all tokens are of two ids a block joins T / 32 parts: 1024
// over 8192 x 512 13.7 and 17.9, 2048 19.9 and 28.1.
constexpr int kJoinMost = 1024;
constexpr int kSortThreads = 1024;
constexpr int kSortCluster = 8;
// Tokens per thread of the sorting cluster, at most.  The whole gradient over
// 131072 x 1024 fp32, by the cluster and by the multi-block sort: 40000 tokens 137
// and 201 us, 65536 170 and 220, 131072 255 and 261; added to an existing one
// 65536 110 and 156, 131072 193 and 207; twice as many over 131072 x 512 333 and
// 242.
constexpr int kSortRounds = 16;
constexpr int64_t kSortMost = (int64_t)kSortThreads * kSortRounds * kSortCluster;
constexpr int kMaxDigit = 9;     // bits per pass
constexpr int kSumUnits = 128;  // 8-column units (threads) per block of the sums

// lanes that share a row: the power of two that holds its units, at most 32
int lanes_per_row(int d) {
  int l = 1;
  while (l < 32 && l * kUnit < d) l *= 2;
  return l;
}

template <pkm_dtype DT>
__global__ void __launch_bounds__(kThreads) embed_fwd_kernel(
    const typename Elem<DT>::T* __restrict__ table, int64_t n_rows, int d, int lpr,
    const int32_t* __restrict__ ids, int64_t T, float scale, int has_pad, int32_t pad,
    typename Elem<DT>::T* __restrict__ out, int32_t* status) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t t = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / lpr;
  if (t >= T) return;
  const int l = threadIdx.x % lpr;
  const int32_t id = ids[t];
  const bool padded = has_pad && id == pad;
  const bool ok = !padded && id >= 0 && id < n_rows;
  if (!ok && !padded && l == 0) set_status(status, PKM_ERR_DEVICE);
  const typename Elem<DT>::T* row = table + (int64_t)(ok ? id : 0) * d;
  typename Elem<DT>::T* dst = out + t * d;
  for (int c0 = l * kUnit; c0 < d; c0 += 4 * lpr * kUnit) {
    Raw8<DT> f[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = c0 + u * lpr * kUnit;
      if (ok && c < d) f[u].load(row + c);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = c0 + u * lpr * kUnit;
      if (c >= d) break;
      float v[8];
      f[u].unpack(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = ok ? v[e] * scale : 0.f;
      store8<DT>(dst + c, v);
    }
  }
}

// The sort key of an id: the id itself, or n_rows (sorts last, never summed)
// for the padding id and ids outside the table.
__device__ __forceinline__ uint32_t embed_key(int32_t id, int64_t n_rows, int has_pad, int32_t pad,
                                              int32_t* status) {
  const bool padded = has_pad && id == pad;
  const bool ok = !padded && id >= 0 && id < n_rows;
  if (!ok && !padded) set_status(status, PKM_ERR_DEVICE);
  return ok ? (uint32_t)id : (uint32_t)n_rows;
}

__global__ void embed_keys_kernel(const int32_t* __restrict__ ids, int64_t T, int64_t n_rows,
                                  int has_pad, int32_t pad, uint32_t* __restrict__ keys,
                                  uint32_t* __restrict__ pos, uint32_t* n_cross,
                                  int32_t* status) {
  if (blockIdx.x == 0 && threadIdx.x == 0) *n_cross = 0;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < T;
       i += (int64_t)gridDim.x * blockDim.x) {
    keys[i] = embed_key(ids[i], n_rows, has_pad, pad, status);
    pos[i] = (uint32_t)i;
  }
}

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

struct EmbedSort {
  const int32_t* ids;
  int64_t T, n_rows;
  int has_pad;
  int32_t pad;
  int digit, passes, rounds;
  uint32_t *key[2], *pos[2];  // [0] receives the sorted list
  uint32_t* bitmap;           // rows that occur, or null
  int64_t words;
  uint32_t* n_cross;          // ids that cross chunks, counted by the sums; zeroed here
  uint32_t* done;             // short lists: parts of such an id, counted; zeroed here
  int n_done;
  uint4* fill;                // zeroed beside the sort, or null
  int64_t fill_units;
};

// Dynamic shared memory: the tokens passed on (short lists) or each token's
// rank (long ones), the warps' digit counts, the CTA's digit totals.
size_t sort_smem(int digit, int rounds, bool shared_list) {
  return ((size_t)32 << digit) * 2 + ((size_t)4 << digit) +
         (size_t)rounds * kSortThreads * (shared_list ? 8 : 2);
}

__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

// One digit's counts and places, shared by the two sorts below: `cnt` holds the
// warps' digit counts, `total` the CTA's.  Afterwards cnt[w][d] is the number
// of this CTA's tokens with digit d in the warps before w and total[d] the
// first place of the CTA's tokens with digit d.  Three CTA barriers' worth of
// work, two of them over the cluster.
__device__ __forceinline__ void sort_places(uint16_t* cnt, uint32_t* total, uint32_t* scan,
                                            int bins, uint32_t ncta, uint32_t rank) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __syncthreads();
  if (tid < bins) {
    uint32_t c[32];
#pragma unroll
    for (int w = 0; w < 32; ++w) c[w] = cnt[w * bins + tid];
    uint32_t run = 0;
#pragma unroll
    for (int w = 0; w < 32; ++w) {
      cnt[w * bins + tid] = (uint16_t)run;
      run += c[w];
    }
    total[tid] = run;
  }
  __syncwarp();
  cluster_sync_all();
  // the smaller digits of every CTA, then the same digit of the CTAs before this one
  uint32_t before = 0, all = 0;
  if (tid < bins) {
#pragma unroll
    for (uint32_t c = 0; c < kSortCluster; ++c) {
      const uint32_t t = c < ncta ? ld_cluster(map_to(&total[tid], c)) : 0u;
      before += c < rank ? t : 0u;
      all += t;
    }
  }
  uint32_t incl = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) scan[warp] = incl;
  __syncwarp();
  cluster_sync_all();  // every CTA has read the totals; `scan` is written
  if (tid < bins) {
    uint32_t base = incl - all + before;
    for (int w = 0; w < warp; ++w) base += scan[w];
    total[tid] = base;
  }
  __syncthreads();
}

// The rank of the lane's digit among the warp's earlier tokens with it.  The
// lanes of equal digit by one ballot a bit (__match_any_sync took 3.5 k cycles
// a round of 32 warps).
__device__ __forceinline__ uint32_t digit_rank(uint16_t* mine, uint32_t d, bool valid, int bits) {
  const uint32_t lt = (1u << (threadIdx.x & 31)) - 1u;
  uint32_t peers = __ballot_sync(0xffffffffu, valid);
#pragma unroll
  for (int b = 0; b < kMaxDigit; ++b) {
    if (b >= bits) break;  // the same for every thread
    const uint32_t one = __ballot_sync(0xffffffffu, (d >> b) & 1);
    peers &= (d >> b) & 1 ? one : ~one;
  }
  const uint32_t before = valid ? mine[d] : 0u;
  __syncwarp();
  if (valid && (peers & lt) == 0) mine[d] = (uint16_t)(before + __popc(peers));
  __syncwarp();
  return before + __popc(peers & lt);
}

__device__ __forceinline__ void sort_clear(uint16_t* cnt, int bins) {
  uint4* c = reinterpret_cast<uint4*>(cnt);
  for (int b = threadIdx.x; b < 4 * bins; b += kSortThreads) c[b] = make_uint4(0, 0, 0, 0);
  __syncthreads();
}

// Sort by counting: token i's place is the number of tokens with a smaller key,
// or the same key and an earlier position.  A block places 32 tokens, one per
// lane, each warp counting over its eighth of the list.  The blocks after them
// fill.
constexpr int kRankWarps = 8;

__global__ void __launch_bounds__(32 * kRankWarps) embed_rank_kernel(const EmbedSort p, int blocks,
                                                                     int32_t* status) {
  pdl_launch_dependents();
  pdl_wait();
  if ((int)blockIdx.x >= blocks) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int64_t i = (int64_t)(blockIdx.x - blocks) * 32 * kRankWarps + threadIdx.x;
         i < p.fill_units; i += (int64_t)(gridDim.x - blocks) * 32 * kRankWarps)
      __stcs(p.fill + i, zero);
    return;
  }
  __shared__ __align__(16) uint32_t keys[kRankMost];
  __shared__ int count[kRankWarps][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, T = (int)p.T;
  if (blockIdx.x == 0 && tid == 0) *p.n_cross = 0;
  for (int i = blockIdx.x * 32 * kRankWarps + tid; i < p.n_done; i += blocks * 32 * kRankWarps)
    p.done[i] = 0;
  for (int i = tid; i < kRankMost; i += 32 * kRankWarps)
    keys[i] = i < T ? embed_key(p.ids[i], p.n_rows, p.has_pad, p.pad,
                                blockIdx.x == 0 ? status : nullptr)
                    : 0xffffffffu;  // after every key
  __syncthreads();
  const int me = blockIdx.x * 32 + lane;
  const uint32_t k = keys[me < T ? me : 0];
  const int each = ((T + kRankWarps - 1) / kRankWarps + 3) / 4 * 4;  // tokens per warp
  int n = 0;
  for (int j = warp * each; j < min(T, (warp + 1) * each); j += 4) {
    const uint4 q = *reinterpret_cast<const uint4*>(keys + j);
    n += (q.x < k) + (q.y < k) + (q.z < k) + (q.w < k);
    n += (q.x == k && j < me) + (q.y == k && j + 1 < me) + (q.z == k && j + 2 < me) +
         (q.w == k && j + 3 < me);
  }
  count[warp][lane] = n;
  __syncthreads();
  if (warp == 0 && me < T) {
    for (int w = 1; w < kRankWarps; ++w) n += count[w][lane];
    p.key[0][n] = k;
    p.pos[0][n] = (uint32_t)me;
  }
}

// Zeroes the first rows of the gradient while the sort before it runs, which
// touches none of them; ends after it, so that who waits for this kernel has
// waited for both.
constexpr int kZeroUnits = 1024;  // of 16 bytes, per block and turn
constexpr int kZeroBlocks = 4 * 140;  // at work at a time, beside the sort's eight
__global__ void __launch_bounds__(kThreads) embed_zero_kernel(uint4* fill, int64_t units) {
  pdl_launch_dependents();
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int64_t i0 = (int64_t)blockIdx.x * kZeroUnits + threadIdx.x; i0 < units;
       i0 += (int64_t)gridDim.x * kZeroUnits)
#pragma unroll
    for (int u = 0; u < kZeroUnits / kThreads; ++u)
      if (i0 + u * kThreads < units) __stcs(fill + i0 + u * kThreads, zero);
  pdl_wait();
}

// Lists of at most R * kSortThreads tokens per CTA: tokens stay in registers
// within a pass and pass to their next CTA through distributed shared memory,
// so global memory (busy with the fill) is met only at both ends.
template <int R>
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const EmbedSort p,
                                                                  int32_t* status) {
  pdl_wait();  // first: the zeros that start now touch what earlier kernels may use
  pdl_launch_dependents();
  const uint32_t ncta = cluster_size(), rank = cluster_rank();
  if (rank == 0 && threadIdx.x == 0) *p.n_cross = 0;
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int kOwn = R * kSortThreads;  // tokens of a CTA
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bins = 1 << p.digit;
  uint2* list = reinterpret_cast<uint2*>(smem);  // [kOwn] key, position
  uint16_t* cnt = reinterpret_cast<uint16_t*>(smem + (size_t)kOwn * 8);  // [32][bins]
  uint32_t* total = reinterpret_cast<uint32_t*>(cnt + 32 * bins);         // [bins]
  __shared__ uint32_t scan[32];
  // a warp owns R * 32 consecutive tokens, so (CTA, warp, round, lane) is the
  // list's order
  const int l0 = warp * R * 32 + lane;
  const int64_t i0 = (int64_t)rank * kOwn + l0;
  uint32_t key[R], pos[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t i = i0 + r * 32;
    pos[r] = (uint32_t)i;
    key[r] = i < p.T ? embed_key(p.ids[i], p.n_rows, p.has_pad, p.pad, status) : 0u;
  }
  if (p.bitmap)
    for (int64_t w = (int64_t)rank * kSortThreads + tid; w < p.words;
         w += (int64_t)ncta * kSortThreads)
      p.bitmap[w] = 0;
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.digit;
    sort_clear(cnt, bins);
    uint32_t rk[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
      rk[r] = digit_rank(cnt + warp * bins, (key[r] >> shift) & (bins - 1), i0 + r * 32 < p.T,
                         p.digit);
    sort_places(cnt, total, scan, bins, ncta, rank);
    const bool last = pass == p.passes - 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (i0 + r * 32 >= p.T) continue;
      const uint32_t d = (key[r] >> shift) & (bins - 1);
      const uint32_t dst = total[d] + cnt[warp * bins + d] + rk[r];
      if (last) {
        p.key[0][dst] = key[r];
        p.pos[0][dst] = pos[r];
        if (p.bitmap && key[r] < p.n_rows) atomicOr(p.bitmap + (key[r] >> 5), 1u << (key[r] & 31));
      } else {
        st_cluster(map_to(&list[dst % kOwn], dst / kOwn), key[r], pos[r]);
      }
    }
    __syncwarp();
    cluster_sync_all();  // the pass's list is complete; `total` may be rewritten
    if (!last) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint2 v = list[l0 + r * 32];
        key[r] = v.x;
        pos[r] = v.y;
      }
    }
  }
}

// Longer lists, up to kSortMost tokens: the passes' lists in global memory.
__global__ void __launch_bounds__(kSortThreads) embed_sort_long_kernel(const EmbedSort p,
                                                                       int32_t* status) {
  pdl_wait();  // first: the zeros that start now touch what earlier kernels may use
  pdl_launch_dependents();
  const uint32_t ncta = cluster_size(), rank = cluster_rank();
  if (rank == 0 && threadIdx.x == 0) *p.n_cross = 0;
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bins = 1 << p.digit;
  uint16_t* cnt = reinterpret_cast<uint16_t*>(smem);               // [32][bins]
  uint32_t* total = reinterpret_cast<uint32_t*>(cnt + 32 * bins);  // [bins]
  uint16_t* ranks = reinterpret_cast<uint16_t*>(total + bins);
  __shared__ uint32_t scan[32];
  const int64_t i0 = (int64_t)rank * p.rounds * kSortThreads + (int64_t)warp * p.rounds * 32 + lane;
  if (p.bitmap)
    for (int64_t w = (int64_t)rank * kSortThreads + tid; w < p.words;
         w += (int64_t)ncta * kSortThreads)
      p.bitmap[w] = 0;
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.digit;
    const int out = (p.passes - 1 - pass) & 1;
    const uint32_t* skey = p.key[out ^ 1];
    const uint32_t* spos = p.pos[out ^ 1];
    sort_clear(cnt, bins);
    for (int r = 0; r < p.rounds; ++r) {
      const int64_t i = i0 + r * 32;
      uint32_t k = 0;
      if (i < p.T)
        k = pass == 0 ? embed_key(p.ids[i], p.n_rows, p.has_pad, p.pad, status)
                      : __ldcg(skey + i);
      ranks[r * kSortThreads + tid] = (uint16_t)digit_rank(
          cnt + warp * bins, (k >> shift) & (bins - 1), i < p.T, p.digit);
    }
    sort_places(cnt, total, scan, bins, ncta, rank);
    for (int r = 0; r < p.rounds; ++r) {
      const int64_t i = i0 + r * 32;
      if (i >= p.T) break;
      const uint32_t k = pass == 0 ? embed_key(p.ids[i], p.n_rows, p.has_pad, p.pad, nullptr)
                                   : __ldcg(skey + i);
      const uint32_t d = (k >> shift) & (bins - 1);
      const uint32_t dst = total[d] + cnt[warp * bins + d] + ranks[r * kSortThreads + tid];
      p.key[out][dst] = k;
      p.pos[out][dst] = pass == 0 ? (uint32_t)i : __ldcg(spos + i);
      if (pass == 0 && p.bitmap && k < p.n_rows) atomicOr(p.bitmap + (k >> 5), 1u << (k & 31));
    }
    __syncwarp();
    cluster_sync_all();  // the pass's list is complete; `total` may be rewritten
  }
}

template <pkm_dtype GT>
__device__ __forceinline__ void write_grad(typename Elem<GT>::T* g, const float* acc, float scale,
                                           bool add) {
  float o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = 0.f;
  if (add) load8<GT>(g, o);
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = add ? fmaf(acc[e], scale, o[e]) : acc[e] * scale;
  store8<GT>(g, o);
}

// Eight columns of a part that another block wrote
__device__ __forceinline__ void part_load(const float* p, float* f) {
#pragma unroll
  for (int e = 0; e < 8; e += 4) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(p + e));
    f[e] = v.x, f[e + 1] = v.y, f[e + 2] = v.z, f[e + 3] = v.w;
  }
}

struct EmbedFill {
  bool on;
  const uint32_t* bitmap;  // rows that occur, or null: look into the sorted keys
  int64_t n_rows, first;   // rows first .. n_rows - 1; `first` is a multiple of 32
};

// Zeroes those of 32 rows that no token reads.
template <pkm_dtype GT>
__device__ __forceinline__ void fill_rows(const EmbedFill& f, int64_t block, int d,
                                          const uint32_t* skey, int T,
                                          typename Elem<GT>::T* grad) {
  const int64_t r0 = f.first + block * 32;
  uint32_t used;
  if (f.bitmap) {
    used = f.bitmap[r0 >> 5];
  } else {
    __shared__ uint32_t found;
    if (threadIdx.x == 0) found = 0;
    __syncthreads();
    uint32_t mine = 0;
    for (int i = threadIdx.x; i < T; i += kSumUnits) {
      const int64_t r = (int64_t)skey[i] - r0;
      if (r >= 0 && r < 32) mine |= 1u << r;
    }
    if (mine) atomicOr(&found, mine);
    __syncthreads();
    used = found;
  }
  const int units = d / Elem<GT>::kVec;  // 16 bytes each
  const int rows = (int)min((int64_t)32, f.n_rows - r0);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // a warp per row where its last turn leaves few lanes idle, else the rows as
  // if they were one (with a division per store)
  if ((units + 31) / 32 * 32 - units > units / 8) {
    uint4* g = reinterpret_cast<uint4*>(grad + r0 * d);
    for (int i = threadIdx.x; i < rows * units; i += kSumUnits)
      if (!(used >> (i / units) & 1)) __stcs(g + i, zero);
    return;
  }
  for (int r = threadIdx.x >> 5; r < rows; r += kSumUnits / 32) {
    if (used >> r & 1) continue;
    uint4* g = reinterpret_cast<uint4*>(grad + (r0 + r) * d);
#pragma unroll 8
    for (int i = threadIdx.x & 31; i < units; i += 32) __stcs(g + i, zero);
  }
}

// The first n_sum blocks: one per chunk and slice of 8 * kSumUnits columns, a
// thread owns 8 columns and walks the chunk's entries in order, kAhead rows in
// flight.  The blocks after them zero the rows without tokens.
// JOIN (short lists): the last block to finish a part of an id over three chunks
// or more, counted in `done`, sums the parts in chunk order, instead of a launch
// of its own.
template <pkm_dtype DT, pkm_dtype GT, bool JOIN>
__global__ void __launch_bounds__(kSumUnits) embed_sum_kernel(
    const uint32_t* __restrict__ skey, const uint32_t* __restrict__ spos, int64_t T,
    uint32_t mark, const typename Elem<DT>::T* __restrict__ dout, int d, float scale, int add,
    typename Elem<GT>::T* __restrict__ grad, float* __restrict__ first, float* __restrict__ last,
    int slices, int64_t n_sum, uint32_t* __restrict__ n_cross, uint4* __restrict__ cross,
    uint32_t* __restrict__ done, const EmbedFill fill) {
  pdl_launch_dependents();
  pdl_wait();
  if ((int64_t)blockIdx.x >= n_sum) {
    fill_rows<GT>(fill, blockIdx.x - n_sum, d, skey, (int)T, grad);
    return;
  }
  // this chunk's keys and the next one's: [0] is the key before the chunk
  __shared__ uint32_t keys[2 * kChunk + 2];
  __shared__ uint32_t rows[2 * kChunk];
  const int64_t c = blockIdx.x / slices, i0 = c * kChunk;
  const int len = (int)min((int64_t)kChunk, T - i0);
  for (int j = threadIdx.x; j < 2 * kChunk + 2; j += blockDim.x) {
    const int64_t i = i0 + j - 1;
    const bool in = i >= 0 && i < T;
    keys[j] = in ? skey[i] : mark;
    if (in && j >= 1 && j <= 2 * kChunk) rows[j - 1] = spos[i];
  }
  // what the 32 chunks after this one begin with
  const int64_t chunks = (T + kChunk - 1) / kChunk;
  uint32_t ahead = mark;
  if (threadIdx.x < 32 && c + 1 + threadIdx.x < chunks)
    ahead = skey[(c + 1 + threadIdx.x) * kChunk];
  // the key before the last chunk (mark sorts last, so it is no earlier key)
  const uint32_t before = i0 > kChunk ? skey[i0 - kChunk - 1] : mark;
  __syncthreads();
  // An id over two chunks is summed whole by the chunk it begins in; one over
  // three or more goes in parts, `first` and `last`, to the join.
  int e0 = 0, e1 = len;
  bool starts = keys[0] != keys[1] || keys[1] == mark;
  if (!starts && before != keys[1] && keys[len + 1] != keys[1]) {
    while (e0 < len && keys[e0 + 1] == keys[0]) ++e0;
    starts = true;
  }
  const uint32_t tail = keys[len];
  const bool goes_over = len == kChunk && tail != mark && keys[len + 1] == tail &&
                         !(keys[0] == tail && keys[1] == tail);
  if (goes_over && keys[2 * kChunk + 1] != tail)
    while (e1 < 2 * kChunk && keys[e1 + 1] == tail) ++e1;
  const bool leads = !starts, trails = goes_over && e1 == len;  // parts for the join
  // the end of a long id that this chunk ends with (the first warp's)
  int64_t stop = c + 1;
  if (threadIdx.x < 32 && (trails || (JOIN && leads && tail == keys[1]))) {
    uint32_t m = __ballot_sync(0xffffffffu, ahead == tail);  // 32 chunks at a time
    while (m == 0xffffffffu) {
      stop += 32;
      const int64_t q = stop + threadIdx.x;
      m = __ballot_sync(0xffffffffu, q < chunks && skey[q * kChunk] == tail);
    }
    stop += __ffs(~m) - 1;
    if (!JOIN && threadIdx.x == 0 && blockIdx.x % slices == 0)  // any order: entries stand alone
      cross[atomicAdd(n_cross, 1u)] = make_uint4((uint32_t)c, (uint32_t)stop, tail, 0);
  }
  const int col = ((int)(blockIdx.x % slices) * kSumUnits + threadIdx.x) * kUnit;
  if (!JOIN && col >= d) return;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  for (int j0 = e0; (!JOIN || col < d) && j0 < e1 && keys[j0 + 1] != mark; j0 += kAhead) {
    Raw8<DT> raw[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (j0 + u < e1 && keys[j0 + u + 1] != mark)
        raw[u].load(dout + (int64_t)rows[j0 + u] * d + col);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = j0 + u;
      if (j >= e1 || keys[j + 1] == mark) break;
      float f[8];
      raw[u].unpack(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += f[e];
      const uint32_t key = keys[j + 1];
      const bool goes_on = keys[j + 2] == key;
      if (goes_on && j + 1 < e1) continue;
      if (!starts)
        store8<PKM_F32>(first + c * d + col, acc);
      else if (goes_on)
        store8<PKM_F32>(last + c * d + col, acc);
      else
        write_grad<GT>(grad + (int64_t)key * d + col, acc, scale, add);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = 0.f;
      starts = true;
    }
  }
  if constexpr (JOIN) {
    if (leads || trails) __threadfence();  // the parts before the counts
    __shared__ uint32_t ids[2][2];         // an id whose parts are all there: begin, end
    const int slice = (int)(blockIdx.x % slices);
    __syncthreads();
    if (threadIdx.x < 32) {
      for (int k = 0; k < 2; ++k) {
        int64_t begin = c, end = stop;
        if (k == 0 && leads) {
          // back over the chunks that begin with the id, to the one it begins in
          if (tail != keys[1]) end = c + 1;
          for (int64_t q0 = c;; q0 -= 32) {
            const int64_t q = q0 - threadIdx.x;
            const uint32_t m = __ballot_sync(0xffffffffu, q >= 0 && skey[q * kChunk] == keys[1]);
            if (m == 0xffffffffu) continue;
            begin = q0 - (__ffs(~m) - 2);
            break;
          }
          if (begin > 0 && skey[begin * kChunk - 1] == keys[1]) --begin;
        }
        if (threadIdx.x == 0) {
          const bool part = k == 0 ? leads : trails;
          const bool all = part && atomicAdd(done + begin * slices + slice, 1u) ==
                                       (uint32_t)(end - begin - 1);
          ids[k][0] = (uint32_t)begin;
          ids[k][1] = all ? (uint32_t)end : 0u;
        }
      }
    }
    __syncthreads();
    for (int k = 0; k < 2; ++k) {
      const int64_t begin = ids[k][0], end = ids[k][1];
      if (end == 0 || col >= d) continue;
      __threadfence();
      part_load(last + begin * d + col, acc);
      for (int64_t q0 = begin + 1; q0 < end; q0 += kAhead) {
        float f[kAhead][8];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          if (q0 + u < end) part_load(first + (q0 + u) * d + col, f[u]);
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          if (q0 + u < end) {
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] += f[u][e];
          }
      }
      write_grad<GT>(grad + (int64_t)skey[(begin + 1) * kChunk] * d + col, acc, scale, add);
    }
  }
}

// An id that begins in chunk x and goes on past the next, to chunk y - 1: its
// parts in chunk order, cut into a run of chunks per warp (a frequent id has many), the runs
// joined in order.  The blocks share the sums' list of such ids.
constexpr int kJoinWarps = 8;
constexpr int kJoinBlocks = 148;

template <pkm_dtype GT>
__device__ __forceinline__ void join_one(const uint4& id, int d, float scale, int add,
                                         typename Elem<GT>::T* grad, const float* first,
                                         const float* last, float (*part)[32 * kUnit]) {
  const int64_t c = id.x, stop = id.y;
  const uint32_t key = id.z;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t run = (stop - c - 1 + kJoinWarps - 1) / kJoinWarps;
  const int64_t q1 = c + 1 + warp * run, q2 = min(stop, q1 + run);
  const int col = (blockIdx.y * 32 + lane) * kUnit;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  if (col < d) {
    if (warp == 0) load8<PKM_F32>(last + c * d + col, acc);
    for (int64_t q0 = q1; q0 < q2; q0 += 4) {
      float f[4][8];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (q0 + u < q2) load8<PKM_F32>(first + (q0 + u) * d + col, f[u]);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (q0 + u < q2) {
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] += f[u][e];
        }
    }
  }
#pragma unroll
  for (int e = 0; e < 8; e += 4)
    *reinterpret_cast<float4*>(&part[warp][lane * kUnit + e]) =
        make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
  __syncthreads();
  if (warp != 0 || col >= d) return;
  for (int w = 1; w < kJoinWarps; ++w)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += part[w][lane * kUnit + e];
  write_grad<GT>(grad + (int64_t)key * d + col, acc, scale, add);
}

template <pkm_dtype GT>
__global__ void __launch_bounds__(32 * kJoinWarps) embed_join_kernel(
    int d, float scale, int add, typename Elem<GT>::T* __restrict__ grad,
    const float* __restrict__ first, const float* __restrict__ last,
    const uint32_t* __restrict__ n_cross, const uint4* __restrict__ cross) {
  __shared__ __align__(16) float part[kJoinWarps][32 * kUnit];
  pdl_launch_dependents();
  pdl_wait();
  // the block's first entry (there are as many places as blocks) beside the count
  uint4 id = cross[blockIdx.x];
  const uint32_t n = *n_cross;
  for (uint32_t i = blockIdx.x; i < n; i += gridDim.x) {
    if (i != blockIdx.x) id = cross[i];
    join_one<GT>(id, d, scale, add, grad, first, last, part);
    __syncthreads();  // `part` may be written again
  }
}

int key_bits(int64_t n_rows) {  // bits that hold the keys 0 .. n_rows
  int b = 1;
  while ((n_rows >> b) != 0) ++b;
  return b;
}

size_t rup(size_t x) { return (x + 255) / 256 * 256; }
bool need16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool need4(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Blocks of the sums: chunks times column slices.
int sum_slices(int d) { return (d / kUnit + kSumUnits - 1) / kSumUnits; }
int64_t sum_blocks(int64_t T, int d) { return (T + kChunk - 1) / kChunk * sum_slices(d); }

struct EmbedLayout {
  size_t keys, pos, skey, spos, radix, bitmap, cross, done, first, last, total;
  bool cluster;  // the list fits the one-cluster sort
};

EmbedLayout embed_layout(const pkm_embed_args* a) {
  EmbedLayout L{};
  size_t off = 0;
  auto take = [&](size_t b) {
    const size_t o = off;
    off += rup(b);
    return o;
  };
  const size_t T = (size_t)a->T, d = (size_t)a->d;
  const size_t chunks = (T + kChunk - 1) / kChunk;
  L.cluster = a->T <= kSortMost;
  L.keys = take(T * 4);
  L.pos = take(T * 4);
  L.skey = take(T * 4);
  L.spos = take(T * 4);
  L.radix = L.cluster ? 0 : take(radix_sort_workspace(a->T));
  L.bitmap = L.cluster && a->T > kRankMost && !a->accumulate
                 ? take((size_t)(a->n_rows + 31) / 32 * 4)
                 : 0;
  L.cross = take((chunks + 1) * 16);  // count, then ids over three chunks or more
  L.done = a->T <= kJoinMost ? take(chunks * (size_t)sum_slices(a->d) * 4) : 0;
  L.first = take(chunks * d * 4);
  L.last = take(chunks * d * 4);
  L.total = off;
  return L;
}

pkm_status embed_validate(const pkm_embed_args* a, bool backward) {
  if (!a || a->T < 0 || a->n_rows < 1 || a->n_rows > 0x7fffffff || a->d < 8 || a->d % 8 ||
      (a->dtype != PKM_F32 && a->dtype != PKM_BF16) || !(a->scale == a->scale))
    return PKM_ERR_INVALID_ARG;
  if (backward && a->grad_dtype != PKM_F32 && a->grad_dtype != PKM_BF16)
    return PKM_ERR_INVALID_ARG;
  if (a->T > (int64_t(1) << 31) - 64 || a->d > 65536) return PKM_ERR_UNSUPPORTED;
  // the sums' grid and the blocks that zero rows share 31 bits
  if (backward && sum_blocks(a->T, a->d) + (a->n_rows + 31) / 32 > 0x7fffffff)
    return PKM_ERR_UNSUPPORTED;
  if (backward && !need16(a->grad)) return PKM_ERR_INVALID_ARG;
  if (a->T == 0) return PKM_OK;
  if (!need4(a->ids)) return PKM_ERR_INVALID_ARG;
  if (!backward) return need16(a->table) && need16(a->out) ? PKM_OK : PKM_ERR_INVALID_ARG;
  if (!need16(a->dout)) return PKM_ERR_INVALID_ARG;
  if (!need16(a->workspace) || a->workspace_bytes < embed_layout(a).total)
    return PKM_ERR_WORKSPACE;
  return PKM_OK;
}

// Rows zeroed beside the sort: about as many bytes as the memory takes in the
// time of the cluster's sort of up to 16384 tokens.  The gradient with 64, 96,
// 112, 128 and 224 MiB: 4096 tokens over 32768 x 1024 32.8, 31.9, 31.8, 32.9 (all
// 128) us, 16384 over 131072 x 1024 102.0, 100.1, 99.9, 99.9 and 101.7, 32768
// 128.4, 124.7, 122.8, 121.3 and 119.9, 131072 256, 255, 254.5, 254 and 249: a longer
// sort would take more.  By counting, with 4, 8, 16, 32 and 64 MiB: 509 over 32003
// x 520 17.0, 17.1, 17.6, 17.6 and 20.6, 512 over 32768 x 1024 25.9, 25.9, 24.7,
// 25.2 and 29.0.
constexpr int64_t kFillBeside = int64_t(112) << 20, kFillBesideRank = int64_t(16) << 20;

template <pkm_dtype DT, pkm_dtype GT>
cudaError_t embed_sums(const pkm_embed_args* a, const EmbedLayout& L, char* ws,
                       const EmbedFill& fill, cudaStream_t st) {
  const uint32_t* skey = reinterpret_cast<const uint32_t*>(ws + L.skey);
  const uint32_t* spos = reinterpret_cast<const uint32_t*>(ws + L.spos);
  float* first = reinterpret_cast<float*>(ws + L.first);
  float* last = reinterpret_cast<float*>(ws + L.last);
  auto* grad = static_cast<typename Elem<GT>::T*>(a->grad);
  const int64_t chunks = (a->T + kChunk - 1) / kChunk;
  const int units = a->d / kUnit;
  const int slices = sum_slices(a->d);
  const int64_t n_sum = sum_blocks(a->T, a->d);
  const int64_t n_fill = fill.on ? (fill.n_rows - fill.first + 31) / 32 : 0;
  uint32_t* n_cross = reinterpret_cast<uint32_t*>(ws + L.cross);
  uint4* cross = reinterpret_cast<uint4*>(ws + L.cross) + 1;
  uint32_t* done = reinterpret_cast<uint32_t*>(ws + L.done);
  const bool joins = a->T <= kJoinMost;
  note_launch();
  const cudaError_t e = launch_maybe_pdl(
      true, joins ? embed_sum_kernel<DT, GT, true> : embed_sum_kernel<DT, GT, false>,
      dim3((unsigned)(n_sum + n_fill)), dim3(kSumUnits), 0, st, skey, spos, a->T,
      (uint32_t)a->n_rows, static_cast<const typename Elem<DT>::T*>(a->dout), a->d, a->scale,
      a->accumulate, grad, first, last, slices, n_sum, n_cross, cross, done, fill);
  // an id that the join sums covers three chunks
  if (e != cudaSuccess || joins || chunks < 3) return e;
  const unsigned blocks = (unsigned)(chunks - 2 < kJoinBlocks ? chunks - 2 : kJoinBlocks);
  note_launch();
  return launch_maybe_pdl(true, embed_join_kernel<GT>, dim3(blocks, (units + 31) / 32),
                          dim3(32 * kJoinWarps), 0, st, a->d, a->scale, a->accumulate, grad, first,
                          last, n_cross, cross);
}

// The one-cluster sort; the rows below fill->first are zeroed beside it.
cudaError_t launch_embed_sort(const pkm_embed_args* a, const EmbedLayout& L, char* ws,
                              EmbedFill* fill, int32_t* status, cudaStream_t st) {
  EmbedSort p{};
  p.ids = a->ids;
  p.T = a->T;
  p.n_rows = a->n_rows;
  p.has_pad = a->has_pad;
  p.pad = a->pad_id;
  const int bits = key_bits(a->n_rows);
  p.passes = (bits + kMaxDigit - 1) / kMaxDigit;
  p.digit = (bits + p.passes - 1) / p.passes;
  const int ncta = kSortCluster;
  p.rounds = (int)((a->T + (int64_t)ncta * kSortThreads - 1) / ((int64_t)ncta * kSortThreads));
  p.key[0] = reinterpret_cast<uint32_t*>(ws + L.skey);
  p.pos[0] = reinterpret_cast<uint32_t*>(ws + L.spos);
  p.key[1] = reinterpret_cast<uint32_t*>(ws + L.keys);
  p.pos[1] = reinterpret_cast<uint32_t*>(ws + L.pos);
  p.n_cross = reinterpret_cast<uint32_t*>(ws + L.cross);
  p.done = reinterpret_cast<uint32_t*>(ws + L.done);
  p.n_done = a->T <= kJoinMost ? (int)((a->T + kChunk - 1) / kChunk) * sum_slices(a->d) : 0;
  const bool by_rank = a->T <= kRankMost;
  if (!a->accumulate) {
    if (!by_rank) {
      p.bitmap = reinterpret_cast<uint32_t*>(ws + L.bitmap);
      p.words = (a->n_rows + 31) / 32;
    }
    const int64_t row = (int64_t)a->d * (a->grad_dtype == PKM_F32 ? 4 : 2);
    int64_t rows = (by_rank ? kFillBesideRank : kFillBeside) / row / 32 * 32;
    if (rows > a->n_rows) rows = a->n_rows / 32 * 32;
    p.fill = static_cast<uint4*>(a->grad);
    p.fill_units = rows * row / 16;
    *fill = EmbedFill{true, p.bitmap, a->n_rows, rows};
  }
  if (by_rank) {
    const int blocks = (int)((a->T + 31) / 32);
    const int64_t want = (p.fill_units + 8 * 256 - 1) / (8 * 256);
    note_launch();
    return launch_maybe_pdl(true, embed_rank_kernel,
                            dim3((unsigned)(blocks + (want < 148 * 6 ? want : 148 * 6))),
                            dim3(32 * kRankWarps), 0, st, p, blocks, status);
  }
  // rounds of the short sort: a power of two, the tokens of a CTA
  int short_rounds = 1;
  while (short_rounds < p.rounds) short_rounds *= 2;
  auto kern = short_rounds == 1   ? embed_sort_kernel<1>
              : short_rounds == 2 ? embed_sort_kernel<2>
              : short_rounds == 4 ? embed_sort_kernel<4>
                                  : embed_sort_long_kernel;
  const bool is_short = short_rounds <= 4;
  const size_t smem = sort_smem(p.digit, is_short ? short_rounds : p.rounds, is_short);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sort_smem(kMaxDigit, is_short ? 4 : kSortRounds,
                                                      is_short));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ncta, 1, 1);
  cfg.blockDim = dim3(kSortThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ncta;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kern, p, status);
  if (e != cudaSuccess) return e;
  note_launch();
  if (p.fill_units == 0) return cudaSuccess;
  note_launch();
  const int64_t zero = (p.fill_units + kZeroUnits - 1) / kZeroUnits;
  return launch_maybe_pdl(true, embed_zero_kernel,
                          dim3((unsigned)(zero < kZeroBlocks ? zero : kZeroBlocks)),
                          dim3(kThreads), 0, st, p.fill, p.fill_units);
}

cudaError_t embed_backward(const pkm_embed_args* a, int32_t* status, cudaStream_t st) {
  const bool b = a->dtype == PKM_BF16, gb = a->grad_dtype == PKM_BF16;
  const EmbedLayout L = embed_layout(a);
  char* ws = static_cast<char*>(a->workspace);
  EmbedFill fill{};
  cudaError_t e = cudaSuccess;
  if (a->T == 0 || !L.cluster) {
    if (!a->accumulate)
      e = cudaMemsetAsync(a->grad, 0,
                          (size_t)a->n_rows * a->d * (a->grad_dtype == PKM_F32 ? 4 : 2), st);
    if (e != cudaSuccess || a->T == 0) return e;
    uint32_t* keys = reinterpret_cast<uint32_t*>(ws + L.keys);
    uint32_t* pos = reinterpret_cast<uint32_t*>(ws + L.pos);
    const int64_t blocks = (a->T + 255) / 256;
    embed_keys_kernel<<<(unsigned)(blocks < 1184 ? blocks : 1184), 256, 0, st>>>(
        a->ids, a->T, a->n_rows, a->has_pad, a->pad_id, keys, pos,
        reinterpret_cast<uint32_t*>(ws + L.cross), status);
    note_launch();
    e = launch_radix_sort(keys, pos, a->T, key_bits(a->n_rows),
                          reinterpret_cast<uint32_t*>(ws + L.skey),
                          reinterpret_cast<uint32_t*>(ws + L.spos), ws + L.radix, st);
  } else {
    e = launch_embed_sort(a, L, ws, &fill, status, st);
  }
  if (e != cudaSuccess) return e;
  return b ? (gb ? embed_sums<PKM_BF16, PKM_BF16>(a, L, ws, fill, st)
                 : embed_sums<PKM_BF16, PKM_F32>(a, L, ws, fill, st))
           : (gb ? embed_sums<PKM_F32, PKM_BF16>(a, L, ws, fill, st)
                 : embed_sums<PKM_F32, PKM_F32>(a, L, ws, fill, st));
}

template <pkm_dtype DT>
cudaError_t embed_forward(const pkm_embed_args* a, int32_t* status, cudaStream_t st) {
  using E = typename Elem<DT>::T;
  const int lpr = lanes_per_row(a->d);
  const int rows = kThreads / lpr;
  note_launch();
  return launch_maybe_pdl(true, embed_fwd_kernel<DT>, dim3((unsigned)((a->T + rows - 1) / rows)),
                          dim3(kThreads), 0, st, static_cast<const E*>(a->table), a->n_rows, a->d,
                          lpr, a->ids, a->T, a->scale, a->has_pad, a->pad_id,
                          static_cast<E*>(a->out), status);
}

}  // namespace
}  // namespace pkm

using namespace pkm;

extern "C" {

PKM_API size_t pkm_embed_workspace_size(const pkm_embed_args* a) {
  return a && a->T > 0 && a->d > 0 && a->n_rows > 0 ? embed_layout(a).total : 0;
}

PKM_API pkm_status pkm_embed_forward(const pkm_embed_args* a, pkm_stream_t stream) {
  const pkm_status s = embed_validate(a, false);
  if (s != PKM_OK || a->T == 0) return s;
  int32_t* status = status_ptr();
  if (!status) return PKM_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = a->dtype == PKM_BF16 ? embed_forward<PKM_BF16>(a, status, st)
                                             : embed_forward<PKM_F32>(a, status, st);
  return e == cudaSuccess ? PKM_OK : PKM_ERR_CUDA;
}

PKM_API pkm_status pkm_embed_backward(const pkm_embed_args* a, pkm_stream_t stream) {
  const pkm_status s = embed_validate(a, true);
  if (s != PKM_OK) return s;
  int32_t* status = status_ptr();
  if (!status) return PKM_ERR_CUDA;
  return embed_backward(a, status, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PKM_OK
             : PKM_ERR_CUDA;
}

}  // extern "C"
