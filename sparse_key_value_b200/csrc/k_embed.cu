// k_embed.cu -- the token embedding with a scale, and its gradient by sorted
// tokens.
//
// Forward: out[t] = scale * table[ids[t]], one rounding.  Bound by memory:
// the distinct rows and the output.
//
// Backward: grad[r] = scale * sum of dout[t] over the tokens t with ids[t] = r,
// every row of the table's gradient written.  Three launches:
//   1. embed_sort_kernel: one cluster sorts the tokens by id (stable radix
//      sort, histograms exchanged through distributed shared memory) and marks
//      the rows that occur in a bitmap, while the other clusters already zero
//      the first rows of the gradient.
//   2. embed_sum_kernel: the sorted list is cut into chunks of kChunk entries,
//      one block sums a chunk's parts in order; the blocks after those zero the
//      rows that no token reads, so each row is written once.
//   3. embed_join_kernel: the parts of an id that crosses chunks, joined in
//      chunk order.
// No atomics on values: the same bits every run, and a frequent id spreads
// over many blocks.  Bound by the gradient's write (n_rows * d), then by the
// launches' latency.  Lists of more than kSortMost tokens go through the
// library's multi-block radix sort.
#include "kernels.h"
#include "q8.cuh"
#include "tc_pair.cuh"

namespace pkm {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 16;   // sorted tokens per block
constexpr int kAhead = 8;    // rows of dout in flight per thread
constexpr int kSortThreads = 1024;
constexpr int kSortCluster = 8;
constexpr int kSortRounds = 16;  // tokens per thread of the sorting cluster, at most
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
    float f[4][8];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = c0 + u * lpr * kUnit;
#pragma unroll
      for (int e = 0; e < 8; ++e) f[u][e] = 0.f;
      if (ok && c < d) load8<DT>(row + c, f[u]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = c0 + u * lpr * kUnit;
      if (c >= d) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) f[u][e] = ok ? f[u][e] * scale : 0.f;
      store8<DT>(dst + c, f[u]);
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
                                  uint32_t* __restrict__ pos, int32_t* status) {
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
  uint4* fill;                // zeroed by the clusters after the first, or null
  int64_t fill_units;
};

// Dynamic shared memory: per-warp digit counts, then the CTA's digit totals,
// then each token's rank within its warp and digit.
size_t sort_smem(int digit, int rounds) {
  return ((size_t)32 << digit) * 2 + ((size_t)4 << digit) + (size_t)rounds * kSortThreads * 2;
}

__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const EmbedSort p,
                                                                  int32_t* status) {
  const uint32_t ncta = cluster_size(), rank = cluster_rank();
  const int tid = threadIdx.x;
  if (blockIdx.x >= ncta) {  // a filling cluster
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int64_t i = (int64_t)(blockIdx.x - ncta) * kSortThreads + tid; i < p.fill_units;
         i += (int64_t)(gridDim.x - ncta) * kSortThreads)
      p.fill[i] = zero;
    return;
  }
  extern __shared__ __align__(16) unsigned char smem[];
  const int bins = 1 << p.digit;
  uint16_t* cnt = reinterpret_cast<uint16_t*>(smem);                       // [32][bins]
  uint32_t* total = reinterpret_cast<uint32_t*>(smem + (size_t)64 * bins);  // [bins]
  uint16_t* ranks = reinterpret_cast<uint16_t*>(smem + (size_t)68 * bins);
  __shared__ uint32_t scan[32];
  const int warp = tid >> 5, lane = tid & 31;
  const uint32_t lt = (1u << lane) - 1u;
  uint16_t* mine = cnt + (size_t)warp * bins;
  // a warp owns rounds * 32 consecutive tokens, so (CTA, warp, round, lane)
  // is the list's order
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
    for (int b = tid; b < 16 * bins; b += kSortThreads)
      reinterpret_cast<uint32_t*>(cnt)[b] = 0;
    __syncthreads();
    for (int r = 0; r < p.rounds; ++r) {
      const int64_t i = i0 + r * 32;
      uint32_t d = bins;  // lanes past the end form their own group
      if (i < p.T) {
        const uint32_t k = pass == 0
                               ? embed_key(p.ids[i], p.n_rows, p.has_pad, p.pad, status)
                               : __ldcg(skey + i);
        d = (k >> shift) & (bins - 1);
      }
      const uint32_t peers = __match_any_sync(0xffffffffu, d);
      const uint32_t before = i < p.T ? mine[d] : 0u;
      __syncwarp();
      if (i < p.T && (peers & lt) == 0) mine[d] = (uint16_t)(before + __popc(peers));
      __syncwarp();
      ranks[r * kSortThreads + tid] = (uint16_t)(before + __popc(peers & lt));
    }
    __syncthreads();
    if (tid < bins) {  // counts -> prefixes over the warps; the CTA's totals
      uint32_t run = 0;
#pragma unroll 8
      for (int w = 0; w < 32; ++w) {
        const uint32_t c = cnt[(size_t)w * bins + tid];
        cnt[(size_t)w * bins + tid] = (uint16_t)run;
        run += c;
      }
      total[tid] = run;
    }
    __syncwarp();
    cluster_sync_all();
    // first place of this CTA's tokens with digit `tid`: the smaller digits
    // of every CTA, then the same digit of the CTAs before this one
    uint32_t before = 0, all = 0;
    if (tid < bins)
      for (uint32_t c = 0; c < ncta; ++c) {
        const uint32_t t = ld_cluster(map_to(&total[tid], c));
        before += c < rank ? t : 0u;
        all += t;
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
    for (int r = 0; r < p.rounds; ++r) {
      const int64_t i = i0 + r * 32;
      if (i >= p.T) break;
      const uint32_t k = pass == 0 ? embed_key(p.ids[i], p.n_rows, p.has_pad, p.pad, nullptr)
                                   : __ldcg(skey + i);
      const uint32_t d = (k >> shift) & (bins - 1);
      const uint32_t dst = total[d] + mine[d] + ranks[r * kSortThreads + tid];
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

struct EmbedFill {
  const uint32_t* bitmap;  // null: nothing to fill
  int64_t n_rows, first;   // rows first .. n_rows - 1; `first` is a multiple of 32
};

// Zeroes the rows of one bitmap word that no token reads.
template <pkm_dtype GT>
__device__ __forceinline__ void fill_rows(const EmbedFill& f, int64_t block, int d,
                                          typename Elem<GT>::T* grad) {
  const int64_t r0 = f.first + block * 32;
  const uint32_t used = f.bitmap[r0 >> 5];
  const uint32_t units = (uint32_t)(d / Elem<GT>::kVec);  // 16 bytes each
  const uint32_t rows = (uint32_t)min((int64_t)32, f.n_rows - r0);
  uint4* g = reinterpret_cast<uint4*>(grad + r0 * d);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (uint32_t i = threadIdx.x; i < rows * units; i += kSumUnits)
    if (!(used >> (i / units) & 1)) __stcs(g + i, zero);
}

// The first n_sum blocks: one per chunk and slice of 8 * kSumUnits columns, a
// thread owns 8 columns and walks the chunk's entries in order, kAhead rows in
// flight.  The blocks after them zero the rows without tokens.
template <pkm_dtype DT, pkm_dtype GT>
__global__ void __launch_bounds__(kSumUnits) embed_sum_kernel(
    const uint32_t* __restrict__ skey, const uint32_t* __restrict__ spos, int64_t T,
    uint32_t mark, const typename Elem<DT>::T* __restrict__ dout, int d, float scale, int add,
    typename Elem<GT>::T* __restrict__ grad, float* __restrict__ first,
    float* __restrict__ last, int slices, int64_t n_sum, const EmbedFill fill) {
  if ((int64_t)blockIdx.x >= n_sum) {
    fill_rows<GT>(fill, blockIdx.x - n_sum, d, grad);
    return;
  }
  __shared__ uint32_t keys[kChunk + 2];  // [0]: the key before the chunk, [len + 1]: after it
  __shared__ uint32_t rows[kChunk];
  const int64_t c = blockIdx.x / slices, i0 = c * kChunk;
  const int len = (int)min((int64_t)kChunk, T - i0);
  for (int j = threadIdx.x; j < len + 2; j += blockDim.x) {
    const int64_t i = i0 + j - 1;
    keys[j] = i >= 0 && i < T ? skey[i] : mark;
    if (j >= 1 && j <= len) rows[j - 1] = spos[i];
  }
  __syncthreads();
  const int col = ((int)(blockIdx.x % slices) * kSumUnits + threadIdx.x) * kUnit;
  if (col >= d) return;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  bool starts = keys[1] == mark || keys[0] != keys[1];  // the current part begins its id
  for (int j0 = 0; j0 < len && keys[j0 + 1] != mark; j0 += kAhead) {
    float f[kAhead][8];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (j0 + u < len && keys[j0 + u + 1] != mark)
        load8<DT>(dout + (int64_t)rows[j0 + u] * d + col, f[u]);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = j0 + u;
      if (j >= len || keys[j + 1] == mark) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += f[u][e];
      const uint32_t key = keys[j + 1];
      const bool goes_on = keys[j + 2] == key;
      if (goes_on && j + 1 < len) continue;
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
}

// The id that begins in chunk c and goes on: its parts in chunk order.
template <pkm_dtype GT>
__global__ void __launch_bounds__(32) embed_join_kernel(
    const uint32_t* __restrict__ skey, int64_t T, uint32_t mark, int d, float scale, int add,
    typename Elem<GT>::T* __restrict__ grad, const float* __restrict__ first,
    const float* __restrict__ last) {
  const int64_t c = blockIdx.x, end = (c + 1) * kChunk;
  if (end >= T) return;
  const uint32_t key = skey[end - 1];
  if (key == mark || skey[end] != key) return;
  if (c > 0 && skey[c * kChunk - 1] == key) return;  // begins in an earlier chunk
  // chunks c + 1 .. stop - 1 hold the rest: 32 chunks looked at at a time
  const int64_t chunks = (T + kChunk - 1) / kChunk;
  int64_t stop = c + 1;
  for (;; stop += 32) {
    const int64_t q = stop + threadIdx.x;  // chunk q begins with the id
    const uint32_t m = __ballot_sync(0xffffffffu, q < chunks && skey[q * kChunk] == key);
    if (m != 0xffffffffu) {
      stop += __ffs(~m) - 1;
      break;
    }
  }
  const int col = (blockIdx.y * 32 + threadIdx.x) * kUnit;
  if (col >= d) return;
  float acc[8];
  load8<PKM_F32>(last + c * d + col, acc);
  for (int64_t q0 = c + 1; q0 < stop; q0 += 4) {
    float f[4][8];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (q0 + u < stop) load8<PKM_F32>(first + (q0 + u) * d + col, f[u]);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (q0 + u < stop) {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += f[u][e];
      }
  }
  write_grad<GT>(grad + (int64_t)key * d + col, acc, scale, add);
}

int key_bits(int64_t n_rows) {  // bits that hold the keys 0 .. n_rows
  int b = 1;
  while ((n_rows >> b) != 0) ++b;
  return b;
}

size_t rup(size_t x) { return (x + 255) / 256 * 256; }
bool need16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct EmbedLayout {
  size_t keys, pos, skey, spos, radix, bitmap, first, last, total;
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
  L.bitmap = L.cluster && !a->accumulate ? take((size_t)(a->n_rows + 31) / 32 * 4) : 0;
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
  if (backward && !need16(a->grad)) return PKM_ERR_INVALID_ARG;
  if (a->T == 0) return PKM_OK;
  if (!need16(a->ids)) return PKM_ERR_INVALID_ARG;
  if (!backward) return need16(a->table) && need16(a->out) ? PKM_OK : PKM_ERR_INVALID_ARG;
  if (!need16(a->dout)) return PKM_ERR_INVALID_ARG;
  if (!need16(a->workspace) || a->workspace_bytes < embed_layout(a).total)
    return PKM_ERR_WORKSPACE;
  return PKM_OK;
}

// Rows that the sort's launch zeroes beside the sort: about as many bytes as
// the memory takes in the sort's time.
constexpr int64_t kFillBeside = int64_t(32) << 20;

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
  const int slices = (units + kSumUnits - 1) / kSumUnits;
  const int64_t n_sum = chunks * slices;
  const int64_t n_fill = fill.bitmap ? (fill.n_rows - fill.first + 31) / 32 : 0;
  if (n_sum + n_fill > 0x7fffffff) return cudaErrorInvalidValue;
  embed_sum_kernel<DT, GT><<<(unsigned)(n_sum + n_fill), kSumUnits, 0, st>>>(
      skey, spos, a->T, (uint32_t)a->n_rows, static_cast<const typename Elem<DT>::T*>(a->dout),
      a->d, a->scale, a->accumulate, grad, first, last, slices, n_sum, fill);
  note_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || chunks < 2) return e;
  embed_join_kernel<GT><<<dim3((unsigned)(chunks - 1), (units + 31) / 32), 32, 0, st>>>(
      skey, a->T, (uint32_t)a->n_rows, a->d, a->scale, a->accumulate, grad, first, last);
  note_launch();
  return cudaGetLastError();
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
  // one CTA for lists that it holds in two rounds: no cluster barriers to wait for
  const int ncta = a->T <= 2 * kSortThreads ? 1 : kSortCluster;
  p.rounds = (int)((a->T + (int64_t)ncta * kSortThreads - 1) / ((int64_t)ncta * kSortThreads));
  p.key[0] = reinterpret_cast<uint32_t*>(ws + L.skey);
  p.pos[0] = reinterpret_cast<uint32_t*>(ws + L.spos);
  p.key[1] = reinterpret_cast<uint32_t*>(ws + L.keys);
  p.pos[1] = reinterpret_cast<uint32_t*>(ws + L.pos);
  int clusters = 1;
  if (!a->accumulate) {
    p.bitmap = reinterpret_cast<uint32_t*>(ws + L.bitmap);
    p.words = (a->n_rows + 31) / 32;
    const int64_t row = (int64_t)a->d * (a->grad_dtype == PKM_F32 ? 4 : 2);
    int64_t rows = kFillBeside / row / 32 * 32;
    if (rows > a->n_rows) rows = a->n_rows / 32 * 32;
    p.fill = static_cast<uint4*>(a->grad);
    p.fill_units = rows * row / 16;
    *fill = EmbedFill{p.bitmap, a->n_rows, rows};
    const int64_t blocks = (p.fill_units + 4 * kSortThreads - 1) / (4 * kSortThreads);
    const int64_t want = (blocks + ncta - 1) / ncta, most = 136 / ncta;
    clusters += (int)(want < most ? want : most);
  }
  const size_t smem = sort_smem(p.digit, p.rounds);
  cudaError_t e = cudaFuncSetAttribute(embed_sort_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sort_smem(kMaxDigit, kSortRounds));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * ncta), 1, 1);
  cfg.blockDim = dim3(kSortThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ncta;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, embed_sort_kernel, p, status);
  if (e == cudaSuccess) note_launch();
  return e;
}

cudaError_t embed_backward(const pkm_embed_args* a, int32_t* status, cudaStream_t st) {
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
        a->ids, a->T, a->n_rows, a->has_pad, a->pad_id, keys, pos, status);
    note_launch();
    e = launch_radix_sort(keys, pos, a->T, key_bits(a->n_rows),
                          reinterpret_cast<uint32_t*>(ws + L.skey),
                          reinterpret_cast<uint32_t*>(ws + L.spos), ws + L.radix, st);
  } else {
    e = launch_embed_sort(a, L, ws, &fill, status, st);
  }
  if (e != cudaSuccess) return e;
  const bool b = a->dtype == PKM_BF16, gb = a->grad_dtype == PKM_BF16;
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
  embed_fwd_kernel<DT><<<(unsigned)((a->T + rows - 1) / rows), kThreads, 0, st>>>(
      static_cast<const E*>(a->table), a->n_rows, a->d, lpr, a->ids, a->T, a->scale, a->has_pad,
      a->pad_id, static_cast<E*>(a->out), status);
  note_launch();
  return cudaGetLastError();
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
