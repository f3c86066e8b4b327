// k_embed.cu -- the token embedding with a scale, and its gradient by sorted
// tokens.
//
// Forward: out[t] = scale * table[ids[t]], one rounding.  Bound by memory:
// the distinct rows and the output.
//
// Backward: grad[r] = scale * sum of dout[t] over the tokens t with ids[t] = r,
// every row of the table's gradient written.  The tokens are sorted by id
// (stable), the sorted list is cut into chunks of kChunk entries, one block
// sums a chunk's parts in order, and the parts of an id that crosses chunks
// are joined in chunk order by a second kernel: no atomics, the same bits
// every run, and a frequent id spreads over many blocks.
#include "kernels.h"
#include "q8.cuh"

namespace pkm {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 32;   // sorted tokens per block
constexpr int kAhead = 8;    // rows of dout in flight per thread
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

// Sort keys: the id, or n_rows (sorts last, never summed) for the padding id
// and ids outside the table.
__global__ void embed_keys_kernel(const int32_t* __restrict__ ids, int64_t T, int64_t n_rows,
                                  int has_pad, int32_t pad, uint32_t* __restrict__ keys,
                                  uint32_t* __restrict__ pos, int32_t* status) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < T;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int32_t id = ids[i];
    const bool padded = has_pad && id == pad;
    const bool ok = !padded && id >= 0 && id < n_rows;
    if (!ok && !padded) set_status(status, PKM_ERR_DEVICE);
    keys[i] = ok ? (uint32_t)id : (uint32_t)n_rows;
    pos[i] = (uint32_t)i;
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

// One block per chunk and slice of 8 * kSumUnits columns; a thread owns 8
// columns and walks the chunk's entries in order, kAhead rows in flight.
template <pkm_dtype DT, pkm_dtype GT>
__global__ void __launch_bounds__(kSumUnits) embed_sum_kernel(
    const uint32_t* __restrict__ skey, const uint32_t* __restrict__ spos, int64_t T,
    uint32_t mark, const typename Elem<DT>::T* __restrict__ dout, int d, float scale, int add,
    typename Elem<GT>::T* __restrict__ grad, float* __restrict__ first,
    float* __restrict__ last) {
  __shared__ uint32_t keys[kChunk + 2];  // [0]: the key before the chunk, [len + 1]: after it
  __shared__ uint32_t rows[kChunk];
  const int64_t c = blockIdx.x, i0 = c * kChunk;
  const int len = (int)min((int64_t)kChunk, T - i0);
  for (int j = threadIdx.x; j < len + 2; j += blockDim.x) {
    const int64_t i = i0 + j - 1;
    keys[j] = i >= 0 && i < T ? skey[i] : mark;
    if (j >= 1 && j <= len) rows[j - 1] = spos[i];
  }
  __syncthreads();
  const int col = (blockIdx.y * kSumUnits + threadIdx.x) * kUnit;
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
  int64_t lo = end, hi = T;  // first entry past the id, by bisection
  while (lo < hi) {
    const int64_t m = (lo + hi) / 2;
    if (skey[m] == key)
      lo = m + 1;
    else
      hi = m;
  }
  const int64_t stop = (lo + kChunk - 1) / kChunk;  // chunks c + 1 .. stop - 1 hold the rest
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
  size_t keys, pos, skey, spos, radix, first, last, total;
};

EmbedLayout embed_layout(int64_t T, int d) {
  EmbedLayout L{};
  size_t off = 0;
  auto take = [&](size_t b) {
    const size_t o = off;
    off += rup(b);
    return o;
  };
  const size_t chunks = (size_t)((T + kChunk - 1) / kChunk);
  L.keys = take((size_t)T * 4);
  L.pos = take((size_t)T * 4);
  L.skey = take((size_t)T * 4);
  L.spos = take((size_t)T * 4);
  L.radix = take(radix_sort_workspace(T));
  L.first = take(chunks * (size_t)d * 4);
  L.last = take(chunks * (size_t)d * 4);
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
  if (!need16(a->workspace) || a->workspace_bytes < embed_layout(a->T, a->d).total)
    return PKM_ERR_WORKSPACE;
  return PKM_OK;
}

template <pkm_dtype DT, pkm_dtype GT>
cudaError_t embed_sums(const pkm_embed_args* a, const EmbedLayout& L, char* ws,
                       cudaStream_t st) {
  const uint32_t* skey = reinterpret_cast<const uint32_t*>(ws + L.skey);
  const uint32_t* spos = reinterpret_cast<const uint32_t*>(ws + L.spos);
  float* first = reinterpret_cast<float*>(ws + L.first);
  float* last = reinterpret_cast<float*>(ws + L.last);
  auto* grad = static_cast<typename Elem<GT>::T*>(a->grad);
  const unsigned chunks = (unsigned)((a->T + kChunk - 1) / kChunk);
  const int units = a->d / kUnit;
  embed_sum_kernel<DT, GT>
      <<<dim3(chunks, (units + kSumUnits - 1) / kSumUnits), kSumUnits, 0, st>>>(
          skey, spos, a->T, (uint32_t)a->n_rows,
          static_cast<const typename Elem<DT>::T*>(a->dout), a->d, a->scale, a->accumulate, grad,
          first, last);
  note_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || chunks < 2) return e;
  embed_join_kernel<GT><<<dim3(chunks - 1, (units + 31) / 32), 32, 0, st>>>(
      skey, a->T, (uint32_t)a->n_rows, a->d, a->scale, a->accumulate, grad, first, last);
  note_launch();
  return cudaGetLastError();
}

cudaError_t embed_backward(const pkm_embed_args* a, int32_t* status, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (!a->accumulate)
    e = cudaMemsetAsync(a->grad, 0,
                        (size_t)a->n_rows * a->d * (a->grad_dtype == PKM_F32 ? 4 : 2), st);
  if (e != cudaSuccess || a->T == 0) return e;
  const EmbedLayout L = embed_layout(a->T, a->d);
  char* ws = static_cast<char*>(a->workspace);
  uint32_t* keys = reinterpret_cast<uint32_t*>(ws + L.keys);
  uint32_t* pos = reinterpret_cast<uint32_t*>(ws + L.pos);
  const int64_t blocks = (a->T + 255) / 256;
  embed_keys_kernel<<<(unsigned)(blocks < 1184 ? blocks : 1184), 256, 0, st>>>(
      a->ids, a->T, a->n_rows, a->has_pad, a->pad_id, keys, pos, status);
  note_launch();
  e = launch_radix_sort(keys, pos, a->T, key_bits(a->n_rows),
                        reinterpret_cast<uint32_t*>(ws + L.skey),
                        reinterpret_cast<uint32_t*>(ws + L.spos), ws + L.radix, st);
  if (e != cudaSuccess) return e;
  const bool b = a->dtype == PKM_BF16, gb = a->grad_dtype == PKM_BF16;
  return b ? (gb ? embed_sums<PKM_BF16, PKM_BF16>(a, L, ws, st)
                 : embed_sums<PKM_BF16, PKM_F32>(a, L, ws, st))
           : (gb ? embed_sums<PKM_F32, PKM_BF16>(a, L, ws, st)
                 : embed_sums<PKM_F32, PKM_F32>(a, L, ws, st));
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
  return a && a->T > 0 && a->d > 0 ? embed_layout(a->T, a->d).total : 0;
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
