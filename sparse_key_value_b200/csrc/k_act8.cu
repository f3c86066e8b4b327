// k_act8.cu -- activations stored in 8 bits and read back (formats and scale
// rule in q8.cuh).
//
// A half-warp holds a group of 128 columns, one 8-column unit per lane, so
// the group's maximum is four shuffles and every row access is a contiguous
// 16-byte (8-byte for the 8-bit side) load or store per lane.  Bound by
// memory: b bytes read and one written per element, four bytes per group for
// the scale.  Measured on one B200 at 8192 x 2048 bf16, stored and read back:
// 17.3 us for 101 MB, 5.8 TB/s with the launches (the 17 MB of 8-bit values
// are read from L2); 2, 4 or 8 groups in flight, blocks of 128 to 512 threads and
// streaming accesses made no difference.
#include "kernels.h"
#include "q8.cuh"

namespace pkm {

namespace {
constexpr int kThreads = 256;
constexpr int kHalves = kThreads / kGroupLanes;  // groups a block handles at a time
constexpr int kAtOnce = 4;                       // groups in flight per half-warp

// Element offset of this lane's unit of group gi, or -1 past the row's end.
__device__ __forceinline__ int64_t unit_at(int64_t gi, int64_t n_groups, int groups, int d) {
  const int in = (threadIdx.x % kGroupLanes) * kUnit;
  if (gi >= n_groups) return -1;
  if (d % kQ8Group == 0) return gi * kQ8Group + in;  // no division
  const int64_t row = gi / groups;
  const int col = (int)(gi - row * groups) * kQ8Group + in;
  return col < d ? row * d + col : -1;
}

template <pkm_dtype DT>
__global__ void __launch_bounds__(kThreads) act8_store_kernel(
    const typename Elem<DT>::T* __restrict__ x, int64_t n_groups, int groups, int d, pkm_q8 fmt,
    uint8_t* __restrict__ q, float* __restrict__ scales) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t g0 = (int64_t)blockIdx.x * (kHalves * kAtOnce) + threadIdx.x / kGroupLanes;
  int64_t at[kAtOnce];
  Raw8<DT> raw[kAtOnce];
#pragma unroll
  for (int u = 0; u < kAtOnce; ++u) {
    at[u] = unit_at(g0 + u * kHalves, n_groups, groups, d);
    raw[u].zero();
    if (at[u] >= 0) raw[u].load(x + at[u]);
  }
#pragma unroll
  for (int u = 0; u < kAtOnce; ++u) {
    float v[8];
    raw[u].unpack(v);
    const float s = q8_scale(group_amax_bits(v), fmt);
    if (at[u] >= 0) *reinterpret_cast<uint2*>(q + at[u]) = q8_encode(v, q8_inverse(s), fmt);
    const int64_t gi = g0 + u * kHalves;
    if (gi < n_groups && threadIdx.x % kGroupLanes == 0) scales[gi] = s;
  }
}

template <pkm_dtype DT>
__global__ void __launch_bounds__(kThreads) act8_load_kernel(
    const uint8_t* __restrict__ q, const float* __restrict__ scales, int64_t n_groups, int groups,
    int d, pkm_q8 fmt, typename Elem<DT>::T* __restrict__ out) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t g0 = (int64_t)blockIdx.x * (kHalves * kAtOnce) + threadIdx.x / kGroupLanes;
  int64_t at[kAtOnce];
  uint2 raw[kAtOnce];
  float s[kAtOnce];
#pragma unroll
  for (int u = 0; u < kAtOnce; ++u) {
    at[u] = unit_at(g0 + u * kHalves, n_groups, groups, d);
    if (at[u] >= 0) {
      raw[u] = *reinterpret_cast<const uint2*>(q + at[u]);
      s[u] = scales[g0 + u * kHalves];
    }
  }
#pragma unroll
  for (int u = 0; u < kAtOnce; ++u)
    if (at[u] >= 0) {
      float v[8];
      q8_decode(raw[u], s[u], fmt, v);
      store8<DT>(out + at[u], v);
    }
}

unsigned group_grid(int64_t n_groups) {
  return (unsigned)((n_groups + kHalves * kAtOnce - 1) / (kHalves * kAtOnce));
}
}  // namespace

cudaError_t launch_act8_store(const void* x, int64_t T, int d, pkm_dtype dt, pkm_q8 fmt, void* q,
                              float* scales, cudaStream_t stream) {
  const int g = q8_groups(d);
  const int64_t n = T * g;
  if (n <= 0) return cudaSuccess;
  const dim3 grid(group_grid(n)), block(kThreads);
  note_launch();
  return dt == PKM_BF16
             ? launch_maybe_pdl(true, act8_store_kernel<PKM_BF16>, grid, block, 0, stream,
                                static_cast<const __nv_bfloat16*>(x), n, g, d, fmt,
                                static_cast<uint8_t*>(q), scales)
             : launch_maybe_pdl(true, act8_store_kernel<PKM_F32>, grid, block, 0, stream,
                                static_cast<const float*>(x), n, g, d, fmt,
                                static_cast<uint8_t*>(q), scales);
}

cudaError_t launch_act8_load(const void* q, const float* scales, int64_t T, int d, pkm_q8 fmt,
                             void* out, pkm_dtype dt, cudaStream_t stream) {
  const int g = q8_groups(d);
  const int64_t n = T * g;
  if (n <= 0) return cudaSuccess;
  const dim3 grid(group_grid(n)), block(kThreads);
  note_launch();
  return dt == PKM_BF16
             ? launch_maybe_pdl(true, act8_load_kernel<PKM_BF16>, grid, block, 0, stream,
                                static_cast<const uint8_t*>(q), scales, n, g, d, fmt,
                                static_cast<__nv_bfloat16*>(out))
             : launch_maybe_pdl(true, act8_load_kernel<PKM_F32>, grid, block, 0, stream,
                                static_cast<const uint8_t*>(q), scales, n, g, d, fmt,
                                static_cast<float*>(out));
}

}  // namespace pkm

using namespace pkm;

namespace {
bool aligned(const void* p, uintptr_t a) {
  return p && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}
pkm_status act8_validate(const void* x, int64_t T, int32_t d, pkm_dtype dtype, pkm_q8 fmt,
                         const void* q, const float* scales) {
  if (T < 0 || d < 8 || d % 8 || (dtype != PKM_F32 && dtype != PKM_BF16) ||
      (fmt != PKM_Q8_E4M3 && fmt != PKM_Q8_INT8))
    return PKM_ERR_INVALID_ARG;
  // the grid holds 64 groups per block
  if (T > kMaxTokens || T > ((int64_t(1) << 31) - 1) * 64 / q8_groups(d))
    return PKM_ERR_UNSUPPORTED;
  if (T > 0 && (!aligned(x, 16) || !aligned(q, 16) || !aligned(scales, 16)))
    return PKM_ERR_INVALID_ARG;
  return PKM_OK;
}
}  // namespace

extern "C" {

PKM_API pkm_status pkm_act8_store(const void* x, int64_t T, int32_t d, pkm_dtype dtype, pkm_q8 fmt,
                                  void* q, float* scales, pkm_stream_t stream) {
  const pkm_status s = act8_validate(x, T, d, dtype, fmt, q, scales);
  if (s != PKM_OK || T == 0) return s;
  return launch_act8_store(x, T, d, dtype, fmt, q, scales,
                           reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PKM_OK
             : PKM_ERR_CUDA;
}

PKM_API pkm_status pkm_act8_load(const void* q, const float* scales, int64_t T, int32_t d,
                                 pkm_q8 fmt, void* out, pkm_dtype dtype, pkm_stream_t stream) {
  const pkm_status s = act8_validate(out, T, d, dtype, fmt, q, scales);
  if (s != PKM_OK || T == 0) return s;
  return launch_act8_load(q, scales, T, d, fmt, out, dtype,
                          reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PKM_OK
             : PKM_ERR_CUDA;
}

}  // extern "C"
