// residual_norm.cu -- what lies between two sub-blocks, in one pass over the
// rows:
//
//   u  = post(branch) * post_weight          (norm after a sub-block)
//   x' = x + r * gate[b] * u                 (gated, scaled residual)
//   y  = pre(x') * pre_weight * (1 + scale[b]) + shift[b]   (norm before the next)
//
// post, pre: no norm, LayerNorm (biased variance) or RMS norm, each with eps
// under the root and statistics in fp32 (LayerNorm: the mean first, then the
// centred squares).  y is formed from x' before it is rounded for storage.
#include "af_internal.h"
#include "ptx.cuh"

namespace af {

namespace {

constexpr int RN_THREADS = 256;

// Sum of v over the block, to every thread.
__device__ __forceinline__ float rn_block_sum(float v, float* red) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();  // the last call's values are read
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int i = 0; i < RN_THREADS / 32; ++i) v += red[i];
  return v;
}
__device__ __forceinline__ float rn_block_max(float v, float* red) {
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < RN_THREADS / 32; ++i) v = fmaxf(v, red[i]);
  return v;
}

// (mean, 1 / root) of the row that this thread holds every RN_THREADS-th
// value of (each thread reads only what it wrote).
__device__ __forceinline__ float2 rn_stats(const float* row, int D, int kind, float eps, float* red) {
  if (kind == NORM_NONE) return make_float2(0.f, 1.f);
  float mean = 0.f;
  if (kind == NORM_LAYER) {
    float s = 0.f;
    for (int d = threadIdx.x; d < D; d += RN_THREADS) s += row[d];
    mean = rn_block_sum(s, red) / D;
  }
  float q = 0.f;
  for (int d = threadIdx.x; d < D; d += RN_THREADS) {
    const float c = row[d] - mean;
    q += c * c;
  }
  return make_float2(mean, rsqrtf(rn_block_sum(q, red) / D + eps));
}

template <typename T>
__device__ __forceinline__ float rn_load(const void* p, size_t i) {
  if constexpr (sizeof(T) == 4) return static_cast<const float*>(p)[i];
  else return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
}
template <typename T>
__device__ __forceinline__ void rn_store(void* p, size_t i, float v) {
  if constexpr (sizeof(T) == 4) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(pack_bf16(v, 0.f));
}

// One CTA per row, the row in shared memory as fp32; any width and alignment.
template <typename T, bool OUT8>
__global__ void __launch_bounds__(RN_THREADS) residual_norm_row_kernel(ResidualNormParams p) {
  extern __shared__ float row[];
  __shared__ float red[RN_THREADS / 32];
  const int D = p.D;
  const size_t r = blockIdx.x, base = r * D;
  const size_t mo = r / p.rows_per_batch * static_cast<size_t>(p.mod_stride);
  if (p.branch) {
    for (int d = threadIdx.x; d < D; d += RN_THREADS) row[d] = rn_load<T>(p.branch, base + d);
    const float2 st = rn_stats(row, D, p.post, p.eps, red);
    for (int d = threadIdx.x; d < D; d += RN_THREADS) {
      float u = (row[d] - st.x) * st.y;
      if (p.post_weight) u *= p.post_weight[d];
      if (p.gate) u *= p.gate[mo + d];
      row[d] = rn_load<T>(p.x, base + d) + p.residual_scale * u;
    }
  } else {
    for (int d = threadIdx.x; d < D; d += RN_THREADS) row[d] = rn_load<T>(p.x, base + d);
  }
  if (p.x_out)
    for (int d = threadIdx.x; d < D; d += RN_THREADS) rn_store<T>(p.x_out, base + d, row[d]);
  if (!p.y) return;
  const float2 st = rn_stats(row, D, p.pre, p.eps, red);
  float amax = 0.f;
  for (int d = threadIdx.x; d < D; d += RN_THREADS) {
    float y = (row[d] - st.x) * st.y;
    if (p.pre_weight) y *= p.pre_weight[d];
    if (p.scale) y *= 1.0f + p.scale[mo + d];
    if (p.shift) y += p.shift[mo + d];
    if constexpr (OUT8) {
      row[d] = y;
      amax = fmaxf(amax, fabsf(y));
    } else {
      rn_store<T>(p.y, base + d, y);
    }
  }
  if constexpr (OUT8) {
    amax = rn_block_max(amax, red);
    const float inv = amax > 0.f ? 448.0f / amax : 1.0f;
    uint8_t* y8 = static_cast<uint8_t*>(p.y) + base;
    for (int d = threadIdx.x; d < D; d += RN_THREADS)
      y8[d] = static_cast<uint8_t>(pack_e4m3x4(row[d] * inv, 0.f, 0.f, 0.f));
    if (threadIdx.x == 0) p.yscale[r] = amax > 0.f ? amax / 448.0f : 1.0f;
  }
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualNormParams& p, bool f32, cudaStream_t s) {
  const size_t rows = static_cast<size_t>(p.B) * p.rows_per_batch;
  const size_t smem = static_cast<size_t>(p.D) * sizeof(float);
  auto launch = [&](auto kernel) {
    if (smem > 48 * 1024) {
      const cudaError_t e =
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
      if (e != cudaSuccess) return e;
    }
    kernel<<<static_cast<unsigned>(rows), RN_THREADS, smem, s>>>(p);
    return cudaGetLastError();
  };
  if (p.yscale) return f32 ? launch(residual_norm_row_kernel<float, true>) : launch(residual_norm_row_kernel<uint16_t, true>);
  return f32 ? launch(residual_norm_row_kernel<float, false>) : launch(residual_norm_row_kernel<uint16_t, false>);
}

}  // namespace af
