// w4.cu -- weights in 4 bits with one scale per group of columns: the
// quantiser, its inverse and the product with a few rows of activations.
//
//   value(n, k) = s[k / G, n] * (c[n, k] - 8),   c in 0..15, G = 32, 64 or 128
//
// Layout (the same for every call): codes [N, ceil(K / G) * G / 2] bytes, code
// k of row n in the low (k even) or high (k odd) nibble of byte k / 2, code 8
// (the value zero) behind column K; scales bf16 [ceil(K / G), scale_stride],
// group-major so the scales of neighbouring rows are neighbours.
#include "af_internal.h"
#include "ptx.cuh"

namespace af {

// ------------------------------------------------------------------ loads / stores of either type
__device__ __forceinline__ float w4_load(const void* p, int f32, size_t i) {
  return f32 ? static_cast<const float*>(p)[i]
             : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
}
__device__ __forceinline__ void w4_store(void* p, int f32, size_t i, float v) {
  if (f32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(pack_bf16(v, 0.f));
}
__device__ __forceinline__ float w4_bf16(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }
__device__ __forceinline__ float w4_silu(float a) { return a / (1.0f + expf(-a)); }

// ------------------------------------------------------------------ quantiser
// Per row and group: a = max |w|, s = bf16(a / 7) to nearest even, c = 8 +
// the whole number nearest to w / s (ties to even), 8 where s is zero.  Both
// divisions are IEEE fp32 ones.  They decide as real numbers would: a border
// between two codes, (j + 1/2) s, and one between two scales, times 7, are
// fp32 numbers (4 x 8 and 9 x 3 bits), and a w or a next to one is off it by
// at least 2^-24 relative, which the rounded quotient still shows.
// One warp per row; a lane takes two neighbouring columns, so a group is
// G / 2 lanes' work: 16, 32, or 32 lanes twice.
template <int G>
__global__ void __launch_bounds__(256) quantize_rows_w4_kernel(const void* __restrict__ w, int f32, int N, int K,
                                                               int groups, uint8_t* __restrict__ codes,
                                                               uint16_t* __restrict__ scales, int scale_stride) {
  const int n = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (n >= N) return;
  uint8_t* cr = codes + static_cast<size_t>(n) * groups * (G / 2);
  const size_t row = static_cast<size_t>(n) * K;
  constexpr int BPL = G == 128 ? 2 : 1;      // bytes (pairs of columns) per lane and step
  constexpr int LPG = G / 2 / BPL;           // lanes that share a group
  for (int j = lane * BPL; j < (groups * (G / 2) + 32 * BPL - 1) / (32 * BPL) * (32 * BPL); j += 32 * BPL) {
    float v[2 * BPL], a = 0.f;
#pragma unroll
    for (int e = 0; e < 2 * BPL; ++e) {
      const int k = 2 * j + e;
      v[e] = k < K ? w4_load(w, f32, row + k) : 0.f;
      a = fmaxf(a, fabsf(v[e]));
    }
#pragma unroll
    for (int o = LPG / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    const uint16_t sb = static_cast<uint16_t>(pack_bf16(__fdiv_rn(a, 7.0f), 0.f));
    const float s = w4_bf16(sb);
    const int g = 2 * j / G;
    if (g >= groups) continue;
    if ((lane & (LPG - 1)) == 0) scales[static_cast<size_t>(g) * scale_stride + n] = sb;
#pragma unroll
    for (int b = 0; b < BPL; ++b) {
      int c[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        c[e] = s > 0.f ? min(15, max(0, 8 + __float2int_rn(__fdiv_rn(v[2 * b + e], s)))) : 8;
      cr[j + b] = static_cast<uint8_t>(c[0] | c[1] << 4);
    }
  }
}

cudaError_t launch_quantize_rows_w4(const void* w, bool f32, int N, int K, int group, uint8_t* codes,
                                    uint16_t* scales, int scale_stride, cudaStream_t s) {
  const int groups = (K + group - 1) / group, blocks = (N + 7) / 8;
  switch (group) {
    case 32: quantize_rows_w4_kernel<32><<<blocks, 256, 0, s>>>(w, f32, N, K, groups, codes, scales, scale_stride); break;
    case 64: quantize_rows_w4_kernel<64><<<blocks, 256, 0, s>>>(w, f32, N, K, groups, codes, scales, scale_stride); break;
    case 128: quantize_rows_w4_kernel<128><<<blocks, 256, 0, s>>>(w, f32, N, K, groups, codes, scales, scale_stride); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

// ------------------------------------------------------------------ values
__global__ void __launch_bounds__(256) dequantize_rows_w4_kernel(const uint8_t* __restrict__ codes,
                                                                 const uint16_t* __restrict__ scales,
                                                                 int scale_stride, int N, int K, int group,
                                                                 void* __restrict__ out, int f32) {
  const int n = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (n >= N) return;
  const uint8_t* cr = codes + static_cast<size_t>(n) * ((K + group - 1) / group) * (group / 2);
  const size_t row = static_cast<size_t>(n) * K;
  for (int k = lane; k < K; k += 32) {
    const int c = (cr[k >> 1] >> (4 * (k & 1))) & 15;
    w4_store(out, f32, row + k, w4_bf16(scales[static_cast<size_t>(k / group) * scale_stride + n]) * (c - 8));
  }
}

cudaError_t launch_dequantize_rows_w4(const uint8_t* codes, const uint16_t* scales, int scale_stride, int N, int K,
                                      int group, void* out, bool f32, cudaStream_t s) {
  dequantize_rows_w4_kernel<<<(N + 7) / 8, 256, 0, s>>>(codes, scales, scale_stride, N, K, group, out, f32);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ product
// out[m, n] = bias[n] + sum_k f(x[m, k]) value(n, k): one warp per weight row,
// eight rows of x at a time, fp32 throughout.
constexpr int W4_MB = 8;

__global__ void __launch_bounds__(256) linear_w4_kernel(W4Params p) {
  const int n = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (n >= p.N) return;
  const int m0 = blockIdx.y * W4_MB, mb = min(W4_MB, p.M - m0);
  const int groups = (p.K + p.group - 1) / p.group;
  const uint8_t* cr = p.codes + static_cast<size_t>(n) * groups * (p.group / 2);
  float acc[W4_MB];
#pragma unroll
  for (int i = 0; i < W4_MB; ++i) acc[i] = 0.f;
  for (int k = lane; k < p.K; k += 32) {
    const int c = (cr[k >> 1] >> (4 * (k & 1))) & 15;
    const float w = w4_bf16(p.scales[static_cast<size_t>(k / p.group) * p.scale_stride + n]) * (c - 8);
#pragma unroll
    for (int i = 0; i < W4_MB; ++i) {
      if (i < mb) {
        float x = w4_load(p.x, p.x_f32, static_cast<size_t>(m0 + i) * p.K + k);
        if (p.silu) x = w4_silu(x);
        acc[i] += w * x;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < W4_MB; ++i) {
    for (int o = 16; o > 0; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    if (lane == 0 && i < mb)
      w4_store(p.out, p.out_f32, static_cast<size_t>(m0 + i) * p.out_stride + n, acc[i] + (p.bias ? p.bias[n] : 0.f));
  }
}

cudaError_t launch_linear_w4(const W4Params& p, cudaStream_t s) {
  linear_w4_kernel<<<dim3((p.N + 7) / 8, (p.M + W4_MB - 1) / W4_MB), 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace af
