// w4.cu -- weights in 4 bits with one scale per group of columns: the
// quantiser, its inverse and the product with a few rows of activations.
//
//   value(n, k) = s[k / G, n] * (c[n, k] - 8),   c in 0..15, G = 32, 64 or 128
//
// Layout (the same for every call): codes [N, ceil(K / G) * G / 2] bytes, code
// k of row n in the low (k even) or high (k odd) nibble of byte k / 2, code 8
// (the value zero) behind column K; scales bf16 [ceil(K / G), scale_stride],
// group-major so the scales of neighbouring rows are neighbours.
#include <atomic>

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
// a / (1 + exp(-a)) to two steps.  Numerator and divisor are a quarter of that, which holds up to exp's largest
// value; an approximate reciprocal's quotient is refined once by its remainder, without the branches of a true
// division (1 x 32 -> 192 and 2 x 3072 -> 18432: 5.6 and 12.0 us with it, 4.2 and 11.6 so).  Below -88.7, where exp(-a) passes fp32: 0, NaN for -infinity.
__device__ __forceinline__ float w4_silu(float a) {
  const float x = 0.25f * a, y = fmaf(0.25f, expf(-a), 0.25f);
  const float r = __fdividef(1.0f, y), q = x * r;
  const float f = fmaf(fmaf(-q, y, x), r, q);
  return a > 88.0f ? a : a < -88.7f ? a * 0.0f : f;
}

// the larger one, NaN if either is
__device__ __forceinline__ float w4_max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// packed fp32 pairs
__device__ __forceinline__ uint64_t w4_pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t w4_add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t w4_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float w4_lo(uint64_t a) { return __uint_as_float(static_cast<uint32_t>(a)); }
__device__ __forceinline__ float w4_hi(uint64_t a) { return __uint_as_float(static_cast<uint32_t>(a >> 32)); }
constexpr float W4_MAGIC = 12582912.0f;    // 1.5 * 2^23: the bits of W4_MAGIC + i are its bits + i for |i| < 2^22

// Eight columns of a row from column k as stored (bf16 in the first vector,
// fp32 in both), zero behind column K, and their values.  vec: rows are whole
// 16-byte vectors.
struct W4Raw {
  uint4 a, b;
};
__device__ __forceinline__ W4Raw w4_load8(const void* p, int f32, int vec, size_t row, int k, int K) {
  W4Raw r{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  if (vec) {
    if (k < K) {
      const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + (row + k) * (f32 ? 4 : 2));
      r.a = s[0];
      if (f32) r.b = s[1];
    }
    return r;
  }
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    w[e] = k + e < K ? (f32 ? static_cast<const uint32_t*>(p)[row + k + e] : static_cast<const uint16_t*>(p)[row + k + e])
                     : 0u;
  if (f32) {
    r.a = make_uint4(w[0], w[1], w[2], w[3]);
    r.b = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
    r.a = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
  }
  return r;
}
__device__ __forceinline__ void w4_values(const W4Raw& r, int f32, float (&v)[8]) {
  const uint32_t q[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    v[e] = f32 ? __uint_as_float(q[e]) : (e & 1) ? bf16_hi(q[e / 2]) : bf16_lo(q[e / 2]);
}

// ------------------------------------------------------------------ quantiser
// Per row and group: a = max |w|, s = bf16(a / 7) to nearest even, c = 8 +
// the whole number nearest to w / s (ties to even), 8 where s is zero, decided
// as real numbers would.  a / 7 is an IEEE fp32 division: a border between two
// scales, times 7, is an fp32 number (9 x 3 bits), and an a next to one is off
// it by at least 2^-24 relative, which the rounded quotient still shows.  For
// fp32 weights a first guess w (1 / s) is put right by what it leaves, w - q s,
// which fp32 holds exactly.  bf16 weights are eight bits over eight bits:
// off a border (j + 1/2) by at least 2^-13, or on it, so w (1 / s) rounded to
// a multiple of 2^-14 decides the same for a third of the instructions; and a
// is never 7 times a border of s (an odd number of nine bits), so a (1 / 7) does.
// Bound: HBM (2.5 or 4.5 bytes a weight).  A CTA takes 32 rows by 256 columns:
// a warp reads four rows, 512 bytes of each in one load per lane, all four in
// flight; a group is G / 8 lanes; the scales of 32 rows go out together.
constexpr int W4Q_ROWS = 4;  // rows per warp

template <int G, bool F32>
__global__ void __launch_bounds__(256, F32 ? 4 : 6) quantize_rows_w4_kernel(const void* __restrict__ w, int vec, int N, int K,
                                                               int groups, uint8_t* __restrict__ codes,
                                                               uint16_t* __restrict__ scales, int scale_stride) {
  __shared__ uint16_t sc[256 / G][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunks = (groups * G + 255) / 256, tile = blockIdx.x / chunks, chunk = blockIdx.x - tile * chunks;
  const int n0 = tile * 32, r0 = n0 + warp * W4Q_ROWS;
  const int k = chunk * 256 + lane * 8, g = lane / (G / 8);
  const bool in = k < groups * G;
  W4Raw raw[W4Q_ROWS];
#pragma unroll
  for (int i = 0; i < W4Q_ROWS; ++i)  // rows behind the last repeat it, and are not written
    raw[i] = w4_load8(w, F32, vec, static_cast<size_t>(min(r0 + i, N - 1)) * K, k, K);
#pragma unroll
  for (int i = 0; i < W4Q_ROWS; ++i) {
    float v[8];
    w4_values(raw[i], F32, v);
    float a = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(v[e]));
#pragma unroll
    for (int o = G / 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    const uint16_t sb = static_cast<uint16_t>(pack_bf16(F32 ? __fdiv_rn(a, 7.0f) : a * (1.0f / 7.0f), 0.f));
    const float s = w4_bf16(sb);
    // w / s rounded to a whole number, as a float
    uint64_t c[4];  // columns 2 e and 2 e + 1
    if (F32 || s < 0x1p-100f) {
      // the nearest of w (1 / s), put right by what is left of w: w - q s is exact
      const float up = s < 0x1p-100f ? 0x1p100f : 1.0f, t = s * up, half = 0.5f * t;
      const float inv = s > 0.f ? __fdividef(1.0f, t) : 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float d[2];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const float x = v[2 * e + o] * up;
          float n = rintf(x * inv);
          const float left = fmaf(-n, t, x), mag = fabsf(left);
          const bool odd = static_cast<int>(n) & 1;
          if (mag > half || (mag == half && odd)) n += copysignf(1.0f, left);
          d[o] = s > 0.f ? fminf(7.f, fmaxf(-8.f, n)) : 0.f;
        }
        c[e] = w4_pack2(d[0], d[1]);
      }
    } else {
      float inv;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
      const uint64_t inv2 = w4_pack2(inv, inv);
      const uint64_t snap = w4_pack2(768.0f, 768.0f), unsnap = w4_pack2(-768.0f, -768.0f);  // 768: steps of 2^-14
      const uint64_t whole = w4_pack2(W4_MAGIC, W4_MAGIC), unwhole = w4_pack2(-W4_MAGIC, -W4_MAGIC);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        c[e] = w4_add2(w4_add2(w4_add2(w4_fma2(w4_pack2(v[2 * e], v[2 * e + 1]), inv2, snap), unsnap), whole),
                       unwhole);
    }
    // nibbles: columns e and e + 2 are 8 bits apart in a half word, the low 16 bits of 2^23 + their whole part;
    // + 8 for every nibble
    uint32_t h[4];
    const uint64_t up = w4_pack2(256.0f, 256.0f), eights = w4_pack2(8388608.0f + 2056.0f, 8388608.0f + 2056.0f);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint64_t t = w4_add2(w4_fma2(c[2 * e + 1], up, c[2 * e]), eights);
      h[2 * e] = static_cast<uint32_t>(t);
      h[2 * e + 1] = static_cast<uint32_t>(t >> 32);
    }
    const uint32_t lo = __byte_perm(h[0], h[2], 0x5410), hi = __byte_perm(h[1], h[3], 0x5410);
    const int n = r0 + i;
    if (n < N && in)
      reinterpret_cast<uint32_t*>(codes + static_cast<size_t>(n) * groups * (G / 2))[k >> 3] = lo | hi << 4;
    if (lane % (G / 8) == 0) sc[g][warp * W4Q_ROWS + i] = sb;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < (256 / G) * 32; i += 256) {
    const int gi = i >> 5, n = n0 + (i & 31), at = chunk * (256 / G) + gi;
    if (n < N && at < groups) scales[static_cast<size_t>(at) * scale_stride + n] = sc[gi][i & 31];
  }
}

static bool w4_vec(const void* p, int K) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && K % 8 == 0;
}

cudaError_t launch_quantize_rows_w4(const void* w, bool f32, int N, int K, int group, uint8_t* codes,
                                    uint16_t* scales, int scale_stride, cudaStream_t s) {
  const int groups = (K + group - 1) / group;
  const int64_t grid = static_cast<int64_t>((groups * group + 255) / 256) * ((N + 31) / 32);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  const int vec = w4_vec(w, K);
#define AF_Q4_CASE(G_)                                                                                              \
  if (group == G_) {                                                                                                \
    auto kernel = f32 ? quantize_rows_w4_kernel<G_, true> : quantize_rows_w4_kernel<G_, false>;                     \
    kernel<<<static_cast<unsigned>(grid), 256, 0, s>>>(w, vec, N, K, groups, codes, scales, scale_stride);          \
    return cudaGetLastError();                                                                                      \
  }
  AF_Q4_CASE(32)
  AF_Q4_CASE(64)
  AF_Q4_CASE(128)
#undef AF_Q4_CASE
  return cudaErrorInvalidValue;
}

// ------------------------------------------------------------------ values
// The quantiser's tiles the other way round, bound by HBM too: a lane turns 4
// bytes of codes into eight values.  8388608 + c is the pattern 0x4B000000 | c.
template <bool VEC>
__global__ void __launch_bounds__(256) dequantize_rows_w4_kernel(const uint8_t* __restrict__ codes,
                                                                 const uint16_t* __restrict__ scales,
                                                                 int scale_stride, int N, int K, int group,
                                                                 void* __restrict__ out, int f32) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunks = (K + 255) / 256, tile = blockIdx.x / chunks;
  const int r0 = tile * 32 + warp * W4Q_ROWS, k = (blockIdx.x - tile * chunks) * 256 + lane * 8;
  const int groups = (K + group - 1) / group;
  if constexpr (!VEC) {  // rows that are not whole vectors: a lane takes every 32nd column, so that stores are coalesced
    const int k0 = k - lane * 8 + lane;
#pragma unroll 1
    for (int i = 0; i < W4Q_ROWS && r0 + i < N; ++i) {
      const uint8_t* cr = codes + static_cast<size_t>(r0 + i) * groups * (group / 2);
      uint8_t b[8];
      uint16_t sb[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int kk = min(k0 + 32 * e, K - 1);
        b[e] = cr[kk >> 1];
        sb[e] = scales[static_cast<size_t>(kk / group) * scale_stride + r0 + i];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (k0 + 32 * e < K)
          w4_store(out, f32, static_cast<size_t>(r0 + i) * K + k0 + 32 * e,
                   w4_bf16(sb[e]) * (((b[e] >> (4 * (k0 & 1))) & 15) - 8));
    }
    return;
  }
  if (k >= K) return;
  uint32_t w[W4Q_ROWS];
  float s[W4Q_ROWS];
#pragma unroll
  for (int i = 0; i < W4Q_ROWS; ++i) {
    const int n = min(r0 + i, N - 1);
    w[i] = reinterpret_cast<const uint32_t*>(codes + static_cast<size_t>(n) * groups * (group / 2))[k >> 3];
    s[i] = w4_bf16(scales[static_cast<size_t>(k / group) * scale_stride + n]);
  }
#pragma unroll
  for (int i = 0; i < W4Q_ROWS; ++i) {
    if (r0 + i >= N) break;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = s[i] * (__uint_as_float(((w[i] >> (4 * e)) & 15u) | 0x4B000000u) - 8388616.0f);
    uint4* d = reinterpret_cast<uint4*>(static_cast<uint8_t*>(out) +
                                        (static_cast<size_t>(r0 + i) * K + k) * (f32 ? 4 : 2));
    if (f32) {
      d[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
      d[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
    } else {
      d[0] = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    }
  }
}

cudaError_t launch_dequantize_rows_w4(const uint8_t* codes, const uint16_t* scales, int scale_stride, int N, int K,
                                      int group, void* out, bool f32, cudaStream_t s) {
  const int64_t grid = static_cast<int64_t>((K + 255) / 256) * ((N + 31) / 32);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  auto kernel = w4_vec(out, K) ? dequantize_rows_w4_kernel<true> : dequantize_rows_w4_kernel<false>;
  kernel<<<static_cast<unsigned>(grid), 256, 0, s>>>(codes, scales, scale_stride, N, K, group, out, f32);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ product
// out[m, n] = bias[n] + sum_k f(x[m, k]) s[k / G, n] (c[n, k] - 8).
//
// Each group's sum runs on mma.sync m16n8k32 in whole numbers: the weights are
// the 16-row operand, the codes c as they are (two masks and a shift unpack
// eight), the columns are rows of x as 32-bit fixed point, cut into four
// signed bytes, a column each.  The step per row of x and 256 columns is a power
// of two, at most 2^-30 (1 + 2^-7) of the largest magnitude a there: a value of
// at least a 2^-6 enters exactly, any other off by at most half a step.  Three
// bytes (24 bits) leave values next to a far larger one with too few bits,
// which shows where the larger one meets a zero weight; the fourth costs
// nothing at one and two rows of x (eight columns are one operand).
// Sums are exact (at most 15 * 128 * 128); sum c q - 8 sum q is formed with
// 8 sum q known per group and column, then multiplied by the group's scale and
// added up in fp32.
// Other operands cost more to make: c - 8 in fp16 (x in two pieces) took 77
// instructions per 16 rows and 64 columns against 46, near the 91 issue slots
// that HBM leaves time for; 743424 x 3072 with two rows of x took 218 us
// against 198 (6.1 TB/s).
// One step does not fit 256 columns of which most are far below the largest:
// the others' last bits show in weights that are zero at the few large ones.
// Where fewer than four, or than one in 16, of the values other than zero reach
// 2^-10 of the largest, these are set aside (W4_FAR a row at most, in the order of
// their columns) and added as fp32 terms of their own to the finished sums; the
// step is that of the rest.  A row with more of them, an infinity or a NaN is
// summed term by term in fp32 (w4_plain_sum).  18432 x 3072 with a value set
// aside in one row of x and in each of seven: 10.3 us and 24 against 9.2 and 18.5;
// one row and seven summed term by term 143 and 634.
//
// Bound: the code bytes from HBM (4.25 bits a weight at G = 64).  One CTA of W
// warps per SM, RW x KW of them: RW blocks of 32 rows by KW ways to
// share the columns, in chunks of 256 (128 bytes of codes).  Each warp streams
// its own 32 rows through its own ring of 4 KB stages: one lane issues the TMA
// loads of a stage as soon as the warp has read it, so no warp waits for
// another until a round's sums are joined.  Rows of a stage are 128-byte lines
// under the 128-byte swizzle.  A lane (g, t) holds an equal share of a row's
// group (4, 8 or 16 bytes at G = 32, 64, 128), read by one load; the rows are
// dealt to g = 0..7 so that each load touches all 32 banks.  Of a word of
// eight codes the even nibbles form one operand register and the odd ones
// another; x lies in shared memory in that order.
// Warps of a CTA by the 8-column blocks of x: with more blocks than one the
// registers of twelve (168 a thread) let 32 rows share the reads of x, and the
// smaller rings leave shared memory for it.  With three columns a row of x,
// sixteen warps of 16 rows against twelve of 32: 743424 x 3072 with eight rows of
// x 305 us and 298, 55296 x 3072 with twenty 65 and 62.  Four columns against
// three, 120000 x 3072 with 1, 4, 8, 10 and 32 rows: 37, 49, 74, 101 and 231 us
// against 38, 50, 63, 165 (x in parts) and 185.
__host__ __device__ constexpr int w4_warps(int nt) { return nt == 1 ? 16 : 12; }
constexpr int W4_ROWS = 32;                               // rows per warp
// Rows of a warp whose sums are joined through shared memory at a time, and the
// floats between rows of x there (16 mod 32: two of them fill the banks).
__host__ __device__ constexpr int w4_red_rows(int nt) { return nt == 1 ? W4_ROWS : 16; }
__host__ __device__ constexpr int w4_red_pitch(int nt) { return nt == 1 ? 48 : 16; }
constexpr int W4_CHUNK = 256;                             // columns per chunk
constexpr int W4_MAX_NT = 4;                              // 8-column blocks
constexpr int W4_SMEM_MAX = 227 * 1024;
constexpr int W4_STATIC = 4096;                           // of it the barriers and values set aside, and spare
constexpr int W4_MAX_STAGES = 4;
constexpr int W4_DIGITS = 4;                              // columns of a row of x, two neighbouring lanes' of a block
constexpr int W4_MAX_ROWS = W4_MAX_NT * 8 / W4_DIGITS;    // rows of x per CTA

struct W4Launch {
  W4Params p;
  int rows_m;               // rows of x per CTA (blockIdx.y: which)
  int rw;                   // row blocks per CTA and round; W / rw warps share a block's chunks
  int blocks, chunks, seg_chunks, segs, stages;
  int x_pitch;              // bytes between columns of x in shared memory
  int x_vec;                // x in 16-byte loads: aligned, K a multiple of 8
};

// Fixed point: a (1 + 2^-7) < 2^(e + 1) counts in steps of 2^(e - 30), so that
// a's number is below 2^31 / (1 + 2^-7) = 2130836295; four signed bytes reach
// 2139062143.  e is kept so that the step is no smaller than fp32's smallest, 2^-149.
constexpr float W4_SMALL = 0x1p-90f;       // where the largest is below this, scaled by 2^24 first
constexpr int W4_FAR = 32;                 // values set aside a row: a warp's lanes
constexpr int W4_NOT_FINITE = 1 << 30;     // their count where the row has an infinity or NaN
constexpr int W4_MAGIC_BITS = 0x4B400000;

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint64_t lds_u64(uint32_t a) {
  uint64_t v;
  asm volatile("ld.shared.u64 %0, [%1];" : "=l"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts_f1(uint32_t a, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ float lds_bf16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return w4_bf16(v);
}
// d = a b + c: 16 rows of codes (unsigned bytes), 8 columns of x (signed), 32 deep.
__device__ __forceinline__ void mma_16832(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1, int c0, int c1, int c2, int c3) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(c0), "r"(c1), "r"(c2), "r"(c3));
}

// sum_k f(x[m, k]) value(n, k) term by term, for rows of x without a fixed point.
__device__ __noinline__ float w4_plain_sum(const W4Params& p, int vec, int m, int n) {
  const size_t row_bytes = static_cast<size_t>((p.K + p.group - 1) / p.group) * (p.group / 2);
  const uint4* cr = reinterpret_cast<const uint4*>(p.codes + n * row_bytes);
  float v = 0.f;
  for (int k = 0; k < p.K; k += 32) {  // 16 bytes of codes, of one group
    const uint4 q = cr[k >> 5];
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    const float s = w4_bf16(p.scales[static_cast<size_t>(k / p.group) * p.scale_stride + n]);
    float part = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x[8];
      w4_values(w4_load8(p.x, p.x_f32, vec, static_cast<size_t>(m) * p.K, k + 8 * j, p.K), p.x_f32, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (p.silu) x[e] = w4_silu(x[e]);
        part = fmaf(x[e], s * (static_cast<int>((w[j] >> (4 * e)) & 15u) - 8), part);
      }
    }
    v += part;
  }
  return v;
}

// Values of x set aside: how many of each row (W4_FAR + 1 and more: it is summed
// term by term), their columns and values.
struct W4Far {
  int n[W4_MAX_ROWS];
  int k[W4_MAX_ROWS][W4_FAR];
  float v[W4_MAX_ROWS][W4_FAR];
};
static_assert(sizeof(W4Far) + 16 * W4_MAX_STAGES * 8 + 64 <= W4_STATIC, "the kernel's own shared memory");

// The values of a row in the order of their columns: their order of arrival is
// not that of the next call, and sums would differ.  A warp a row.
__device__ __forceinline__ void w4_sort_far(W4Far& F, int m, int lane) {
  const int n = F.n[m];
  if (n < 2 || n > W4_FAR) return;
  const int k = lane < n ? F.k[m][lane] : INT32_MAX;
  const float v = lane < n ? F.v[m][lane] : 0.f;
  int rank = 0;
  for (int i = 0; i < n; ++i) rank += __shfl_sync(0xffffffffu, k, i) < k;
  __syncwarp();
  if (lane < n) {
    F.k[m][rank] = k;
    F.v[m][rank] = v;
  }
}

// What the set-aside values of row m add to row n of the weights.
__device__ __noinline__ float w4_far_sum(const W4Params& p, const W4Far& F, int m, int n) {
  const size_t row_bytes = static_cast<size_t>((p.K + p.group - 1) / p.group) * (p.group / 2);
  const uint8_t* cr = p.codes + n * row_bytes;
  float v = 0.f;
  for (int i = 0; i < F.n[m]; ++i) {
    const int k = F.k[m][i], c = (cr[k >> 1] >> (4 * (k & 1))) & 15;
    v = fmaf(F.v[m][i], w4_bf16(p.scales[static_cast<size_t>(k / p.group) * p.scale_stride + n]) * (c - 8), v);
  }
  return v;
}

// Where x lies in shared memory, as addresses: `cols` columns of bytes, the
// chunks' factors [chunk][NT * 8] and the groups' offsets [group][NT * 8].
struct W4X {
  uint32_t x, fac, off;
};

// `chunks` chunks of this CTA's rows of x from column k0 (zero behind column K)
// into shared memory.  A warp takes a row's chunk, a lane eight columns: of
// each digit one 8-byte store in the order 0, 2, 4, 6, 1, 3, 5, 7, as a word of
// codes unpacks.  fac: what the chunk's sums of a digit stand for; off: minus
// the magic number and 8 sum q of each group.  Values set aside go to F, in
// any order.  Returns whether this thread found one, or one that is not finite.
template <int G, int W, int NT>
__device__ __forceinline__ bool w4_stage_x(const W4Launch& L, int m0, int rows, const W4X& X, W4Far& F, int k0,
                                           int chunks) {
  bool found = false;
  const W4Params& p = L.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int items = rows * chunks;
  auto load = [&](int i) {
    const int j = min(i, items - 1), m = j / chunks;
    return w4_load8(p.x, p.x_f32, L.x_vec, static_cast<size_t>(m0 + m) * p.K, k0 + 8 * ((j - m * chunks) * 32 + lane),
                    p.K);
  };
  // the next item's loads are in flight while one is converted; one body, as
  // its instructions are fetched anew by every small call
  W4Raw next = load(warp);
#pragma unroll 1
  for (int i = warp; i < items; i += W) {
    const W4Raw raw = next;
    next = load(i + W);
    const int m = i / chunks, c = i - m * chunks;
    float v[8], a = 0.f;
    w4_values(raw, p.x_f32, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (p.silu) v[e] = w4_silu(v[e]);
      a = w4_max_nan(a, fabsf(v[e]));
    }
    float mine = a;
    asm volatile("redux.sync.max.abs.NaN.f32 %0, %0, 0xffffffff;" : "+f"(a));
    const bool fine = a < INFINITY;
    if (!fine && lane == 0) atomicMax(&F.n[m], W4_NOT_FINITE);
    found |= !fine;
    // 16 lanes with a value within 2^10 of the largest, or four and half as many as have any, are one in 16 at
    // least: nothing is set aside.  Else the values are counted; each turn takes some off and the next largest is
    // 2^10 below, so there are fewer than 30 turns.
    while (fine) {
      const float least = a * 0x1p-10f;
      const int lanes = __popc(__ballot_sync(0xffffffffu, mine >= least));
      if (lanes >= 16 || (lanes >= 4 && __popc(__ballot_sync(0xffffffffu, mine > 0.f)) <= 2 * lanes)) break;
      int count = 0;  // values of at least that, and 65536 for each that is not zero
#pragma unroll
      for (int e = 0; e < 8; ++e) count += (fabsf(v[e]) >= least ? 1 : 0) + (v[e] != 0.f ? 65536 : 0);
      count = __reduce_add_sync(0xffffffffu, count);
      const int near = count & 65535, some = count >> 16;
      if (some <= near || (near >= 4 && some <= 16 * near)) break;
      found = true;
      mine = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (fabsf(v[e]) >= least) {
          const int at = atomicAdd(&F.n[m], 1);
          if (at < W4_FAR) {
            F.k[m][at] = k0 + 8 * (c * 32 + lane) + e;
            F.v[m][at] = v[e];
          }
          v[e] = 0.f;
        }
        mine = fmaxf(mine, fabsf(v[e]));
      }
      a = mine;
      asm volatile("redux.sync.max.abs.f32 %0, %0, 0xffffffff;" : "+f"(a));
    }
    const bool small = a < W4_SMALL;
    if (small) {
      a *= 0x1p24f;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= 0x1p24f;
    }
    // biased e: 32 at least, which after the 2^24 is a step of 2^-149
    const int exp = max(static_cast<int>(__float_as_uint(fmaf(a, 0x1p-7f, a)) >> 23), 32);
    const float up = __uint_as_float(static_cast<uint32_t>(284 - exp) << 23);
    const float down = __uint_as_float(static_cast<uint32_t>(exp - 30) << 23) * (small ? 0x1p-24f : 1.0f);
    uint32_t f[8];  // four signed bytes each: q = d0 + 256 d1 + 65536 d2 + 16777216 d3
#pragma unroll
    for (int e = 0; e < 8; ++e)
      f[e] = (static_cast<uint32_t>(__float2int_rn(v[e] * up)) + 0x80808080u) ^ 0x80808080u;
#pragma unroll
    for (int d = 0; d < W4_DIGITS; ++d) {
      const uint32_t sel = 0x40u + 0x11u * d;  // byte d of both
      const uint32_t lo = __byte_perm(__byte_perm(f[0], f[2], sel), __byte_perm(f[4], f[6], sel), 0x5410);
      const uint32_t hi = __byte_perm(__byte_perm(f[1], f[3], sel), __byte_perm(f[5], f[7], sel), 0x5410);
      int sum = __dp4a(static_cast<int>(lo), 0x01010101, __dp4a(static_cast<int>(hi), 0x01010101, 0));
#pragma unroll
      for (int o = G / 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const int col = W4_DIGITS * m + d;
      asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(X.x + col * L.x_pitch + 8 * (c * 32 + lane)), "r"(lo),
                   "r"(hi)
                   : "memory");
      if (lane % (G / 8) == 0)
        sts_f1(X.off + ((c * (W4_CHUNK / G) + lane / (G / 8)) * (NT * 8) + col) * 4, -(W4_MAGIC + 8 * sum));
      if (lane == d) sts_f1(X.fac + (c * (NT * 8) + col) * 4, down * static_cast<float>(1 << (8 * d)));
    }
  }
  return found;
}

// N words at a shared-memory address.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&w)[N], uint32_t a) {
  if constexpr (N == 1) {
    w[0] = lds32(a);
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a));
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                   : "r"(a + 4 * i));
  }
}

template <int NT, int G>
__global__ void __launch_bounds__(32 * w4_warps(NT), 1)
    linear_w4_kernel(const __grid_constant__ CUtensorMap tm_codes, const __grid_constant__ CUtensorMap tm_scales,
                     const __grid_constant__ W4Launch L) {
  extern __shared__ uint8_t w4_raw[];
  constexpr int W = w4_warps(NT), THREADS = 32 * W;
  constexpr int ROWS = W4_ROWS, H = ROWS / 16;       // rows per warp, 16-row operands
  constexpr int STAGE = ROWS * W4_CHUNK / 2;         // code bytes per stage
  constexpr int RED = w4_red_rows(NT), RED_LD = w4_red_pitch(NT);
  constexpr int XR = NT * 8 / W4_DIGITS;             // rows of x of the columns
  __shared__ uint64_t full[W][W4_MAX_STAGES];
  __shared__ int abort_flag;
  __shared__ W4Far far;
  constexpr int GPC = W4_CHUNK / G;              // groups per chunk
  constexpr int WORDS = G / 32;                  // words of a lane per row and group
  constexpr int SC_STAGE = (ROWS * GPC * 2 + 127) / 128 * 128;  // scale bytes per stage
  const W4Params& p = L.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rw_n = L.rw, kw_n = W / rw_n;
  const int rw = warp % rw_n, kw = warp / rw_n;
  const uint32_t base = (smem_u32(w4_raw) + 1023u) & ~1023u;
  const uint32_t codes_s = base + warp * L.stages * STAGE;
  const uint32_t sc_s = base + W * L.stages * STAGE + warp * L.stages * SC_STAGE;
  const uint32_t red_base = base + W * L.stages * (STAGE + SC_STAGE);
  const int m0 = blockIdx.y * L.rows_m, rows = min(L.rows_m, p.M - m0), cols = W4_DIGITS * rows;
  W4X X;
  X.x = red_base + W * XR * RED_LD * 4;
  X.fac = X.x + W4_DIGITS * L.rows_m * L.x_pitch;
  X.off = X.fac + L.seg_chunks * NT * 32;
  if (threadIdx.x < W4_MAX_ROWS) far.n[threadIdx.x] = 0;
  if (threadIdx.x == 0) abort_flag = 0;
  if (lane == 0) {
    for (int i = 0; i < L.stages; ++i) mbar_init(smem_u32(&full[warp][i]), 1);
    fence_mbar_init();
  }

  const uint32_t bar0 = smem_u32(&full[warp][0]);
  // this warp's stages in order: row block by row block, its chunks kw, kw + KW, ...
  // Row blocks are dealt to the CTAs in turn, RW per round: in the last round
  // every CTA has about as many as the others.
  const int first_block = rw * gridDim.x + blockIdx.x, round_blocks = rw_n * gridDim.x;
  int ld_block = kw < L.chunks ? first_block : L.blocks, ld_chunk = kw, ld_st = 0;  // the next to load (lane 0)
  auto load_next = [&] {
    if (ld_block >= L.blocks) return;
    const int n0 = ld_block * ROWS;
    const uint32_t bar = bar0 + 8 * ld_st;
    mbar_arrive_expect_tx(bar, STAGE + ROWS * GPC * 2);
    tma_load_2d(codes_s + ld_st * STAGE, &tm_codes, bar, ld_chunk * (W4_CHUNK / 2), n0);
    tma_load_2d(sc_s + ld_st * SC_STAGE, &tm_scales, bar, n0, ld_chunk * GPC);
    if (++ld_st == L.stages) ld_st = 0;
    ld_chunk += kw_n;
    if (ld_chunk >= L.chunks) {
      ld_chunk = kw;
      ld_block += round_blocks;
    }
  };
  if (lane == 0) {
    prefetch_tmap(&tm_codes);
    prefetch_tmap(&tm_scales);
    for (int i = 0; i < L.stages; ++i) load_next();
  }
  __syncwarp();

  const int g = lane >> 2, t = lane & 3;
  // the row (of 8) that g stands for: the lanes of one bank cycle (32, 16, 8
  // at 4, 8, 16 bytes a lane) must differ in the 16-byte piece they read
  const int r8 = WORDS == 1 ? g : WORDS == 2 ? 2 * (g & 3) + (g >> 2) : 4 * (g & 1) + (g >> 1);
  uint32_t xcol[NT];  // this lane's column of each 8-column block; those past the last repeat it, unused
#pragma unroll
  for (int i = 0; i < NT; ++i) xcol[i] = X.x + min(8 * i + g, cols - 1) * L.x_pitch + 8 * WORDS * t;
  // this lane's bytes of group 0 in row r8 of a stage; group gi is at ^ (gi * 16 * WORDS)
  const uint32_t mine = r8 * 128 + ((((WORDS * t) >> 2) ^ r8) << 4) + 4 * ((WORDS * t) & 3);
  const uint32_t red = red_base + warp * XR * RED_LD * 4;
  int4 magic;  // four registers of their own: the first sum of a group starts from them
  asm volatile("mov.b32 %0, %4; mov.b32 %1, %4; mov.b32 %2, %4; mov.b32 %3, %4;"
               : "=r"(magic.x), "=r"(magic.y), "=r"(magic.z), "=r"(magic.w)
               : "n"(W4_MAGIC_BITS));
  bool ok = true;
  int st = 0;
  uint32_t ph = 0;
  int any_far = 0;  // of the whole CTA
  if (L.segs == 1) {
    __syncthreads();  // far.n is clear
    any_far = __syncthreads_or(w4_stage_x<G, W, NT>(L, m0, rows, X, far, 0, L.seg_chunks));
    // (segs > 1: at the first part, before the first wait too)
  }
  for (int round = 0; round * round_blocks < L.blocks; ++round) {
    const int block = first_block + round * round_blocks;
    float acc[H][NT][2];  // this lane's two digits of a row of x together; rows r8 and r8 + 8
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[h][i][0] = acc[h][i][1] = 0.f;
    int xc = kw;  // the chunk's place in the part of x at hand
    for (int chunk = 0; chunk < L.chunks; chunk += kw_n, xc += kw_n) {
      if (L.segs > 1 && chunk % L.seg_chunks == 0) {  // x does not fit whole: its next part
        __syncthreads();
        if (chunk == 0 && any_far) {  // x anew
          if (threadIdx.x < W4_MAX_ROWS) far.n[threadIdx.x] = 0;
          __syncthreads();
        }
        any_far |= __syncthreads_or(w4_stage_x<G, W, NT>(L, m0, rows, X, far, chunk * W4_CHUNK, L.seg_chunks));
        xc = kw;
      }
      if (block >= L.blocks || chunk + kw >= L.chunks) continue;  // the last round, a last step: nothing for this warp
      if (ok) ok = mbar_wait(bar0 + 8 * st, ph, p.err, &abort_flag);
      if (ok) {
        const uint32_t row = codes_s + st * STAGE + mine;
        const uint32_t sc = sc_s + st * SC_STAGE + 2 * r8;
        uint32_t xk[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) xk[i] = xcol[i] + xc * W4_CHUNK;
        const uint32_t off = X.off + (xc * GPC * (NT * 8) + 2 * t) * 4;
        uint64_t part[H][NT][2];  // the chunk's sums, before the factor of x
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int i = 0; i < NT; ++i) part[h][i][0] = part[h][i][1] = 0;
#pragma unroll
        for (int gi = 0; gi < GPC; ++gi) {
          int sum[H][NT][4];
          uint32_t w[2 * H][WORDS];  // rows r8, r8 + 8, ...
          uint32_t b[NT][2 * WORDS];
#pragma unroll
          for (int q = 0; q < 2 * H; ++q) lds_words<WORDS>(w[q], (row ^ (gi * 16 * WORDS)) + q * 8 * 128);
#pragma unroll
          for (int i = 0; i < NT; ++i) lds_words<2 * WORDS>(b[i], xk[i] + gi * G);
#pragma unroll
          for (int j = 0; j < WORDS; ++j)
#pragma unroll
            for (int h = 0; h < H; ++h) {
              const uint32_t w0 = w[2 * h][j], w1 = w[2 * h + 1][j];
              const uint32_t a0 = w0 & 0x0F0F0F0Fu, a1 = w1 & 0x0F0F0F0Fu;
              const uint32_t a2 = (w0 >> 4) & 0x0F0F0F0Fu, a3 = (w1 >> 4) & 0x0F0F0F0Fu;
#pragma unroll
              for (int i = 0; i < NT; ++i) {
                int(&d)[4] = sum[h][i];
                if (j == 0) mma_16832(d, a0, a1, a2, a3, b[i][0], b[i][1], magic.x, magic.y, magic.z, magic.w);
                else mma_16832(d, a0, a1, a2, a3, b[i][2 * j], b[i][2 * j + 1], d[0], d[1], d[2], d[3]);
              }
            }
          float sc8[2 * H];  // scales of the rows
#pragma unroll
          for (int q = 0; q < 2 * H; ++q) sc8[q] = lds_bf16(sc + gi * (2 * ROWS) + 16 * q);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            const uint64_t o = lds_u64(off + (gi * (NT * 8) + 8 * i) * 4);
#pragma unroll
            for (int h = 0; h < H; ++h) {
#pragma unroll
              for (int e = 0; e < 2; ++e)
                part[h][i][e] = w4_fma2(w4_pack2(sc8[2 * h + e], sc8[2 * h + e]),
                                        w4_add2(w4_pack2(__int_as_float(sum[h][i][2 * e]),
                                                         __int_as_float(sum[h][i][2 * e + 1])), o),
                                        part[h][i][e]);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const uint64_t f = lds_u64(X.fac + (xc * (NT * 8) + 8 * i + 2 * t) * 4);
#pragma unroll
          for (int h = 0; h < H; ++h) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
              acc[h][i][e] = fmaf(w4_hi(f), w4_hi(part[h][i][e]), fmaf(w4_lo(f), w4_lo(part[h][i][e]), acc[h][i][e]));
          }
        }
        __syncwarp();
        if (lane == 0) load_next();  // into the stage just read
      }
      if (++st == L.stages) {
        st = 0;
        ph ^= 1u;
      }
    }
    if (any_far && (L.segs > 1 || round == 0)) {
      if (warp < rows) w4_sort_far(far, warp, lane);
      __syncthreads();
    }
    // the round's sums, RED rows of each warp at a time: the neighbouring lanes' halves of a row of x, then
    // over the KW warps
#pragma unroll
    for (int h0 = 0; h0 < H; h0 += RED / 16) {
      if (kw_n > 1) __syncthreads();  // the last ones are read
      else __syncwarp();
#pragma unroll
      for (int h = 0; h < RED / 16; ++h)
#pragma unroll
        for (int i = 0; i < NT; ++i) {  // even lanes finish row r8, odd ones r8 + 8
          const float a0 = acc[h0 + h][i][0], a1 = acc[h0 + h][i][1];
          const bool odd = t & 1;
          const float v = (odd ? a1 : a0) + __shfl_xor_sync(0xffffffffu, odd ? a0 : a1, 1);
          sts_f1(red + ((2 * i + (t >> 1)) * RED_LD + 16 * h + r8 + 8 * (t & 1)) * 4, v);
        }
      if (kw_n > 1) __syncthreads();
      else __syncwarp();
      auto finish = [&](int m, int from, int r) {  // row r of the block of the row warps' `from`
        const int n = ((round * rw_n + from) * gridDim.x + blockIdx.x) * ROWS + 16 * h0 + r;
        if (n >= p.N || !ok) return;
        float v = 0.f;
        if (any_far && far.n[m] > W4_FAR) {
          v = w4_plain_sum(p, L.x_vec, m0 + m, n);
        } else {
          const uint32_t at = red_base + ((from * XR + m) * RED_LD + r) * 4;
          for (int k = 0; k < kw_n && k < L.chunks; ++k)
            v += __uint_as_float(lds32(at + k * rw_n * XR * RED_LD * 4));
          if (any_far) v += w4_far_sum(p, far, m, n);
        }
        if (p.bias) v += p.bias[n];
        w4_store(p.out, p.out_f32, static_cast<size_t>(m0 + m) * p.out_stride + n, v);
      };
      // all warps finish the rows of a KW > 1 round, else each its own
      if (kw_n > 1) {
        for (int i = threadIdx.x; i < rw_n * RED * rows; i += THREADS) {
          const int q = i / RED, m = q / rw_n;
          finish(m, q - m * rw_n, i % RED);
        }
      } else {
        for (int i = lane; i < RED * rows; i += 32) finish(i / RED, rw, i % RED);
      }
    }
  }
  if (!ok) {  // copies in flight land before the CTA ends
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 200000ull) {
    }
  }
}

template <int NT, int G>
static cudaError_t linear_w4_launch(const W4Launch& L, const CUtensorMap& tc, const CUtensorMap& ts, size_t smem,
                                    dim3 grid, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};  // one bit per device: the kernel's shared-memory opt-in
  int dev = 0;
  cudaGetDevice(&dev);
  if (!((done >> dev) & 1u)) {
    const cudaError_t e =
        cudaFuncSetAttribute(linear_w4_kernel<NT, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, W4_SMEM_MAX - W4_STATIC);
    if (e != cudaSuccess) return e;
    done |= uint64_t(1) << dev;
  }
  linear_w4_kernel<NT, G><<<grid, 32 * w4_warps(NT), smem, s>>>(tc, ts, L);
  return cudaGetLastError();
}

cudaError_t launch_linear_w4(const W4Params& whole_p, cudaStream_t s) {
  W4Params p = whole_p;
  constexpr int MOST = W4_MAX_ROWS * 65535;  // a grid's second dimension of CTAs
  if (p.M > MOST) {  // the rows behind them by a launch of their own
    p.M -= MOST;
    p.x = static_cast<const uint8_t*>(p.x) + static_cast<size_t>(MOST) * p.K * (p.x_f32 ? 4 : 2);
    p.out = static_cast<uint8_t*>(p.out) + MOST * p.out_stride * (p.out_f32 ? 4 : 2);
    const cudaError_t e = launch_linear_w4(p, s);
    if (e != cudaSuccess) return e;
    p = whole_p;
    p.M = MOST;
  }
  static const int sms = device_sm_count();
  const int groups = (p.K + p.group - 1) / p.group;
  const int row_bytes = groups * (p.group / 2);
  W4Launch L;
  L.p = p;
  L.chunks = (row_bytes + W4_CHUNK / 2 - 1) / (W4_CHUNK / 2);
  L.x_vec = w4_vec(p.x, p.K);
  const int passes = (p.M + W4_MAX_ROWS - 1) / W4_MAX_ROWS;
  L.rows_m = (p.M + passes - 1) / passes;
  const int cols = W4_DIGITS * L.rows_m, nt = (cols + 7) / 8, warps = w4_warps(nt), rows = W4_ROWS;
  const int stage = warps * (rows * W4_CHUNK / 2 + rows * (W4_CHUNK / p.group) * 2);
  const int fixed = warps * nt * 8 / W4_DIGITS * w4_red_pitch(nt) * 4 + 1024 + W4_STATIC;  // sums, alignment, static
  // x lies in shared memory whole if two stages fit beside it, else in parts
  // of `seg` chunks, a multiple of the chunks that share a row; columns are
  // spaced so that the lanes of a bank cycle differ
  const int pad = p.group == 32 ? 32 : p.group == 64 ? 64 : 16;
  const int chunk_bytes = cols * W4_CHUNK + nt * 32 * (1 + W4_CHUNK / p.group);
  const int room = (W4_SMEM_MAX - fixed - 2 * stage - cols * pad) / chunk_bytes;  // chunks
  const bool whole = L.chunks <= room;
  const int per = passes < sms ? sms / passes : 1;  // CTAs per part of x's rows
  // the split with the least time on the busiest SM: rounds of row blocks, each
  // a chunk time per step, the round's bytes and a fixed end.  Against one warp
  // per row block (KW = 1): 18432 x 3072, two rows of x, 11.7 us and 18.5;
  // 3072 x 3072, one row, 4.8 and 16.3; 4099 x 2051, seven rows, 11.7 and 30.1; with
  // 743424 rows of weights both 198; with 120000 it is off by a little, 39.0 and 36.6.
  L.blocks = (p.N + rows - 1) / rows;
  float best = 0.f;
  L.rw = 0;
  for (int rw = warps; rw >= 1; --rw) {
    if (warps % rw) continue;
    const int kw = warps / rw;
    if (!whole && kw > room) break;
    const float cost = static_cast<float>((L.blocks + rw * per - 1) / (rw * per)) *
                       (0.5f * ((L.chunks + kw - 1) / kw) + 0.5f * rw * L.chunks / warps + 0.5f);
    if (L.rw == 0 || cost < best) {
      best = cost;
      L.rw = rw;
    }
  }
  if (L.rw == 0) return cudaErrorInvalidValue;
  const int kw = warps / L.rw;
  L.seg_chunks = whole ? L.chunks : room / kw * kw;
  L.segs = (L.chunks + L.seg_chunks - 1) / L.seg_chunks;
  L.x_pitch = L.seg_chunks * W4_CHUNK + pad;
  const int x_bytes = cols * pad + L.seg_chunks * chunk_bytes;
  const int left = W4_SMEM_MAX - fixed - x_bytes;
  L.stages = left / stage < W4_MAX_STAGES ? left / stage : W4_MAX_STAGES;
  const size_t smem = fixed - W4_STATIC + static_cast<size_t>(x_bytes) + static_cast<size_t>(L.stages) * stage;
  CUtensorMap tc, ts;
  if (!encode_tmap_2d(&tc, p.codes, row_bytes, p.N, row_bytes, W4_CHUNK / 2, rows, true) ||
      !encode_tmap_2d(&ts, p.scales, p.N, groups, static_cast<uint64_t>(p.scale_stride) * 2, rows,
                      W4_CHUNK / p.group, false, 0))
    return cudaErrorInvalidValue;
  const int need = (L.blocks + L.rw - 1) / L.rw;
  const dim3 grid(need < per ? need : per, passes);
#define AF_W4_CASE(NT_)                                                            \
  if (nt == NT_)                                                                   \
    return p.group == 32   ? linear_w4_launch<NT_, 32>(L, tc, ts, smem, grid, s)   \
           : p.group == 64 ? linear_w4_launch<NT_, 64>(L, tc, ts, smem, grid, s)   \
                           : linear_w4_launch<NT_, 128>(L, tc, ts, smem, grid, s);
  AF_W4_CASE(1)
  AF_W4_CASE(2)
  AF_W4_CASE(3)
  AF_W4_CASE(4)
#undef AF_W4_CASE
  return cudaErrorInvalidValue;
}

}  // namespace af
