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
// out[m, n] = bias[n] + sum_k f(x[m, k]) s[k / G, n] (c[n, k] - 8).
//
// Each group's sum of f(x) (c - 8) runs on mma.sync m16n8k16: the weights are
// the 16-row operand, as the whole numbers c - 8, exact in bf16; the columns
// are rows of x.  bf16 x is one column; fp32 x (and SiLU of either) is cut
// into three bf16 pieces of 8 bits each that add up to it exactly, three
// columns, so with the eight columns an instruction has anyway one or two
// fp32 rows cost what one bf16 row does.  Products are exact, sums fp32, and
// a group's sum is multiplied by its fp32 scale once.
//
// Bound: the code bytes from HBM (4.25 bits a weight at G = 64).  A 512-thread
// CTA per SM streams them with a TMA producer warp through a ring of 32 KB
// stages; 16 consumer warps are RW x KW: RW blocks of 16 rows by KW chunks of
// 256 columns (128 bytes of codes).  Rows of a stage are 128-byte lines under
// the 128-byte swizzle, so the fragment reads (lane (g, t): 4 bytes = 8 codes
// of row g, word t of a 16-byte piece) touch all 32 banks.  Of a word the
// codes p and p + 4 form one operand register; x lies in shared memory in
// that order (0, 4, 1, 5, 2, 6, 3, 7 of every eight).
constexpr int W4_WARPS = 16;
constexpr int W4_THREADS = 32 * (W4_WARPS + 1);
constexpr int W4_CHUNK = 256;                             // columns per chunk
constexpr int W4_STAGE = W4_WARPS * 16 * W4_CHUNK / 2;    // code bytes per stage
constexpr int W4_RED_LD = 20;                             // floats between columns of a warp's sums: no bank conflicts
constexpr int W4_MAX_NT = 4;                              // 8-column blocks
constexpr int W4_SMEM_MAX = 227 * 1024;
constexpr int W4_MAX_STAGES = 8;

struct W4Launch {
  W4Params p;
  int m0, rows_m, parts;    // this launch's rows of x and pieces (columns) of each
  int rw;                   // row blocks of 16 per CTA tile; W4_WARPS / rw chunks per stage
  int tiles, chunks, seg_chunks, segs, stages;
  int x_pitch;              // bytes between columns of x in shared memory
};

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ float lds_bf16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return w4_bf16(v);
}
// two codes of a word, c in the low and high half, as bf16 c - 8: 128 + c is
// the pattern 0x4300 | c, and the difference to 136 is exact
__device__ __forceinline__ uint32_t w4_pair(uint32_t w) {
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x000F000F, 0x43004300, 0xEA;" : "=r"(r) : "r"(w));  // (a & b) | c
  asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(r) : "r"(0x43084308u));
  return r;
}
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Columns [k0, k0 + n) of this launch's rows of x (zero behind column K) into
// shared memory.  A thread takes eight columns of a row: one 16-byte store
// per piece.  Each piece is the value's leading 8 bits, truncated; the last
// is what remains.  Infinities and NaN stay whole in the first piece.
__device__ __forceinline__ void w4_stage_x(const W4Launch& L, uint32_t xs, int k0, int n) {
  const W4Params& p = L.p;
  const int per = n / 8;
  for (int i = threadIdx.x; i < L.rows_m * per; i += 32 * W4_WARPS) {
    const int m = i / per, j = 8 * (i - m * per);
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int k = k0 + j + e;
      v[e] = k < p.K ? w4_load(p.x, p.x_f32, static_cast<size_t>(L.m0 + m) * p.K + k) : 0.f;
      if (p.silu) v[e] = w4_silu(v[e]);
    }
    const uint32_t dst = xs + m * L.parts * L.x_pitch + 2 * j;
    for (int part = 0; part < L.parts; ++part) {
      uint32_t h[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[e] = __float_as_uint(v[e]) & 0xFFFF0000u;
        const float hv = __uint_as_float(h[e]);
        if (L.parts > 1 && (h[e] & 0x7F800000u) == 0x7F800000u) {
          if (v[e] != v[e]) h[e] = 0x7FC00000u;  // a NaN may have its payload in the bits cut off
          v[e] = 0.f;
        } else {
          v[e] -= hv;
        }
      }
      sts128(dst + part * L.x_pitch, make_uint4((h[0] >> 16) | h[4], (h[1] >> 16) | h[5], (h[2] >> 16) | h[6],
                                                (h[3] >> 16) | h[7]));
    }
  }
}

template <int NT, int G>
__global__ void __launch_bounds__(W4_THREADS, 1)
    linear_w4_kernel(const __grid_constant__ CUtensorMap tm_codes, const __grid_constant__ CUtensorMap tm_scales,
                     const W4Launch L) {
  extern __shared__ uint8_t w4_raw[];
  __shared__ uint64_t full[W4_MAX_STAGES], empty[W4_MAX_STAGES];
  __shared__ int abort_flag;
  constexpr int GPC = W4_CHUNK / G;                    // groups per chunk
  constexpr int SC_STAGE = W4_WARPS * 16 * GPC * 2;    // scale bytes per stage
  const W4Params& p = L.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rw_n = L.rw, kw_n = W4_WARPS / rw_n;
  const uint32_t base = (smem_u32(w4_raw) + 1023u) & ~1023u;
  const uint32_t sc_base = base + L.stages * W4_STAGE;
  const uint32_t red_base = sc_base + L.stages * SC_STAGE;
  const uint32_t xs = red_base + W4_WARPS * NT * 8 * W4_RED_LD * 4;
  if (threadIdx.x == 0) {
    for (int i = 0; i < L.stages; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), W4_WARPS);
    }
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const int stages_per_tile = (L.chunks + kw_n - 1) / kw_n;

  if (warp == W4_WARPS) {  // producer: one thread streams the tiles' stages in order
    if (lane != 0) return;
    prefetch_tmap(&tm_codes);
    prefetch_tmap(&tm_scales);
    int st = 0;
    uint32_t ph = 0;
    for (int tile = blockIdx.x; tile < L.tiles; tile += gridDim.x) {
      const int n0 = tile * rw_n * 16;
      for (int s = 0; s < stages_per_tile; ++s) {
        if (!mbar_wait(smem_u32(&empty[st]), ph ^ 1u, p.err, &abort_flag)) {
          const uint64_t t0 = globaltimer();  // copies in flight land before the CTA ends
          while (globaltimer() - t0 < 200000ull) {
          }
          return;
        }
        const int nc = min(kw_n, L.chunks - s * kw_n);
        mbar_arrive_expect_tx(smem_u32(&full[st]), nc * rw_n * 2048 + SC_STAGE);
        for (int c = 0; c < nc; ++c)
          tma_load_2d(base + st * W4_STAGE + c * rw_n * 2048, &tm_codes, smem_u32(&full[st]),
                      (s * kw_n + c) * (W4_CHUNK / 2), n0);
        tma_load_2d(sc_base + st * SC_STAGE, &tm_scales, smem_u32(&full[st]), n0, s * kw_n * GPC);
        if (++st == L.stages) {
          st = 0;
          ph ^= 1u;
        }
      }
    }
    return;
  }

  auto consumers_sync = [] { asm volatile("bar.sync 1, %0;" ::"r"(32 * W4_WARPS) : "memory"); };
  const int rw = warp % rw_n, kw = warp / rw_n;
  const int g = lane >> 2, t = lane & 3;
  const int cols = L.rows_m * L.parts;
  uint32_t xcol[NT];  // this lane's column of each 8-column block; those past the last repeat it, unused
#pragma unroll
  for (int i = 0; i < NT; ++i) xcol[i] = xs + min(8 * i + g, cols - 1) * L.x_pitch + 16 * t;
  const uint32_t red = red_base + warp * NT * 8 * W4_RED_LD * 4;
  const int seg_k = L.seg_chunks * W4_CHUNK;
  bool ok = true;
  int st = 0;
  uint32_t ph = 0;
  if (L.segs == 1) {
    w4_stage_x(L, xs, 0, seg_k);
    consumers_sync();
  }
  for (int tile = blockIdx.x; tile < L.tiles; tile += gridDim.x) {
    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
    for (int s = 0; s < stages_per_tile; ++s) {
      const int chunk = s * kw_n + kw;
      if (L.segs > 1 && (s * kw_n) % L.seg_chunks == 0) {  // x no longer fits whole: its next part
        consumers_sync();
        w4_stage_x(L, xs, s * kw_n * W4_CHUNK, seg_k);
        consumers_sync();
      }
      if (ok) ok = mbar_wait(smem_u32(&full[st]), ph, p.err, &abort_flag);
      if (ok && chunk < L.chunks) {
        const uint32_t row = base + st * W4_STAGE + kw * rw_n * 2048 + (rw * 16 + g) * 128 + 4 * t;
        const uint32_t sc = sc_base + st * SC_STAGE + (kw * GPC * rw_n * 16 + rw * 16 + g) * 2;
        const uint32_t xk = (chunk % L.seg_chunks) * (W4_CHUNK * 2);
#pragma unroll
        for (int gi = 0; gi < GPC; ++gi) {
          float sum[NT][4];
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[i][e] = 0.f;
#pragma unroll
          for (int j = 0; j < G / 32; ++j) {
            const int c = gi * (G / 32) + j;  // 32 columns, a 16-byte piece of a row
            const uint32_t off = static_cast<uint32_t>(c ^ g) << 4;
            const uint32_t w0 = lds32(row + off), w1 = lds32(row + 8 * 128 + off);
            const uint32_t a0 = w4_pair(w0), a1 = w4_pair(w1), a2 = w4_pair(w0 >> 4), a3 = w4_pair(w1 >> 4);
            const uint32_t a4 = w4_pair(w0 >> 8), a5 = w4_pair(w1 >> 8), a6 = w4_pair(w0 >> 12),
                           a7 = w4_pair(w1 >> 12);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              const uint4 b = lds128(xcol[i] + xk + 64 * c);
              mma_16816(sum[i], a0, a1, a2, a3, b.x, b.y);
              mma_16816(sum[i], a4, a5, a6, a7, b.z, b.w);
            }
          }
          const float s0 = lds_bf16(sc + gi * rw_n * 32), s1 = lds_bf16(sc + gi * rw_n * 32 + 16);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            acc[i][0] += s0 * sum[i][0];
            acc[i][1] += s0 * sum[i][1];
            acc[i][2] += s1 * sum[i][2];
            acc[i][3] += s1 * sum[i][3];
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&empty[st]));
      if (++st == L.stages) {
        st = 0;
        ph ^= 1u;
      }
    }
    // the tile's sums: columns of 16 rows per warp, then over the KW warps and the pieces of each row of x
    if (kw_n > 1) consumers_sync();  // the last tile's are read
    else __syncwarp();
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const uint32_t a = red + ((8 * i + 2 * t) * W4_RED_LD + g) * 4;
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(acc[i][0]) : "memory");
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(a + W4_RED_LD * 4), "f"(acc[i][1]) : "memory");
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(a + 32), "f"(acc[i][2]) : "memory");
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(a + W4_RED_LD * 4 + 32), "f"(acc[i][3]) : "memory");
    }
    if (kw_n > 1) consumers_sync();
    else __syncwarp();
    // rows of the tile this warp finishes: all warps share a KW > 1 tile's, else each its own 16
    const int span = kw_n > 1 ? rw_n * 16 : 16;
    const int first = kw_n > 1 ? threadIdx.x : lane, step = kw_n > 1 ? 32 * W4_WARPS : 32;
    for (int i = first; i < span * L.rows_m; i += step) {
      const int m = i / span, r = i - m * span + (kw_n > 1 ? 0 : rw * 16);
      const int n = tile * rw_n * 16 + r;
      if (n >= p.N || !ok) continue;
      float v = 0.f;
      for (int part = 0; part < L.parts; ++part)
        for (int k = 0; k < kw_n; ++k)
          v += __uint_as_float(lds32(red_base + (((k * rw_n + r / 16) * NT * 8 + m * L.parts + part) * W4_RED_LD +
                                                 r % 16) * 4));
      if (p.bias) v += p.bias[n];
      w4_store(p.out, p.out_f32, static_cast<size_t>(L.m0 + m) * p.out_stride + n, v);
    }
  }
}

template <int NT, int G>
static cudaError_t linear_w4_launch(const W4Launch& L, const CUtensorMap& tc, const CUtensorMap& ts, size_t smem,
                                    int grid, cudaStream_t s) {
  static uint64_t done = 0;  // one bit per device: the kernel's shared-memory opt-in
  int dev = 0;
  cudaGetDevice(&dev);
  if (!((done >> dev) & 1u)) {
    const cudaError_t e =
        cudaFuncSetAttribute(linear_w4_kernel<NT, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, W4_SMEM_MAX - 1024);
    if (e != cudaSuccess) return e;
    done |= uint64_t(1) << dev;
  }
  linear_w4_kernel<NT, G><<<grid, W4_THREADS, smem, s>>>(tc, ts, L);
  return cudaGetLastError();
}

cudaError_t launch_linear_w4(const W4Params& p, cudaStream_t s) {
  static int sms = 0;
  if (!sms) sms = device_sm_count();
  const int groups = (p.K + p.group - 1) / p.group;
  const int row_bytes = groups * (p.group / 2);
  W4Launch L;
  L.p = p;
  L.chunks = (row_bytes + W4_CHUNK / 2 - 1) / (W4_CHUNK / 2);
  L.parts = p.x_f32 || p.silu ? 3 : 1;
  const int most = W4_MAX_NT * 8 / L.parts;
  const int passes = (p.M + most - 1) / most, per_pass = (p.M + passes - 1) / passes;
  const int stage = W4_STAGE + W4_WARPS * 16 * (W4_CHUNK / p.group) * 2;
  for (L.m0 = 0; L.m0 < p.M; L.m0 += per_pass) {
    L.rows_m = p.M - L.m0 < per_pass ? p.M - L.m0 : per_pass;
    const int cols = L.rows_m * L.parts, nt = (cols + 7) / 8;
    const int fixed = W4_WARPS * nt * 8 * W4_RED_LD * 4 + 2048;  // sums, alignment, static barriers
    // x lies in shared memory whole if three stages fit beside it, else in
    // parts of `seg` chunks, a multiple of the chunks of a stage
    const int room = (W4_SMEM_MAX - fixed - 3 * stage) / cols - 64;  // bytes per column
    const bool whole = L.chunks * W4_CHUNK * 2 <= room;
    // the split with the least time on the busiest SM: rounds of tiles, each a
    // chunk time per stage, the tile's bytes and a fixed end
    float best = 0.f;
    L.rw = 0;
    for (int rw = W4_WARPS; rw >= 1; rw /= 2) {
      const int tiles = (p.N + rw * 16 - 1) / (rw * 16), kw = W4_WARPS / rw;
      if (!whole && kw * W4_CHUNK * 2 > room) break;
      const float cost = static_cast<float>((tiles + sms - 1) / sms) *
                         (0.5f * ((L.chunks + kw - 1) / kw) + 0.5f * rw * L.chunks / W4_WARPS + 0.5f);
      if (L.rw == 0 || cost < best) {
        best = cost;
        L.rw = rw;
        L.tiles = tiles;
      }
    }
    if (L.rw == 0) return cudaErrorInvalidValue;
    const int kw = W4_WARPS / L.rw;
    L.seg_chunks = whole ? L.chunks : room / (W4_CHUNK * 2) / kw * kw;
    L.segs = (L.chunks + L.seg_chunks - 1) / L.seg_chunks;
    L.x_pitch = L.seg_chunks * W4_CHUNK * 2 + 64;
    const int left = W4_SMEM_MAX - fixed - cols * L.x_pitch;
    L.stages = left / stage < W4_MAX_STAGES ? left / stage : W4_MAX_STAGES;
    const size_t smem = fixed - 1024 + static_cast<size_t>(cols) * L.x_pitch + static_cast<size_t>(L.stages) * stage;
    CUtensorMap tc, ts;
    if (!encode_tmap_2d(&tc, p.codes, row_bytes, p.N, row_bytes, W4_CHUNK / 2, L.rw * 16, true) ||
        !encode_tmap_2d(&ts, p.scales, p.N, groups, static_cast<uint64_t>(p.scale_stride) * 2, L.rw * 16,
                        kw * (W4_CHUNK / p.group), false, 0))
      return cudaErrorInvalidValue;
    const int grid = L.tiles < sms ? L.tiles : sms;
    cudaError_t e = cudaErrorInvalidValue;
#define AF_W4_CASE(NT_)                                                                     \
  if (nt == NT_) {                                                                          \
    e = p.group == 32   ? linear_w4_launch<NT_, 32>(L, tc, ts, smem, grid, s)               \
        : p.group == 64 ? linear_w4_launch<NT_, 64>(L, tc, ts, smem, grid, s)               \
                        : linear_w4_launch<NT_, 128>(L, tc, ts, smem, grid, s);             \
  }
    AF_W4_CASE(1)
    AF_W4_CASE(2)
    AF_W4_CASE(3)
    AF_W4_CASE(4)
#undef AF_W4_CASE
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace af
