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
#include <atomic>

#include "af_internal.h"
#include "ptx.cuh"

namespace af {

namespace {

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

// ------------------------------------------------------------------ any width and alignment
// TG threads per row, E columns a thread in registers, one load or store per
// value.  Up to 128 columns TG is a power of two within a warp, the columns TG
// apart, and a CTA takes 256 / TG rows; wider rows take whole warps, each E times
// 32 neighbouring columns (constant offsets), and above a warp a CTA each.
// Bound: the loads and stores of single values (two 4360 x 3072 bf16 samples off
// 16-byte boundaries 103 us, 42 on them).  With 16 columns a thread, rows above
// 8192 columns, registers do not hold them all: 340 to 948 bytes a thread go to
// local memory; 2400 rows of 9001 columns take 82 us in bf16 and 135 in fp32,
// where HBM would allow 26 and 53.
constexpr int RN_THREADS = 256;

template <typename T, bool OUT8, int E, bool WIDE>
__global__ void __launch_bounds__(1024)
    residual_norm_any_kernel(const __grid_constant__ ResidualNormParams p, int tg) {
  __shared__ float red[2][32];
  const int tid = tg > 32 ? threadIdx.x : threadIdx.x & (tg - 1), D = p.D;
  const int c0 = WIDE ? (tid >> 5) * (32 * E) + (tid & 31) : tid, step = WIDE ? 32 : tg;
  const int64_t rows = static_cast<int64_t>(p.B) * p.rows_per_batch;
  const int64_t r = tg > 32 ? blockIdx.x : (static_cast<int64_t>(blockIdx.x) * RN_THREADS + threadIdx.x) / tg;
  const bool live = r < rows;
  const size_t base = static_cast<size_t>(live ? r : rows - 1) * D;  // lanes behind the last row repeat it
  const size_t mo = static_cast<size_t>((live ? r : rows - 1) / p.rows_per_batch) * p.mod_stride;
  const float inv_d = 1.0f / static_cast<float>(D);
  int buf = 0;
  auto join = [&](float v, bool max) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (o < tg) {
        const float t = __shfl_xor_sync(0xffffffffu, v, o);
        v = max ? fmaxf(v, t) : v + t;
      }
    if (tg <= 32) return v;
    float* w = red[buf];  // two buffers in turn: one barrier per sum
    buf ^= 1;
    if ((threadIdx.x & 31) == 0) w[threadIdx.x >> 5] = v;
    __syncthreads();
    v = w[0];
    for (int i = 1; i < tg >> 5; ++i) v = max ? fmaxf(v, w[i]) : v + w[i];
    return v;
  };
  auto normalise = [&](float (&v)[E], int kind) {
    if (kind == NORM_NONE) return;
    float mean = 0.f, q = 0.f;
    if (kind == NORM_LAYER) {
#pragma unroll
      for (int i = 0; i < E; ++i) mean += v[i];  // zero behind D
      mean = join(mean, false) * inv_d;
    }
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (c0 + i * step < D) {
        v[i] -= mean;
        q += v[i] * v[i];
      }
    const float f = rsqrtf(join(q, false) * inv_d + p.eps);
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] *= f;
  };
  // everything the row needs is asked for at once, before any of it is used
  auto load = [&](const float* f, size_t at, float none, float (&v)[E]) {
    if (f) {
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = c0 + i * step < D ? __ldg(f + at + c0 + i * step) : none;
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = none;
    }
  };
  auto load_row = [&](const void* t, float (&v)[E]) {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = c0 + i * step < D ? rn_load<T>(t, base + c0 + i * step) : 0.f;
  };
  float x[E], u[E], fg[E], fa[E], fs[E];
  load_row(p.x, x);
  if (p.branch) load_row(p.branch, u);
  load(p.gate, mo, 1.f, fg);
  load(p.scale, mo, 0.f, fa);
  load(p.shift, mo, 0.f, fs);
  if (p.post_weight) {
    float w[E];
    load(p.post_weight, 0, 0.f, w);
#pragma unroll
    for (int i = 0; i < E; ++i) fg[i] *= w[i];
  }
#pragma unroll
  for (int i = 0; i < E; ++i) fa[i] += 1.f;
  if (p.pre_weight) {
    float w[E];
    load(p.pre_weight, 0, 0.f, w);
#pragma unroll
    for (int i = 0; i < E; ++i) fa[i] *= w[i];
  }
  if (p.branch) {
    normalise(u, p.post);
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] += p.residual_scale * fg[i] * u[i];
  }
  if (p.x_out && live) {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (c0 + i * step < D) rn_store<T>(p.x_out, base + c0 + i * step, x[i]);
  }
  if (!p.y) return;
  normalise(x, p.pre);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int d = c0 + i * step;
    if (d >= D) continue;
    x[i] = x[i] * fa[i] + fs[i];
    if constexpr (OUT8) amax = fmaxf(amax, fabsf(x[i]));
    else if (live) rn_store<T>(p.y, base + d, x[i]);
  }
  if constexpr (OUT8) {
    amax = join(amax, true);
    const float inv = amax > 0.f ? 448.0f / amax : 1.0f;
    if (!live) return;
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (c0 + i * step < D)
        static_cast<uint8_t*>(p.y)[base + c0 + i * step] = static_cast<uint8_t>(pack_e4m3x4(x[i] * inv, 0.f, 0.f, 0.f));
    if (tid == 0) p.yscale[r] = amax > 0.f ? amax / 448.0f : 1.0f;
  }
}

// ------------------------------------------------------------------ rows in registers
// Widths that are multiples of 8 with 16-byte aligned tensors: TG threads per
// row, a thread holding V vectors of eight neighbouring columns in registers
// from the load to the stores, so HBM sees each tensor once.  A CTA stays
// within one sample, whose factors
//   r gate post_weight,   pre_weight (1 + scale),   shift
// it keeps in shared memory (from the tensors each time they would take three
// times the row's own bytes); a CTA with one round of rows reads them directly.
// Bound: HBM with many rows (three reads and writes of 2 or 4 bytes a value), the
// launch and one chain of loads and joins with few.
// RING (many rows with a norm of the branch, whole warps per row): rows stream through a ring of the row
// group in shared memory, bulk copies issued by its first thread as soon as
// the group has a row in registers; at 3072 columns seven groups keep two rows
// each, 168 KB, in flight.
// Registers: bf16 fits up to 16 bytes a thread in local memory (the ring, 80 of
// them); fp32 at three and four vectors has 104 to 220 bytes there.
// Statistics are two-pass; sums are joined by shuffles and, for rows wider
// than a warp, through shared memory at the row group's named barrier, two
// buffers in turn so that one barrier per sum is enough.  Packed fp32 pairs.
__device__ __forceinline__ uint64_t rn_pack(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 rn_unpack(uint64_t r) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(r));
  return v;
}
__device__ __forceinline__ uint64_t rn_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t rn_add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t rn_mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Eight columns as stored.
template <typename T>
struct RnRaw {
  uint4 q[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ RnRaw<T> rn_load8(const void* p, size_t i) {
  RnRaw<T> r;
  const uint4* s = reinterpret_cast<const uint4*>(static_cast<const T*>(p) + i);
#pragma unroll
  for (int e = 0; e < static_cast<int>(sizeof(T) / 2); ++e) r.q[e] = s[e];
  return r;
}
// The same for the columns before `end`, zero behind it.
template <typename T>
__device__ __forceinline__ RnRaw<T> rn_load_some(const void* p, int64_t i, int64_t end) {
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (sizeof(T) == 4) w[e] = i + e < end ? static_cast<const uint32_t*>(p)[i + e] : 0u;
    else w[e] = i + e < end ? static_cast<const uint16_t*>(p)[i + e] : 0u;
  }
  RnRaw<T> r;
  if constexpr (sizeof(T) == 4) {
    r.q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    r.q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
    r.q[0] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void rn_expand(const RnRaw<T>& r, uint64_t (&v)[4]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      v[2 * e] = rn_pack(__uint_as_float(r.q[e].x), __uint_as_float(r.q[e].y));
      v[2 * e + 1] = rn_pack(__uint_as_float(r.q[e].z), __uint_as_float(r.q[e].w));
    }
  } else {
    const uint32_t w[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = rn_pack(bf16_lo(w[e]), bf16_hi(w[e]));
  }
}
template <typename T>
__device__ __forceinline__ void rn_store8(void* p, size_t i, const uint64_t (&v)[4]) {
  uint4* d = reinterpret_cast<uint4*>(static_cast<T*>(p) + i);
  float2 f[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = rn_unpack(v[e]);
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      d[e] = make_uint4(__float_as_uint(f[2 * e].x), __float_as_uint(f[2 * e].y), __float_as_uint(f[2 * e + 1].x),
                        __float_as_uint(f[2 * e + 1].y));
  } else {
    d[0] = make_uint4(pack_bf16(f[0].x, f[0].y), pack_bf16(f[1].x, f[1].y), pack_bf16(f[2].x, f[2].y),
                      pack_bf16(f[3].x, f[3].y));
  }
}

struct RnPlan {
  int tg, groups;  // threads per row (a power of two below 32, or whole warps), rows of a CTA at a time
  int per;         // CTAs per sample
  int staged;      // factors in shared memory
  int fvec;        // their tensors in 16-byte loads
  int stages;      // RING: rows in flight per row group
};
// Floats of a plane of the shifted kernel's factors: an entry before and one
// behind the columns, and 4 mod 32 so that eight planes fill the banks.
__host__ __device__ constexpr int rn_plane(int D) { return ((D + 7) / 8 + 2 + 27) / 32 * 32 + 4; }
constexpr int RN_SMEM_MAX = 222 * 1024;  // beside the static barriers and sums
constexpr int RN_RING_THREADS = 672;  // 21 warps of 80 registers
constexpr int RN_MAX_GROUPS = 21, RN_MAX_STAGES = 8;

// EXACT: the row is exactly TG threads of V vectors, TG whole warps.
template <typename T, bool OUT8, int V, bool EXACT, bool RING>
__global__ void __launch_bounds__(RING ? RN_RING_THREADS : 512, V == 1 ? 2 : 1)
    residual_norm_kernel(const __grid_constant__ ResidualNormParams p, const RnPlan plan) {
  // [3][2][D / 2]: of every eight columns the first four, then the last four, so
  // that neighbouring lanes read neighbouring 16 bytes
  extern __shared__ __align__(16) float factors[];
  __shared__ float red[15][2][16];  // [row group][buffer][warp]
  __shared__ uint64_t full[RING ? RN_MAX_GROUPS : 1][RN_MAX_STAGES];
  __shared__ int abort_flag;
  const int tg = plan.tg, warps = tg >> 5;
  const int grp = threadIdx.x / tg, tid = threadIdx.x - grp * tg;
  const int lane = threadIdx.x & 31, warp = tid >> 5;
  const int b = blockIdx.x / plan.per, cta = blockIdx.x - b * plan.per;
  const int D = p.D;
  // a warp's vectors are neighbours, 256 columns apart: constant offsets
  const int c0 = EXACT || warps ? 8 * (warp * (32 * V) + lane) : 8 * tid;
  const size_t sample = static_cast<size_t>(b) * p.rows_per_batch;
  const size_t mo = static_cast<size_t>(b) * p.mod_stride;
  auto gate_of = [&](int d) {
    float f = p.residual_scale;
    if (p.gate) f *= __ldg(p.gate + mo + d);
    if (p.post_weight) f *= __ldg(p.post_weight + d);
    return f;
  };
  auto mul_of = [&](int d) {
    float f = 1.f;
    if (p.scale) f += __ldg(p.scale + mo + d);
    if (p.pre_weight) f *= __ldg(p.pre_weight + d);
    return f;
  };
  auto add_of = [&](int d) { return p.shift ? __ldg(p.shift + mo + d) : 0.f; };
  // eight columns of the factors from column c
  auto eight = [&](int which, int c, uint64_t (&f)[4]) {
    if (RING || plan.staged) {  // a ring has more rows than CTAs
      const float4 lo = *reinterpret_cast<const float4*>(factors + which * D + c / 2);
      const float4 hi = *reinterpret_cast<const float4*>(factors + which * D + D / 2 + c / 2);
      f[0] = rn_pack(lo.x, lo.y);
      f[1] = rn_pack(lo.z, lo.w);
      f[2] = rn_pack(hi.x, hi.y);
      f[3] = rn_pack(hi.z, hi.w);
    } else if (plan.fvec) {
      // eight columns of a vector as packed pairs, or `none` of them
      auto pairs = [&](const float* v, size_t at, float none, uint64_t (&o)[4]) {
        float4 lo = make_float4(none, none, none, none), hi = lo;
        if (v) {
          lo = __ldg(reinterpret_cast<const float4*>(v + at + c));
          hi = __ldg(reinterpret_cast<const float4*>(v + at + c + 4));
        }
        o[0] = rn_pack(lo.x, lo.y);
        o[1] = rn_pack(lo.z, lo.w);
        o[2] = rn_pack(hi.x, hi.y);
        o[3] = rn_pack(hi.z, hi.w);
      };
      uint64_t w[4];
      if (which == 0) {
        pairs(p.gate, mo, 1.f, f);
        pairs(p.post_weight, 0, 1.f, w);
        const uint64_t r2 = rn_pack(p.residual_scale, p.residual_scale);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = rn_mul2(rn_mul2(r2, f[e]), w[e]);
      } else if (which == 1) {
        pairs(p.scale, mo, 0.f, f);
        pairs(p.pre_weight, 0, 1.f, w);
        const uint64_t one = rn_pack(1.f, 1.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = rn_mul2(rn_add2(one, f[e]), w[e]);
      } else {
        pairs(p.shift, mo, 0.f, f);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = c + 2 * e;
        f[e] = which == 0   ? rn_pack(gate_of(d), gate_of(d + 1))
               : which == 1 ? rn_pack(mul_of(d), mul_of(d + 1))
                            : rn_pack(add_of(d), add_of(d + 1));
      }
    }
  };
  int buf = 0;
  auto join = [&](float s, bool max) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (!EXACT && warps == 0 && o >= tg) continue;
      const float t = __shfl_xor_sync(0xffffffffu, s, o);
      s = max ? fmaxf(s, t) : s + t;
    }
    if (warps <= 1) return s;
    float* r = red[grp][buf];
    buf ^= 1;
    if (lane == 0) r[warp] = s;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "r"(tg) : "memory");
    s = r[0];
    for (int i = 1; i < warps; ++i) s = max ? fmaxf(s, r[i]) : s + r[i];
    return s;
  };
  const float inv_d = 1.0f / static_cast<float>(D);
  // the mean to take off and the factor of a norm of the V x 8 values that get(i, v) yields
  auto stats = [&](auto get, const bool (&on)[V], int kind, uint64_t& m2, uint64_t& r2) {
    m2 = 0;
    r2 = rn_pack(1.f, 1.f);
    if (kind == NORM_NONE) return;
    if (kind == NORM_LAYER) {
      uint64_t s = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        uint64_t v[4];
        get(i, v);  // zero behind D
#pragma unroll
        for (int e = 0; e < 4; ++e) s = rn_add2(s, v[e]);
      }
      const float2 f = rn_unpack(s);
      const float mean = join(f.x + f.y, false) * inv_d;
      m2 = rn_pack(-mean, -mean);
    }
    uint64_t q = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      uint64_t v[4];
      get(i, v);
      if (on[i]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint64_t c = rn_add2(v[e], m2);
          q = rn_fma2(c, c, q);
        }
      }
    }
    const float2 f = rn_unpack(q);
    const float r = rsqrtf(join(f.x + f.y, false) * inv_d + p.eps);
    r2 = rn_pack(r, r);
  };

  RnRaw<T> xq[V], bq[V];
  auto fetch = [&](int r) {
    if (EXACT && r >= p.rows_per_batch) return;
    const size_t at = (sample + r) * D + c0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (!EXACT) {
        xq[i] = RnRaw<T>{};
        bq[i] = RnRaw<T>{};
        if (r >= p.rows_per_batch || c0 + 256 * i >= D) continue;
      }
      xq[i] = rn_load8<T>(p.x, at + 256 * i);
      if (p.branch) bq[i] = rn_load8<T>(p.branch, at + 256 * i);
    }
  };
  const int step = plan.per * plan.groups;
  int r = cta + plan.per * grp;  // rows dealt to the CTAs in turn: their counts differ by one at most
  const uint32_t row_bytes = D * sizeof(T), stage_bytes = p.branch ? 2 * row_bytes : row_bytes;
  uint32_t ring = 0;  // this group's stages, behind the factors
  auto copy_row = [&](int r, int st) {
    const uint32_t bar = smem_u32(&full[grp][st]), dst = ring + st * stage_bytes;
    const size_t at = (sample + r) * D;
    mbar_arrive_expect_tx(bar, stage_bytes);
    bulk_load(dst, static_cast<const T*>(p.x) + at, row_bytes, bar);
    if (p.branch) bulk_load(dst + row_bytes, static_cast<const T*>(p.branch) + at, row_bytes, bar);
  };
  if constexpr (RING) {
    ring = smem_u32(factors) + D * 12 + grp * plan.stages * stage_bytes;
    if (threadIdx.x == 0) abort_flag = 0;
    if (tid == 0) {
      for (int i = 0; i < plan.stages; ++i) mbar_init(smem_u32(&full[grp][i]), 1);
      fence_mbar_init();
      for (int i = 0; i < plan.stages && r + i * step < p.rows_per_batch; ++i) copy_row(r + i * step, i);
    }
  } else {
    fetch(r);
  }
  if (RING || plan.staged) {
    for (int d = 4 * threadIdx.x; d < D; d += 4 * blockDim.x) {  // four columns: their loads overlap
      const int at = (d & 4 ? D / 2 : 0) + (d >> 3) * 4;
      float f[3][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[0][e] = gate_of(d + e);
        f[1][e] = mul_of(d + e);
        f[2][e] = add_of(d + e);
      }
#pragma unroll
      for (int w = 0; w < 3; ++w)
        *reinterpret_cast<float4*>(factors + w * D + at) = make_float4(f[w][0], f[w][1], f[w][2], f[w][3]);
    }
  }
  if (RING || plan.staged) __syncthreads();
  // a warp's row groups go round together: first row of the warp's
  const int ahead = warps ? 0 : lane / tg * plan.per;
  int st = 0;
  uint32_t ph = 0;
  for (; r - ahead < p.rows_per_batch; r += step) {
    if constexpr (RING) {
      const bool got = mbar_wait(smem_u32(&full[grp][st]), ph, nullptr, &abort_flag);
      const uint32_t src = ring + st * stage_bytes + c0 * sizeof(T);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const bool in = EXACT || c0 + 256 * i < D;
#pragma unroll
        for (int e = 0; e < static_cast<int>(sizeof(T) / 2); ++e) {
          const uint32_t o = 256 * i * sizeof(T) + 16 * e;
          xq[i].q[e] = in ? lds128(src + o) : make_uint4(0, 0, 0, 0);
          bq[i].q[e] = in && p.branch ? lds128(src + row_bytes + o) : make_uint4(0, 0, 0, 0);
        }
      }
      // the whole group has the row (or has given up): the stage is free
      uint32_t failed;
      if (warps == 1) {
        failed = __any_sync(0xffffffffu, !got);
        __syncwarp();  // the vote alone does not order the lanes' reads before the next copy
      } else {
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.u32 p, %1, 0;\n\t"
            "bar.red.or.pred q, %2, %3, p;\n\t"
            "selp.u32 %0, 1, 0, q;\n\t}"
            : "=r"(failed)
            : "r"(static_cast<uint32_t>(!got)), "r"(1 + grp), "r"(tg)
            : "memory");
      }
      if (failed) {  // copies in flight land before the CTA ends
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 200000ull) {
        }
        return;
      }
      if (tid == 0 && r + plan.stages * step < p.rows_per_batch) copy_row(r + plan.stages * step, st);
      if (++st == plan.stages) {
        st = 0;
        ph ^= 1u;
      }
    }
    const bool live = r < p.rows_per_batch;
    bool on[V];
#pragma unroll
    for (int i = 0; i < V; ++i) on[i] = EXACT || (live && c0 + 256 * i < D);
    uint64_t x[V][4], m2, r2;
    if (p.branch) {
      stats([&](int i, uint64_t (&v)[4]) { rn_expand<T>(bq[i], v); }, on, p.post, m2, r2);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        uint64_t u[4], f[4] = {0, 0, 0, 0};
        rn_expand<T>(xq[i], x[i]);
        rn_expand<T>(bq[i], u);
        if (on[i]) {
          eight(0, c0 + 256 * i, f);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (p.post != NORM_NONE) u[e] = rn_mul2(rn_add2(u[e], m2), r2);
            x[i][e] = rn_fma2(f[e], u[e], x[i][e]);
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) rn_expand<T>(xq[i], x[i]);
    }
    if constexpr (!RING) fetch(r + step);
    const size_t base = (sample + r) * D + c0;
    if (p.x_out) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (on[i]) rn_store8<T>(p.x_out, base + 256 * i, x[i]);
    }
    if (!p.y) continue;
    stats([&](int i, uint64_t (&v)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = x[i][e];
    }, on, p.pre, m2, r2);
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!on[i]) continue;
      uint64_t fa[4], fs[4];
      eight(1, c0 + 256 * i, fa);
      eight(2, c0 + 256 * i, fs);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[i][e] = rn_fma2(rn_mul2(rn_add2(x[i][e], m2), r2), fa[e], fs[e]);
        if constexpr (OUT8) {
          const float2 f = rn_unpack(x[i][e]);
          amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      if constexpr (!OUT8) rn_store8<T>(p.y, base + 256 * i, x[i]);
    }
    if constexpr (OUT8) {
      amax = join(amax, true);
      const float inv = amax > 0.f ? 448.0f / amax : 1.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (!on[i]) continue;
        float2 f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = rn_unpack(x[i][e]);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.y) + base + 256 * i) =
            make_uint2(pack_e4m3x4(f[0].x * inv, f[0].y * inv, f[1].x * inv, f[1].y * inv),
                       pack_e4m3x4(f[2].x * inv, f[2].y * inv, f[3].x * inv, f[3].y * inv));
      }
      if (tid == 0 && live) p.yscale[sample + r] = amax > 0.f ? amax / 448.0f : 1.0f;
    }
  }
}

// ------------------------------------------------------------------ many rows of any width
// Widths that are not multiples of 8: a row starts anywhere in a 16-byte
// vector, so threads hold the aligned vectors that the row touches.  Element e
// of vector g is column 8 g + e - off, off = the row's first element mod 8; in
// the first and the last vector some of the eight belong to the neighbouring
// rows: they are read with the rest, taken as zero, and not written.  Factors
// lie in shared memory in eight planes by column mod 8, where the lanes' columns
// 8 apart are neighbours whatever off is.
// Bound: instructions, the 24 factors of a vector read one by one and the masks:
// two 4360 x 3001 bf16 samples 57 us (32 at HBM's rate).  In fp32 four vectors a
// thread do not fit the registers: 684 to 804 bytes go to local memory.
template <typename T, bool OUT8, int V>
__global__ void __launch_bounds__(512, 1)
    residual_norm_shift_kernel(const __grid_constant__ ResidualNormParams p, const RnPlan plan) {
  extern __shared__ __align__(16) float factors[];  // [3][8][plane]
  __shared__ float red[15][2][16];
  const int tg = plan.tg, warps = tg >> 5, D = p.D;
  const int plane = rn_plane(D);
  const int grp = threadIdx.x / tg, tid = threadIdx.x - grp * tg;
  const int lane = threadIdx.x & 31, warp = tid >> 5;
  const int b = blockIdx.x / plan.per, cta = blockIdx.x - b * plan.per;
  const int g0 = warps ? warp * (32 * V) + lane : tid;  // this thread's vectors: g0 + 32 i
  const int64_t sample = static_cast<int64_t>(b) * p.rows_per_batch;
  const int64_t total = static_cast<int64_t>(p.B) * p.rows_per_batch * D;
  const size_t mo = static_cast<size_t>(b) * p.mod_stride;
  for (int d = threadIdx.x; d < D; d += blockDim.x) {
    float f = p.residual_scale, m = 1.f;
    if (p.gate) f *= __ldg(p.gate + mo + d);
    if (p.post_weight) f *= __ldg(p.post_weight + d);
    if (p.scale) m += __ldg(p.scale + mo + d);
    if (p.pre_weight) m *= __ldg(p.pre_weight + d);
    float* at = factors + (d & 7) * plane + (d >> 3) + 1;
    at[0] = f;
    at[8 * plane] = m;
    at[16 * plane] = p.shift ? __ldg(p.shift + mo + d) : 0.f;
  }
  __syncthreads();
  int buf = 0;
  auto join = [&](float s, bool max) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (warps == 0 && o >= tg) continue;
      const float t = __shfl_xor_sync(0xffffffffu, s, o);
      s = max ? fmaxf(s, t) : s + t;
    }
    if (warps <= 1) return s;
    float* r = red[grp][buf];
    buf ^= 1;
    if (lane == 0) r[warp] = s;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "r"(tg) : "memory");
    s = r[0];
    for (int i = 1; i < warps; ++i) s = max ? fmaxf(s, r[i]) : s + r[i];
    return s;
  };
  auto off_of = [&](int r) { return static_cast<int>((((sample + r) & 7) * (D & 7)) & 7); };
  RnRaw<T> xq[V], bq[V];
  auto fetch = [&](int r) {
    if (r >= p.rows_per_batch) return;
    const int off = off_of(r);
    const int64_t first = (sample + r) * D - off;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int g = g0 + 32 * i;
      const int64_t at = first + 8 * g;
      xq[i] = RnRaw<T>{};
      bq[i] = RnRaw<T>{};
      if (8 * g >= off + D) continue;
      if (at + 8 <= total) {
        xq[i] = rn_load8<T>(p.x, at);
        if (p.branch) bq[i] = rn_load8<T>(p.branch, at);
      } else {  // the tensors end inside the vector
        xq[i] = rn_load_some<T>(p.x, at, total);
        if (p.branch) bq[i] = rn_load_some<T>(p.branch, at, total);
      }
    }
  };
  const float inv_d = 1.0f / static_cast<float>(D);
  const int step = plan.per * plan.groups;
  int r = cta + plan.per * grp;
  const int ahead = warps ? 0 : lane / tg * plan.per;
  fetch(r);
  for (; r - ahead < p.rows_per_batch; r += step) {
    const bool live = r < p.rows_per_batch;
    const int off = live ? off_of(r) : 0;
    const int64_t first = (sample + r) * D - off;
    uint32_t mask[V];  // which of the eight are the row's
    float x[V][8], u[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int g = g0 + 32 * i, end = off + D - 8 * g;
      mask[i] = !live || end <= 0 ? 0u : (0xFFu << (g == 0 ? off : 0)) & (end >= 8 ? 0xFFu : (1u << end) - 1u);
      uint64_t v[4];
      auto put = [&](const RnRaw<T>& q, float (&o)[8]) {
        rn_expand<T>(q, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = rn_unpack(v[e]);
          o[2 * e] = f.x;
          o[2 * e + 1] = f.y;
        }
        if (mask[i] != 0xFFu) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (!((mask[i] >> e) & 1u)) o[e] = 0.f;
        }
      };
      put(xq[i], x[i]);
      put(bq[i], u[i]);
    }
    fetch(r + step);
    // element e's factor: column 8 g + e - off
    auto factor = [&](int which, int g, int e) {
      const int c = e - off;
      return factors[(8 * which + (c & 7)) * plane + g + (c >> 3) + 1];
    };
    auto normalise = [&](float (&v)[V][8], int kind) {
      if (kind == NORM_NONE) return;
      float mean = 0.f, q = 0.f;
      if (kind == NORM_LAYER) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) mean += v[i][e];
        mean = join(mean, false) * inv_d;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] -= mean;
        if (mask[i] != 0xFFu) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (!((mask[i] >> e) & 1u)) v[i][e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) q = fmaf(v[i][e], v[i][e], q);
      }
      const float f = rsqrtf(join(q, false) * inv_d + p.eps);
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] *= f;
    };
    auto store = [&](void* t, int i, const float (&v)[8]) {
      const int64_t at = first + 8 * (g0 + 32 * i);
      if (mask[i] == 0xFFu) {
        const uint64_t o[4] = {rn_pack(v[0], v[1]), rn_pack(v[2], v[3]), rn_pack(v[4], v[5]), rn_pack(v[6], v[7])};
        rn_store8<T>(t, at, o);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if ((mask[i] >> e) & 1u) rn_store<T>(t, at + e, v[e]);
      }
    };
    if (p.branch) {
      normalise(u, p.post);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (mask[i]) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[i][e] = fmaf(factor(0, g0 + 32 * i, e), u[i][e], x[i][e]);
          if (mask[i] != 0xFFu) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (!((mask[i] >> e) & 1u)) x[i][e] = 0.f;
          }
        }
    }
    if (p.x_out) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (mask[i]) store(p.x_out, i, x[i]);
    }
    if (!p.y) continue;
    normalise(x, p.pre);
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!mask[i]) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[i][e] = fmaf(x[i][e], factor(1, g0 + 32 * i, e), factor(2, g0 + 32 * i, e));
        if (OUT8 && ((mask[i] >> e) & 1u)) amax = fmaxf(amax, fabsf(x[i][e]));
      }
      if constexpr (!OUT8) store(p.y, i, x[i]);
    }
    if constexpr (OUT8) {
      amax = join(amax, true);
      const float inv = amax > 0.f ? 448.0f / amax : 1.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (!mask[i]) continue;
        const uint32_t lo = pack_e4m3x4(x[i][0] * inv, x[i][1] * inv, x[i][2] * inv, x[i][3] * inv);
        const uint32_t hi = pack_e4m3x4(x[i][4] * inv, x[i][5] * inv, x[i][6] * inv, x[i][7] * inv);
        uint8_t* at = static_cast<uint8_t*>(p.y) + first + 8 * (g0 + 32 * i);
        if (mask[i] == 0xFFu) {
          *reinterpret_cast<uint2*>(at) = make_uint2(lo, hi);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if ((mask[i] >> e) & 1u) at[e] = static_cast<uint8_t>((e < 4 ? lo : hi) >> (8 * (e & 3)));
        }
      }
      if (tid == 0 && live) p.yscale[sample + r] = amax > 0.f ? amax / 448.0f : 1.0f;
    }
  }
}

}  // namespace

template <typename T, bool OUT8, int V, bool EXACT, bool RING>
static cudaError_t rn_go(const ResidualNormParams& p, const RnPlan& plan, unsigned grid, int threads, size_t smem,
                         cudaStream_t s) {
  // The opt-in at every size: what launches without it is 48 KB less the kernel's
  // own arrays (2 KB of sums), which the factors alone reach at 3944 columns.
  static std::atomic<uint64_t> done{0};  // one bit per device: the kernel's shared-memory opt-in
  int dev = 0;
  cudaGetDevice(&dev);
  if (!((done >> dev) & 1u)) {
    const cudaError_t e = cudaFuncSetAttribute(residual_norm_kernel<T, OUT8, V, EXACT, RING>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, RN_SMEM_MAX);
    if (e != cudaSuccess) return e;
    done |= uint64_t(1) << dev;
  }
  residual_norm_kernel<T, OUT8, V, EXACT, RING><<<grid, threads, smem, s>>>(p, plan);
  return cudaGetLastError();
}

template <typename T, bool OUT8>
static cudaError_t rn_launch(const ResidualNormParams& p, cudaStream_t s) {
  static const int sms = device_sm_count();
  const int n8 = p.D / 8;
  RnPlan plan;
  int v;
  if (n8 <= 32) {  // rows narrower than a warp share it
    plan.tg = 4;
    while (plan.tg < n8) plan.tg *= 2;
    v = 1;
  } else {
    // many rows: few threads with long rows each (fewer joins, more loads in
    // flight; two 4360 x 3072 samples at 4, 3 and 2 vectors a thread: 39, 47, 60
    // us); up to two and a half waves of one-vector threads: as many threads per
    // row as there are (3072 columns, 1, 300, 600 and 1200 rows: 3.8, 6.7, 9.6
    // and 13.1 us against 5.6, 10.4, 11.4 and 11.1; 1024, 600 and 4096 rows: 4.6
    // and 12.0 against 6.9 and 11.3)
    const bool few = static_cast<int64_t>(p.B) * p.rows_per_batch * n8 <= static_cast<int64_t>(2560) * sms;
    const int cap = few ? (n8 + 511) / 512 : sizeof(T) == 4 ? 2 : 4;
    const int w = (n8 + 32 * cap - 1) / (32 * cap);
    plan.tg = 32 * (w < 16 ? w : 16);
    v = (n8 + plan.tg - 1) / plan.tg;
  }
  const int factor_bytes = p.D * 12, row_bytes = p.D * static_cast<int>(sizeof(T)) * (p.branch ? 2 : 1);
  // rows at a time: as many as the threads give, 15 where they need a barrier
  auto split = [&](int threads) {
    const int fit = threads / plan.tg;
    plan.groups = plan.tg > 32 && fit > 15 ? 15 : fit;
    if (plan.groups > p.rows_per_batch && plan.tg >= 32) plan.groups = p.rows_per_batch;
    return (p.rows_per_batch + plan.groups - 1) / plan.groups;  // rounds of a sample's rows
  };
  const int one = max(1, sms / p.B);  // CTAs per sample at one per SM
  plan.stages = 0;
  int rounds = split(RN_RING_THREADS);
  // The ring where two norms in a row leave loads straight to registers, one row
  // ahead, too few in flight: two 9480 x 3072 samples 81 us against 98, two of 2000
  // rows 23.5 against 27.6; with the second norm alone it is the other way, 91
  // against 81 (4360 rows 41.5 against 41.1, in fp32 77 against 74).
  if (p.branch && p.post != NORM_NONE && v > 1 && rounds > 2 * one) {
    const int fit = (RN_SMEM_MAX - factor_bytes) / (row_bytes * plan.groups);
    if (fit >= 2) plan.stages = fit < RN_MAX_STAGES ? fit : RN_MAX_STAGES;
  }
  const bool ring = plan.stages > 0;
  if (!ring) rounds = split(512);
  const int threads = plan.tg * plan.groups;
  const int want = ring ? one : max(1, (v == 1 ? 1024 : 512) / threads * sms / p.B);
  plan.per = rounds < want ? rounds : want;
  plan.staged = rounds > plan.per;
  auto al = [](const void* a) { return (reinterpret_cast<uintptr_t>(a) & 15) == 0; };
  plan.fvec = al(p.gate) && al(p.scale) && al(p.shift) && al(p.post_weight) && al(p.pre_weight) && p.mod_stride % 4 == 0;
  const unsigned grid = static_cast<unsigned>(p.B) * plan.per;
  const size_t smem =
      (plan.staged ? factor_bytes : 0) + static_cast<size_t>(plan.stages) * plan.groups * row_bytes;
  const bool exact = plan.tg >= 32 && plan.tg * v == n8;
#define AF_RN_CASE(V_)                                                                                         \
  if (v == V_) {                                                                                               \
    if constexpr (V_ > 1) {                                                                                    \
      if (ring)                                                                                                \
        return exact ? rn_go<T, OUT8, V_, true, true>(p, plan, grid, threads, smem, s)                          \
                     : rn_go<T, OUT8, V_, false, true>(p, plan, grid, threads, smem, s);                        \
    }                                                                                                          \
    return rn_go<T, OUT8, V_, false, false>(p, plan, grid, threads, smem, s);                                  \
  }
  AF_RN_CASE(1)
  AF_RN_CASE(2)
  AF_RN_CASE(3)
  AF_RN_CASE(4)
#undef AF_RN_CASE
  return cudaErrorInvalidValue;
}

template <typename T, bool OUT8, int V>
static cudaError_t rn_shift(const ResidualNormParams& p, const RnPlan& plan, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};  // one bit per device: the kernel's shared-memory opt-in
  int dev = 0;
  cudaGetDevice(&dev);
  if (!((done >> dev) & 1u)) {
    const cudaError_t e = cudaFuncSetAttribute(residual_norm_shift_kernel<T, OUT8, V>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, RN_SMEM_MAX);
    if (e != cudaSuccess) return e;
    done |= uint64_t(1) << dev;
  }
  residual_norm_shift_kernel<T, OUT8, V><<<static_cast<unsigned>(p.B) * plan.per, plan.tg * plan.groups,
                                           24 * rn_plane(p.D) * sizeof(float), s>>>(p, plan);
  return cudaGetLastError();
}

template <typename T, bool OUT8>
static cudaError_t rn_any(const ResidualNormParams& p, bool aligned, cudaStream_t s) {
  const size_t rows = static_cast<size_t>(p.B) * p.rows_per_batch;
  static const int sms = device_sm_count();
  // enough rows for every SM to take more than a round of them: aligned vectors
  // of each row.  1001 columns, value by value against this (us): 1 row 3.1 and
  // 5.5, 500 rows 4.0 and 7.1, 1200 rows 6.1 and 7.5, 2400 rows 11.2 and 12.3; 6000
  // rows of 101 columns 6.8 and 5.5; two 4360 x 3001 samples 102 and 56.
  const int nv = (p.D + 14) / 8;  // vectors that a row may touch
  RnPlan plan{};
  plan.tg = 4;
  while (plan.tg < 32 && plan.tg < nv) plan.tg *= 2;
  if (nv > 32) plan.tg = (nv + 127) / 128 * 32;
  if (aligned && plan.tg <= 512) {
    const int v = plan.tg < 32 ? 1 : (nv + plan.tg - 1) / plan.tg;
    plan.groups = 512 / plan.tg;
    if (plan.tg > 32 && plan.groups > 15) plan.groups = 15;
    const int one = max(1, sms / p.B), rounds = (p.rows_per_batch + plan.groups - 1) / plan.groups;
    plan.per = rounds < one ? rounds : one;
    if (4 * rounds >= 5 * one) {
      if (v == 1) return rn_shift<T, OUT8, 1>(p, plan, s);
      if (v == 2) return rn_shift<T, OUT8, 2>(p, plan, s);
      if (v == 3) return rn_shift<T, OUT8, 3>(p, plan, s);
      return rn_shift<T, OUT8, 4>(p, plan, s);
    }
  }
  int tg = 4, threads = RN_THREADS;
  if (p.D <= 128) {  // four columns a thread
    while (tg < 32 && tg * 4 < p.D) tg *= 2;
  } else {  // eight, sixteen above 8192
    tg = (p.D + 255) / 256 * 32;
    if (tg > 1024) tg = 1024;
    if (tg > 32) threads = tg;
  }
  const int e = (p.D + tg - 1) / tg;
  const unsigned grid = static_cast<unsigned>((rows * tg + threads - 1) / threads);
  auto kernel = p.D <= 128 ? residual_norm_any_kernel<T, OUT8, 4, false>
                : e <= 8   ? residual_norm_any_kernel<T, OUT8, 8, true>
                           : residual_norm_any_kernel<T, OUT8, 16, true>;
  kernel<<<grid, threads, 0, s>>>(p, tg);
  return cudaGetLastError();
}

cudaError_t launch_residual_norm(const ResidualNormParams& p, bool f32, cudaStream_t s) {
  auto al = [](const void* a) { return (reinterpret_cast<uintptr_t>(a) & 15) == 0; };
  const bool aligned = al(p.x) && al(p.branch) && al(p.x_out) && al(p.y), vec = aligned && p.D % 8 == 0;
  if (p.yscale) {
    if (vec) return f32 ? rn_launch<float, true>(p, s) : rn_launch<uint16_t, true>(p, s);
    return f32 ? rn_any<float, true>(p, aligned, s) : rn_any<uint16_t, true>(p, aligned, s);
  }
  if (vec) return f32 ? rn_launch<float, false>(p, s) : rn_launch<uint16_t, false>(p, s);
  return f32 ? rn_any<float, false>(p, aligned, s) : rn_any<uint16_t, false>(p, aligned, s);
}

}  // namespace af
