// Root-mean-square norm with the residual's addition and an output in E4M3 with scales, the
// activations of lhcal_matvec.
//
// Per row: r = x + residual rounded to the stored type; v = r w / sqrt(mean(r^2) + eps); out: r, v
// rounded to the stored type, and E4M3 of v / s with s = max|v| / 448 over the row or 128 channels.
//
// The root's factor is common to a row: with m = max|r w|, s = m / (448 rms) and v / s = r w 448 / m.
// So the maximum needs no root, sum and maximum meet in one reduction, and the E4M3 values do not
// wait for it where scales are per 128 channels.
//
// One CTA a row (four rows of one warp). r w stays in registers until the output, so that each tensor
// is read and written once; rows of more than 16384 channels (fp32: 8192) are read again. CTAs are small,
// so that the SM always has rows that load, rows that reduce and rows that store.
//
// Measured: 16384 x 4096 bf16 with residual to E4M3 per 128 channels 73.8 us (6.4 TB/s), bf16 to bf16 83 us
// (6.5 TB/s), fp32 8192 x 4096 70 us (6.2 TB/s), 1037 x 2560 bf16 4.6 us, one row of 4096 2.7 us: HBM, and
// for few rows the latency of a load, a reduction and a store. Without a residual the 8-bit output is
// bound by instructions (16384 x 2560: 36 us, 3.5 TB/s).
#include <cuda_fp8.h>

#include <cfloat>

#include "common.cuh"

namespace lhcal {
namespace {

constexpr float kE4m3Max = 448.f;

// A unit of K channels as loaded, in 16-byte parts. Ordinary loads, not the read-only path: the residual may be
// written in place and (long rows) read again by this kernel.
template <typename T, int K>
struct Raw {
  static constexpr int kParts = K * sizeof(T) / 16;
  uint4 a[kParts];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kParts; ++i) a[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kParts; ++i) reinterpret_cast<uint4*>(p)[i] = a[i];
  }
  __device__ __forceinline__ void get(float* v) const {
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      const uint32_t u[4] = {a[i].x, a[i].y, a[i].z, a[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(T) == 4) {
          v[4 * i + k] = __uint_as_float(u[k]);
        } else {
          v[8 * i + 2 * k] = __uint_as_float(u[k] << 16);
          v[8 * i + 2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
        }
      }
    }
  }
  __device__ __forceinline__ void set(const float* v) {  // rounds
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      uint32_t u[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(T) == 4) {
          u[k] = __float_as_uint(v[4 * i + k]);
        } else {
          const __nv_bfloat162 b = __floats2bfloat162_rn(v[8 * i + 2 * k], v[8 * i + 2 * k + 1]);
          u[k] = *reinterpret_cast<const uint32_t*>(&b);
        }
      }
      a[i] = make_uint4(u[0], u[1], u[2], u[3]);
    }
  }
};

// The sum of one value and the maximum of another over the CTA, the same and in the same order in
// every thread.
__device__ __forceinline__ void block_reduce(float& sum, float& top, float2* red) {
  auto tree = [&]() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
  };
  tree();
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(sum, top);
  __syncthreads();
  const float2 v = (threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : make_float2(0.f, 0.f);
  sum = v.x;
  top = v.y;
  tree();
}

// A row's tensors; NULL for those that are not there.
template <typename T>
struct Row {
  const T *x, *residual;
  T *residual_out, *y;
  uint8_t* y8;
  float* scale;
  __device__ __forceinline__ Row(const RmsnormArgs& a, int64_t row)
      : x(static_cast<const T*>(a.x) + row * a.ldx),
        residual(a.residual ? static_cast<const T*>(a.residual) + row * a.ldr : nullptr),
        residual_out(a.residual_out ? static_cast<T*>(a.residual_out) + row * a.ldro : nullptr),
        y(a.y ? static_cast<T*>(a.y) + row * a.ldy : nullptr),
        y8(a.y8 ? a.y8 + row * a.ldy8 : nullptr),
        scale(a.y8 ? a.y8_scale + row * (a.scale_block ? (static_cast<uint32_t>(a.cin) + LHCAL_SCALE_BLOCK - 1) / LHCAL_SCALE_BLOCK : 1)
                   : nullptr) {}
};

// r = x + residual of a unit, rounded to the stored type, into x.
template <typename T, int K>
__device__ __forceinline__ void add(Raw<T, K>& x, const Raw<T, K>& res) {
  float u[K], v[K];
  x.get(u);
  res.get(v);
#pragma unroll
  for (int i = 0; i < K; ++i) u[i] += v[i];
  x.set(u);
}
// v = r w of a unit, r in v before, and its largest magnitude; the sum of r's squares goes on.
template <typename WT, int K>
__device__ __forceinline__ float weigh(const WT* weight, float* v, float& sum) {
#pragma unroll
  for (int i = 0; i < K; ++i) sum = fmaf(v[i], v[i], sum);
  if (weight) {
    float w[K];
    Raw<WT, K> raw;
    raw.load(weight);
    raw.get(w);
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] *= w[i];
  }
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < K; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}
template <typename T, typename WT, int K>
__device__ __forceinline__ float weigh(const WT* weight, const Raw<T, K>& r, float* v, float& sum) {
  r.get(v);
  return weigh<WT, K>(weight, v, sum);
}

// Two fp32 values in a 64-bit register, as one instruction multiplies them.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// A unit as E4M3 of v 448 / m (cvt.satfinite: at most 448; NaN stays NaN). bf16 rows times bf16 weights have
// 16 bits, so that 1 in 2400 of these quotients is a tie of two E4M3 values, which an error in the last place
// would decide at random. Hence q0 = a / b by the approximate reciprocal, the exact remainder a - q0 b of one
// fma, and q = q0 + (a - q0 b) / b, rounded once; a = 7/8 v and b = m / 512 are exact for 16 bits and do not
// overflow. Against a product with 448 / m: 16384 x 4096 with residual 74.9 in place of 74.1 us, 16384 x 2560
// without 36.9 in place of 35.5. For fp32 rows the pairs below cost more than they save (8192 x 4096: 77 us, 71
// one by one).
template <bool PAIRS, int K>
__device__ __forceinline__ void quantise(uint8_t* to, const float* v, float m) {
  const bool tiny = m < 0x1p-60f;  // 512 / m or the remainders might leave fp32's range; 0 has no quotient
  const float b = m * (tiny ? 0x1p91f : 0x1p-9f), in = tiny ? 0.875f * 0x1p100f : 0.875f;
  float by;
  asm("rcp.approx.f32 %0, %1;" : "=f"(by) : "f"(b));
  by = m > 0.f ? by : 0.f;
  float q[K];
  if constexpr (PAIRS) {
    const uint64_t by2 = pair(by, by), minus_b2 = pair(-b, -b), in2 = pair(in, in);
#pragma unroll
    for (int i = 0; i < K; i += 2) {
      const uint64_t a = mul2(pair(v[i], v[i + 1]), in2), q0 = mul2(a, by2), left = fma2(q0, minus_b2, a);
      asm("mov.b64 {%0, %1}, %2;" : "=f"(q[i]), "=f"(q[i + 1]) : "l"(fma2(left, by2, q0)));
    }
  } else {
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const float a = v[i] * in, q0 = a * by;
      q[i] = fmaf(fmaf(-q0, b, a), by, q0);
    }
  }
  uint32_t h[K / 4];
#pragma unroll
  for (int i = 0; i < K / 4; ++i)
    h[i] = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(q[4 * i], q[4 * i + 1]), __NV_SATFINITE, __NV_E4M3)) |
           static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(q[4 * i + 2], q[4 * i + 3]), __NV_SATFINITE, __NV_E4M3)) << 16;
  if constexpr (K == 16)
    *reinterpret_cast<uint4*>(to) = make_uint4(h[0], h[1], h[2], h[3]);
  else
    *reinterpret_cast<uint2*>(to) = make_uint2(h[0], h[1]);
}

// The outputs of unit u: v = r w, m its scale's maximum. The scale is m / (448 rms); where it is 0, so
// are the values.
template <typename T, int K>
__device__ __forceinline__ void write(const Row<T>& row, bool by_block, int u, const float* v, float rstd, float m) {
  if (row.y) {
    float n[K];
#pragma unroll
    for (int i = 0; i < K; ++i) n[i] = v[i] * rstd;
    Raw<T, K> y;
    y.set(n);
    y.store(row.y + u * K);
  }
  if (!row.y8) return;
  const float s = m > 0.f ? m * rstd * (1.f / kE4m3Max) : 0.f;
  constexpr int kUnits = LHCAL_SCALE_BLOCK / K;
  if (by_block ? u % kUnits == 0 : u == 0) row.scale[by_block ? u / kUnits : 0] = s;
  quantise<sizeof(T) == 2, K>(row.y8 + u * K, v, s == 0.f ? 0.f : m);
}

// Maximum over the units of a 128-channel block, which lie in consecutive lanes of one warp.
template <int K>
__device__ __forceinline__ float block_max(float m) {
#pragma unroll
  for (int o = LHCAL_SCALE_BLOCK / K / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

__device__ __forceinline__ float inverse_rms(const RmsnormArgs& a, float sum) {
  return __fdiv_rn(1.f, __fsqrt_rn(sum / static_cast<float>(a.cin) + a.eps));
}

// Whether r w and the sum of r's squares kept fp32's precision; NaN is not. The common case in two comparisons: the
// sum in [2^-60, 2^100] and the largest |r w| too.
__device__ __forceinline__ bool ordinary(const RmsnormArgs& a, float sum, float top) {
  constexpr uint32_t kLow = 67u << 23, kSpan = (227u - 67u) << 23;
  if (__float_as_uint(sum) - kLow <= kSpan && __float_as_uint(top) - kLow <= kSpan) return true;
  return sum <= 0x1p100f && top <= 0x1p100f && (top >= 0x1p-60f || top == 0.f) && (sum >= 0x1p-60f || a.eps >= 0x1p-90f);
}

// The outputs of any other row, with r and the root of eps divided by the power of two that brings the larger
// to [1/2, 1): that leaves v as it is. Three passes over the row, from residual_out where there is one, since the
// residual may have been updated in place. A call, with its arguments by value, and registers bounded to what the
// kernels need without it: inlined, or by reference, it costs them 2 to 4% (16384 x 4096 to E4M3 per 128: 74.6 us
// without it, 75.1, 76.4, 77.8).
template <typename T, typename WT>
__device__ __noinline__ void scaled_row(const RmsnormArgs a, int64_t at, float2* red) {
  constexpr int K = 8;
  const Row<T> row(a, at);
  const int units = static_cast<int>(a.cin / K), span = blockDim.x, tid = threadIdx.x;
  auto get_r = [&](int u, float* v) {
    Raw<T, K> r;
    r.load((row.residual_out ? row.residual_out : row.x) + u * K);
    if (row.residual && !row.residual_out) {
      Raw<T, K> res;
      res.load(row.residual + u * K);
      add(r, res);
    }
    r.get(v);
  };
  auto weight_of = [&](int u) { return a.weight ? static_cast<const WT*>(a.weight) + u * K : nullptr; };
  auto reduce = [&](float& sum, float& top) {
    if (span > 32) __syncthreads();  // the last sums are read
    block_reduce(sum, top, red);
  };
  __syncwarp();  // other threads have written residual_out: of one warp here, else block_reduce's barrier lies between
  float v[K], sum = 0.f, top = 0.f;
  for (int u = tid; u < units; u += span) {
    get_r(u, v);
#pragma unroll
    for (int i = 0; i < K; ++i) top = fmaxf(top, fabsf(v[i]));
  }
  reduce(sum, top);
  int e = -200, e_eps = 0;
  if (top > 0.f && top <= FLT_MAX) frexpf(top, &e);
  if (a.eps > 0.f) {
    frexpf(a.eps, &e_eps);
    e = max(e, (e_eps + 1) >> 1);
  }
  if (e == -200) e = 0;
  const float f1 = __int_as_float((127 - (e >> 1)) << 23), f2 = __int_as_float((127 - (e - (e >> 1))) << 23);
  auto get = [&](int u, float* v) {
    get_r(u, v);
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = v[i] * f1 * f2;
  };
  sum = top = 0.f;
  for (int u = tid; u < units; u += span) {
    get(u, v);
    top = fmaxf(top, weigh<WT, K>(weight_of(u), v, sum));
  }
  reduce(sum, top);
  const float rstd = __fdiv_rn(1.f, __fsqrt_rn(sum / static_cast<float>(a.cin) + a.eps * f1 * f2 * f1 * f2));
  for (int u = tid; u - tid < units; u += span) {
    float m = 0.f, unused = 0.f;
    if (u < units) {
      get(u, v);
      m = weigh<WT, K>(weight_of(u), v, unused);
    }
    if (row.y8 && a.scale_block) m = block_max<K>(m);
    if (u < units) write<T, K>(row, a.scale_block, u, v, rstd, a.scale_block ? m : top);
  }
}

// Rows of at most U units a thread: i * blockDim.x + thread. Rows of one warp: blockDim.y of them.
template <typename T, typename WT, int K, int U>
__global__ void __launch_bounds__(U == 1 ? 1024 : 512, K == 8 && U == 2 && sizeof(T) == 2 ? 3 : 2) rmsnorm_kernel(const RmsnormArgs a) {
  __shared__ float2 red[32];
  const int64_t at = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (at >= a.tokens) return;  // blockDim.y > 1: no barrier follows
  const Row<T> row(a, at);
  const int units = static_cast<int>(a.cin / K), span = blockDim.x, tid = threadIdx.x;
  Raw<T, K> r[U], res[U];
#pragma unroll
  for (int i = 0; i < U; ++i)
    if (i * span + tid < units) r[i].load(row.x + (i * span + tid) * K);
  if (row.residual) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (i * span + tid < units) res[i].load(row.residual + (i * span + tid) * K);
  }
  float v[U][K], m[U], sum = 0.f, top = 0.f;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int u = i * span + tid;
    m[i] = 0.f;
    if (u < units) {
      if (row.residual) add(r[i], res[i]);
      if (row.residual_out) r[i].store(row.residual_out + u * K);
      m[i] = weigh<T, WT, K>(a.weight ? static_cast<const WT*>(a.weight) + u * K : nullptr, r[i], v[i], sum);
      top = fmaxf(top, m[i]);
    }
  }
  if (row.y8 && a.scale_block) {
#pragma unroll
    for (int i = 0; i < U; ++i) m[i] = block_max<K>(m[i]);
  }
  block_reduce(sum, top, red);
  if (!ordinary(a, sum, top)) return scaled_row<T, WT>(a, at, red);
  const float rstd = inverse_rms(a, sum);
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int u = i * span + tid;
    if (u < units) write<T, K>(row, a.scale_block, u, v[i], rstd, a.scale_block ? m[i] : top);
  }
}

// Rows of any length, read again for the output: from residual_out where there is one, since the
// residual may have been updated in place.
template <typename T, typename WT, int K>
__global__ void __launch_bounds__(1024, sizeof(T) == 4 ? 2 : 1) rmsnorm_long_kernel(const RmsnormArgs a) {
  __shared__ float2 red[32];
  const Row<T> row(a, blockIdx.x);
  const int units = static_cast<int>(a.cin / K), span = blockDim.x, tid = threadIdx.x;
  auto weight_of = [&](int u) { return a.weight ? static_cast<const WT*>(a.weight) + u * K : nullptr; };
  auto get_r = [&](int u) {
    Raw<T, K> r;
    r.load(row.x + u * K);
    if (row.residual) {
      Raw<T, K> res;
      res.load(row.residual + u * K);
      add(r, res);
    }
    return r;
  };
  float v[K], sum = 0.f, top = 0.f;
  for (int u = tid; u < units; u += span) {
    const Raw<T, K> r = get_r(u);
    if (row.residual_out) r.store(row.residual_out + u * K);
    top = fmaxf(top, weigh<T, WT, K>(weight_of(u), r, v, sum));
  }
  block_reduce(sum, top, red);
  if (!ordinary(a, sum, top)) return scaled_row<T, WT>(a, blockIdx.x, red);
  const float rstd = inverse_rms(a, sum);
  for (int u = tid; u - tid < units; u += span) {
    float m = 0.f, unused = 0.f;
    if (u < units) {
      Raw<T, K> r;
      if (row.residual_out)
        r.load(row.residual_out + u * K);
      else
        r = get_r(u);
      m = weigh<T, WT, K>(weight_of(u), r, v, unused);
    }
    if (row.y8 && a.scale_block) m = block_max<K>(m);
    if (u < units) write<T, K>(row, a.scale_block, u, v, rstd, a.scale_block ? m : top);
  }
}

template <typename T, typename WT, int K, int U>
void launch_rows(const RmsnormArgs& a, cudaStream_t stream) {
  const unsigned threads = static_cast<unsigned>(ceil_div(ceil_div(a.cin, K * U), 32) * 32);
  const unsigned rows = threads == 32 ? 4 : 1;  // rows of one warp: four a CTA
  void* args[] = {const_cast<RmsnormArgs*>(&a)};
  // 0.2 us less on the host than the launch syntax.
  cudaLaunchKernel(reinterpret_cast<const void*>(rmsnorm_kernel<T, WT, K, U>), dim3(static_cast<unsigned>(ceil_div(a.tokens, rows))),
                   dim3(threads, rows), args, 0, stream);
}

// How a row is shared out (bf16, us; 8 x 1: a unit of 8 channels a thread; measured before the quotients were
// corrected by their remainders, which adds 1 to 4% to each form with an 8-bit output):
//   one 16-byte load a thread where the SMs then hold all rows at once, and for rows of one warp:
//     600 x 1024 8 x 1 3.1, 8 x 2 3.5, 16 x 2 3.9; 60000 x 256 22.3, 24.6, 32.7;
//   else, with an 8-bit output, fewer and longer units, for fewer maxima to be joined and quotients:
//     16384 x 4096 98, 80, 72.7; 16384 x 2560 62, 54, 48.7; 30000 x 768 34.5, 36.6, 29.7;
//   but not where they leave lanes without work: 16384 x 1280 32.7, 29.9, 30.9; 60000 x 512 44.8, 37.0, 38.9;
//   nor without that output while there are few waves: 1037 x 2560 5.3, 4.4, 5.1, 2000 x 4096 10.8, 9.4, 8.8.
// fp32 has units of 8 channels (32 bytes): of 16, a warp's loads lie 64 bytes apart (16384 x 2560: 108 against 84).
template <typename T, typename WT>
void launch(const RmsnormArgs& a, cudaStream_t stream) {
  constexpr int K = sizeof(T) == 2 ? 16 : 8;
  const int64_t n = a.tokens * a.cin, full = ceil_div(a.cin, 32 * 32) * 32 * 32;  // full: channels of whole warps, 16 x 2
  if (a.cin > 512 * 2 * K)
    rmsnorm_long_kernel<T, WT, K><<<static_cast<unsigned>(a.tokens), 1024, 0, stream>>>(a);
  else if (a.cin <= 256 || (a.cin <= 1024 * 8 && n <= kNumSms * 8192))
    launch_rows<T, WT, 8, 1>(a, stream);
  else if (a.cin <= 512 * 2 * 8 && (K == 8 || a.cin * 10 < full * 7 || (a.y8 == nullptr && n <= kNumSms * 40960)))
    launch_rows<T, WT, 8, 2>(a, stream);
  else
    launch_rows<T, WT, K, 2>(a, stream);
}

}  // namespace

lhcal_status launch_rmsnorm(const RmsnormArgs& a, cudaStream_t stream) {
  const bool w32 = a.wtype == LHCAL_F32;
  if (a.dtype == LHCAL_BF16)
    w32 ? launch<__nv_bfloat16, float>(a, stream) : launch<__nv_bfloat16, __nv_bfloat16>(a, stream);
  else
    w32 ? launch<float, float>(a, stream) : launch<float, __nv_bfloat16>(a, stream);
  return check_launch("rmsnorm");
}

}  // namespace lhcal
