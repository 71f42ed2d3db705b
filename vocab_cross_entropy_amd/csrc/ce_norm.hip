// RMS norm with the residual's addition, its 8-bit form and its gradient.
//
//   s = x + residual,  y = s rstd w,  rstd = (mean s^2 + eps)^(-1/2)
//   ds = rstd (dy w) - s rstd^3 mean(dy w s) + dsum,   dw = sum over rows of dy s rstd
// The sum s is held in FP32; y comes from it unrounded, and its rounding to the
// input's type is the residual stream that is written.  The gradient takes
// that written s as its input.  Squares, means and dw are FP32 sums in a
// fixed order.
//
// 8-bit form: per group of columns, scale = max(max |y| / 448, 2^-126), and the
// e4m3 value of y / scale (448 is e4m3's largest; the floor keeps 1 / scale
// finite for a row of zeros).
//
// Bound: each input read once and each output written once.  A row's columns
// stay in one workgroup's registers between the sum of squares and the output;
// narrow rows take one wave each.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ce_internal.h"
#include "ce_vec.h"

namespace vce {
namespace {

constexpr float kFp8Max = 448.f;
constexpr float kScaleMin = 1.17549435e-38f;  // 2^-126, the smallest normal

// The sum (or largest) of v over the T threads of a row; every thread gets it.
// T = 64: one wave.  Else `red` holds T / 64 floats, and the call synchronises
// the workgroup twice.
template <int T>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = wave_sum(v);
  if constexpr (T > 64) {
    const int w = (int)threadIdx.x >> 6;
    __syncthreads();  // `red` may still be read from the last call
    if ((threadIdx.x & 63) == 0) red[w] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int k = 1; k < T / 64; ++k) v += red[k];
  }
  return v;
}
template <int T>
__device__ __forceinline__ float row_max(float v, float* red) {
  v = wave_max(v);
  if constexpr (T > 64) {
    const int w = (int)threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[w] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int k = 1; k < T / 64; ++k) v = fmaxf(v, red[k]);
  }
  return v;
}

__device__ __forceinline__ void load_weight(const char* w, int32_t wdtype, int64_t j, int64_t D, float (&f)[kG]) {
  if (wdtype == CE_BF16)
    load_f32<CE_BF16>(w, j, D, f);
  else
    load_f32<CE_F32>(w, j, D, f);
}

// eight e4m3 values (OCP, round to nearest even), little-endian
__device__ __forceinline__ uint2 pack_fp8(const float (&f)[kG]) {
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[4], f[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[6], f[7], hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}

__device__ __forceinline__ void store_fp8(uint8_t* row, int64_t j, int64_t D, uint2 v) {
  typedef unsigned u32x2v __attribute__((ext_vector_type(2)));
  typedef u32x2v u32x2_a1 __attribute__((aligned(1)));
  if (j + kG <= D) {
    const u32x2v w = {v.x, v.y};
    *reinterpret_cast<u32x2_a1*>(row + j) = w;
  } else {
#pragma unroll
    for (int e = 0; e < kG - 1; ++e)
      if (j + e < D) row[j + e] = (uint8_t)((e < 4 ? v.x : v.y) >> (8 * (e & 3)));
  }
}

// A row of at most T x P groups by T threads, P groups each (group p T + t):
// T = 64: a wave per row, four rows per workgroup; else a workgroup per row.
template <int DT, int T, int P, bool QUANT>
__global__ __launch_bounds__(T < 256 ? 256 : T) void k_norm(NormArgs a) {
  __shared__ float red[T / 64];
  constexpr int RPW = T < 256 ? 256 / T : 1;
  const int t = (int)threadIdx.x % T;
  const int64_t stride = (int64_t)gridDim.x * RPW;
  constexpr int EB = VecT<DT>::EB;
  // a workgroup's threads share one row where they synchronise (T > 64)
  for (int64_t r = (int64_t)blockIdx.x * RPW + (int)threadIdx.x / T; r < a.N; r += stride) {
    const char* x = a.x + r * a.x_ld * EB;
    const char* res = a.residual ? a.residual + r * a.r_ld * EB : nullptr;
    float v[P][kG];
    float ss = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int64_t j = (int64_t)(p * T + t) * kG;
      if (j < a.D) {
        load_f32<DT>(x, j, a.D, v[p]);
        if (res) {
          float b[kG];
          load_f32<DT>(res, j, a.D, b);
#pragma unroll
          for (int e = 0; e < kG; ++e) v[p][e] += b[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < kG; ++e) v[p][e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < kG; ++e) ss = __builtin_fmaf(v[p][e], v[p][e], ss);
    }
    ss = row_sum<T>(ss, red);
    const float rstd = 1.f / sqrtf(ss / (float)a.D + a.eps);
    float top = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int64_t j = (int64_t)(p * T + t) * kG;
      if (j < a.D) {
        if (a.sum) store_group<DT>(a.sum + r * a.sum_ld * EB, j, a.D, f32_to_raw<DT>(v[p]));
        float w[kG];
        load_weight(a.weight, a.wdtype, j, a.D, w);
#pragma unroll
        for (int e = 0; e < kG; ++e) v[p][e] = v[p][e] * rstd * w[e];
        if constexpr (!QUANT) store_group<DT>(a.y + r * a.y_ld * EB, j, a.D, f32_to_raw<DT>(v[p]));
      }
      if constexpr (QUANT) {
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < kG; ++e) m = fmaxf(m, fabsf(v[p][e]));
        if (a.group) {  // 32, 64 or 128 columns: 4, 8 or 16 neighbouring lanes
          for (int k = 1; k < a.group / kG; k <<= 1) m = fmaxf(m, __shfl_xor(m, k, 64));
          const float sc = fmaxf(m / kFp8Max, kScaleMin);
          const float inv = 1.f / sc;
          if (j < a.D) {
#pragma unroll
            for (int e = 0; e < kG; ++e) v[p][e] *= inv;
            store_fp8(a.q + r * a.q_ld, j, a.D, pack_fp8(v[p]));
            if (j % a.group == 0) a.scales[r * ((a.D + a.group - 1) / a.group) + j / a.group] = sc;
          }
        } else {
          top = fmaxf(top, m);
        }
      }
    }
    if constexpr (QUANT) {
      if (!a.group) {
        top = row_max<T>(top, red);
        const float sc = fmaxf(top / kFp8Max, kScaleMin);
        const float inv = 1.f / sc;
        if (t == 0) a.scales[r] = sc;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const int64_t j = (int64_t)(p * T + t) * kG;
          if (j < a.D) {
#pragma unroll
            for (int e = 0; e < kG; ++e) v[p][e] *= inv;
            store_fp8(a.q + r * a.q_ld, j, a.D, pack_fp8(v[p]));
          }
        }
      }
    }
  }
}

// The gradient: rows r, r + G, ... of the grid's G row slots, with the slot's
// share of dw in registers; a second kernel adds the slots' shares.
template <int DT, int T, int P>
__global__ __launch_bounds__(T < 256 ? 256 : T) void k_norm_grad(NormGradArgs a) {
  __shared__ float red[T / 64];
  constexpr int RPW = T < 256 ? 256 / T : 1;
  const int t = (int)threadIdx.x % T;
  const int64_t slot = (int64_t)blockIdx.x * RPW + (int)threadIdx.x / T;
  const int64_t slots = (int64_t)gridDim.x * RPW;
  constexpr int EB = VecT<DT>::EB;
  float acc[P][kG];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int e = 0; e < kG; ++e) acc[p][e] = 0.f;
  for (int64_t r = slot; r < a.N; r += slots) {
    const char* sr = a.s + r * a.s_ld * EB;
    const char* dyr = a.dy + r * a.dy_ld * EB;
    Raw<DT> s[P], dy[P];
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int64_t j = (int64_t)(p * T + t) * kG;
      if (j < a.D) {
        s[p] = load_group<DT>(sr, j, a.D);
        dy[p] = load_group<DT>(dyr, j, a.D);
        float f[kG], g[kG], w[kG];
        raw_to_f32<DT>(s[p], f);
        raw_to_f32<DT>(dy[p], g);
        load_weight(a.weight, a.wdtype, j, a.D, w);
#pragma unroll
        for (int e = 0; e < kG; ++e) {
          ss = __builtin_fmaf(f[e], f[e], ss);
          dot = __builtin_fmaf(g[e] * w[e], f[e], dot);
        }
      }
    }
    ss = row_sum<T>(ss, red);
    dot = row_sum<T>(dot, red);
    const float rstd = 1.f / sqrtf(ss / (float)a.D + a.eps);
    const float k = rstd * rstd * rstd * (dot / (float)a.D);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int64_t j = (int64_t)(p * T + t) * kG;
      if (j < a.D) {
        float f[kG], g[kG], w[kG], d[kG];
        raw_to_f32<DT>(s[p], f);
        raw_to_f32<DT>(dy[p], g);
        load_weight(a.weight, a.wdtype, j, a.D, w);
        if (a.dsum)
          load_f32<DT>(a.dsum + r * a.dsum_ld * EB, j, a.D, d);
        else
#pragma unroll
          for (int e = 0; e < kG; ++e) d[e] = 0.f;
#pragma unroll
        for (int e = 0; e < kG; ++e) {
          acc[p][e] = __builtin_fmaf(g[e], f[e] * rstd, acc[p][e]);
          d[e] += __builtin_fmaf(g[e] * w[e], rstd, -(f[e] * k));
        }
        if (a.dx) store_group<DT>(a.dx + r * a.dx_ld * EB, j, a.D, f32_to_raw<DT>(d));
      }
    }
  }
  if (a.dweight) {
    char* part = reinterpret_cast<char*>(a.parts + slot * a.D);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int64_t j = (int64_t)(p * T + t) * kG;
      if (j < a.D) store_group<CE_F32>(part, j, a.D, f32_to_raw<CE_F32>(acc[p]));
    }
  }
}

// dw[j] (+)= the slots' shares: 64 columns per workgroup, wave k adds slots k, k + 4, ..., in order,
// and the waves are added in order.
constexpr int kDwWaves = 16;
__global__ __launch_bounds__(64 * kDwWaves) void k_norm_dw(const float* parts, int64_t slots, int64_t D, float* dw,
                                                           int32_t accumulate) {
  __shared__ float part[kDwWaves][64];
  const int lane = (int)threadIdx.x & 63, w = (int)threadIdx.x >> 6;
  const int64_t j = (int64_t)blockIdx.x * 64 + lane;
  float v = 0.f;
  if (j < D)
    for (int64_t k = w; k < slots; k += kDwWaves) v += parts[k * D + j];
  part[w][lane] = v;
  __syncthreads();
  if (w == 0 && j < D) {
    for (int k = 1; k < kDwWaves; ++k) v += part[k][lane];
    dw[j] = accumulate ? dw[j] + v : v;
  }
}

// Row slots of the gradient kernel for N rows (one workgroup holds 4 where a
// wave takes a row).
int64_t grad_slots(int64_t N, int64_t D) {
  const int64_t most = D <= 2048 ? 2048 : 512;
  int64_t s = N < most ? N : most;
  if (D <= 2048) s = (s + 3) & ~(int64_t)3;
  return s;
}

template <int DT, bool QUANT>
void norm_shape(const NormArgs& a, hipStream_t stream) {
  constexpr int64_t most = 1 << 22;  // a launch holds below 2^32 work-items
  const int64_t g = (a.D + kG - 1) / kG;
  const int64_t rows = a.N < most ? a.N : most;
  const int64_t rows4 = (a.N + 3) / 4 < most ? (a.N + 3) / 4 : most;
#define VCE_NORM(T, P, R) hipLaunchKernelGGL((k_norm<DT, T, P, QUANT>), dim3((uint32_t)(R)), dim3(T < 256 ? 256 : T), 0, stream, a)
  if (g <= 64) VCE_NORM(64, 1, rows4);
  else if (g <= 128) VCE_NORM(64, 2, rows4);
  else if (g <= 256) VCE_NORM(64, 4, rows4);
  else if (g <= 512) VCE_NORM(256, 2, rows);
  else if (g <= 1024) VCE_NORM(256, 4, rows);
  else if (g <= 2048) VCE_NORM(1024, 2, rows);
  else VCE_NORM(1024, 4, rows);
#undef VCE_NORM
}

template <int DT>
void grad_shape(const NormGradArgs& a, hipStream_t stream) {
  const int64_t g = (a.D + kG - 1) / kG;
  const int64_t slots = grad_slots(a.N, a.D);
#define VCE_GRAD(T, P, R) hipLaunchKernelGGL((k_norm_grad<DT, T, P>), dim3((uint32_t)(R)), dim3(T < 256 ? 256 : T), 0, stream, a)
  if (g <= 64) VCE_GRAD(64, 1, slots / 4);
  else if (g <= 128) VCE_GRAD(64, 2, slots / 4);
  else if (g <= 256) VCE_GRAD(64, 4, slots / 4);
  else if (g <= 512) VCE_GRAD(256, 2, slots);
  else if (g <= 1024) VCE_GRAD(256, 4, slots);
  else if (g <= 2048) VCE_GRAD(1024, 2, slots);
  else VCE_GRAD(1024, 4, slots);
#undef VCE_GRAD
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
  if (a.N == 0) return hipSuccess;
  if (a.dtype == CE_BF16)
    a.q ? norm_shape<CE_BF16, true>(a, stream) : norm_shape<CE_BF16, false>(a, stream);
  else
    a.q ? norm_shape<CE_F32, true>(a, stream) : norm_shape<CE_F32, false>(a, stream);
  return hipGetLastError();
}

size_t norm_grad_workspace(int64_t N, int64_t D) { return (size_t)grad_slots(N, D) * (size_t)D * 4u; }

hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t stream) {
  hipError_t e = hipSuccess;
  if (a.N > 0) {
    a.dtype == CE_BF16 ? grad_shape<CE_BF16>(a, stream) : grad_shape<CE_F32>(a, stream);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (a.dweight) {
    hipLaunchKernelGGL(k_norm_dw, dim3((uint32_t)((a.D + 63) / 64)), dim3(64 * kDwWaves), 0, stream, a.parts,
                       a.N > 0 ? grad_slots(a.N, a.D) : (int64_t)0, a.D, a.dweight, a.accumulate);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace vce
