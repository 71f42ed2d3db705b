// RMS norm with the residual's addition, its 8-bit form and its gradient.
//
//   s = x + residual,  y = s rstd w,  rstd = (mean s^2 + eps)^(-1/2)
//   n = s rstd,  ds = rstd (dy w - n mean(dy w n)) + dsum,  dw = sum over rows of dy n
// The sum s is held in FP32; y comes from it unrounded, and its rounding to the
// input's type is the residual stream that is written.  The gradient takes
// that written s as its input, and forms n first: the cube of rstd leaves FP32 for
// rows of an rms above 1e13 or, at eps 0, below 1e-13.  Squares, means and dw are
// FP32 sums in a fixed order.
//
// 8-bit form: per group of columns, scale = max(max |y| / 448, 2^-126), and the
// e4m3 value of the FP32 quotient y / scale (448 is e4m3's largest; the floor keeps
// 1 / scale finite for a row of zeros).
//
// Bound: each input read once and each output written once.  A row's columns
// stay in one workgroup's registers between the sum of squares and the output;
// narrow rows take one wave each.  Columns are 32-bit offsets from a uniform row
// pointer (64-bit ones cost two registers an access and a third of the waves).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ce_internal.h"
#include "ce_vec.h"

namespace vce {
namespace {

constexpr float kFp8Max = 448.f;
constexpr float kScaleMin = 1.17549435e-38f;  // 2^-126, the smallest normal

// Sums of N values over the T threads of a row; every thread gets them.  T = 64:
// one wave.  Else the waves exchange them in LDS with one barrier: `red` holds
// two sets, and a row takes the one its predecessor did not (`turn`), whose
// readers have all passed the predecessor's barrier.
template <int T, int N>
struct RowRed {
  float v[2][N][T / 64];
};
template <int T, int N, bool MAX = false>
__device__ __forceinline__ void row_reduce(float (&v)[N], RowRed<T, N>& red, int turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = MAX ? wave_max(v[i]) : wave_sum(v[i]);
  if constexpr (T > 64) {
    const int w = (int)(threadIdx.x % T) >> 6;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((threadIdx.x & 63) == 0) red.v[turn][i][w] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = red.v[turn][i][0];
#pragma unroll
      for (int k = 1; k < T / 64; ++k) v[i] = MAX ? fmaxf(v[i], red.v[turn][i][k]) : v[i] + red.v[turn][i][k];
    }
  }
}

__device__ __forceinline__ void load_weight(const char* w, int32_t wdtype, uint32_t j, uint32_t D, float (&f)[kG]) {
  if (wdtype == CE_BF16)
    load_f32<CE_BF16>(w, j, D, f);
  else
    load_f32<CE_F32>(w, j, D, f);
}

// y / scale for a group's values: 1 / scale rounded down, and what that leaves out, so
// that a quotient is a product and a multiply-add whose sum is off by 2^-46 of it before
// its last rounding (2^-29 for scales above 2^80, where `rest` leaves the normal range).
// Times 1 / scale alone, values next to a border of the type came out as the neighbour;
// a division for each takes 46 us where this and that take 42.6 (8192 x 4096 BF16).
// Both parts are >= 0, so that quotients keep their zeros' signs.
struct Divisor {
  float inv, rest;
};
__device__ __forceinline__ Divisor divisor(float scale) {
  Divisor d;
  d.inv = 1.f / scale;
  float left = __builtin_fmaf(-d.inv, scale, 1.f);
  if (left < 0.f) {
    d.inv = __int_as_float(__float_as_int(d.inv) - 1);
    left = __builtin_fmaf(-d.inv, scale, 1.f);
  }
  d.rest = scale < __builtin_inff() ? left * d.inv : 0.f;
  return d;
}
__device__ __forceinline__ void divide(float (&f)[kG], Divisor d) {
#pragma unroll
  for (int e = 0; e < kG; ++e) f[e] = __builtin_fmaf(f[e], d.inv, f[e] * d.rest);
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

__device__ __forceinline__ void store_fp8(uint8_t* row, uint32_t j, uint32_t D, uint2 v) {
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

// Which of its workgroup's rows a thread works on, as a uniform value
template <int T>
__device__ __forceinline__ int row_of() {
  return T < 256 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x / T) : 0;
}

// A row of at most T x P groups by T threads, P groups each (group p T + t):
// T = 64: a wave per row, four rows per workgroup; else a workgroup per row.
// WHOLE: D is a multiple of 8.  NT: outputs with the non-temporal bit, for those
// that no cache could hold until they are read (8192 x 4096 BF16 to e4m3, new inputs
// and outputs at every call: 43.2 against 45.3 us; with one set of outputs written over
// and over, 41.9 against 41.3, and in BF16 46.9 against 42.4).
template <int DT, int T, int P, bool QUANT, bool WHOLE, bool NT>
__global__ __launch_bounds__(T < 256 ? 256 : T) void k_norm(NormArgs a) {
  __shared__ RowRed<T, 1> red, red_top;
  constexpr int RPW = T < 256 ? 256 / T : 1;
  const int t = (int)threadIdx.x % T;
  const uint32_t D = (uint32_t)a.D;
  const int64_t stride = (int64_t)gridDim.x * RPW;
  constexpr int EB = VecT<DT>::EB;
  int turn = 0;
  // a workgroup's threads share one row where they synchronise (T > 64)
  for (int64_t r = (int64_t)blockIdx.x * RPW + row_of<T>(); r < a.N; r += stride, turn ^= 1) {
    const char* x = a.x + r * a.x_ld * EB;
    Raw<DT> xr[P], rr[P];
#pragma unroll
    for (int p = 0; p < P; ++p) xr[p] = fetch_group<DT, WHOLE>(x, (uint32_t)(p * T + t) * kG, D);
    if (a.residual) {
      const char* res = a.residual + r * a.r_ld * EB;
#pragma unroll
      for (int p = 0; p < P; ++p) rr[p] = fetch_group<DT, WHOLE>(res, (uint32_t)(p * T + t) * kG, D);
    }
    float v[P][kG];
    float ss[1] = {0.f};
#pragma unroll
    for (int p = 0; p < P; ++p) {
      raw_to_f32<DT>(xr[p], v[p]);
      if (a.residual) {
        float b[kG];
        raw_to_f32<DT>(rr[p], b);
#pragma unroll
        for (int e = 0; e < kG; ++e) v[p][e] += b[e];
      }
      const bool in = (uint32_t)(p * T + t) * kG < D;
#pragma unroll
      for (int e = 0; e < kG; ++e) {
        v[p][e] = in ? v[p][e] : 0.f;
        ss[0] = __builtin_fmaf(v[p][e], v[p][e], ss[0]);
      }
    }
    row_reduce<T, 1>(ss, red, turn);
    const float rstd = 1.f / sqrtf(ss[0] / (float)D + a.eps);
    float top[1] = {0.f};
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t j = (uint32_t)(p * T + t) * kG;
      if (j < D) {
        if (a.sum) store_group<DT, NT>(a.sum + r * a.sum_ld * EB, j, D, f32_to_raw<DT>(v[p]));
        float w[kG];
        load_weight(a.weight, a.wdtype, j, D, w);
#pragma unroll
        for (int e = 0; e < kG; ++e) v[p][e] = v[p][e] * rstd * w[e];
        if constexpr (!QUANT) store_group<DT, NT>(a.y + r * a.y_ld * EB, j, D, f32_to_raw<DT>(v[p]));
      }
      if constexpr (QUANT) {
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < kG; ++e) m = fmaxf(m, fabsf(v[p][e]));
        if (a.group) {  // 32, 64 or 128 columns: 4, 8 or 16 neighbouring lanes
          m = row_max16(m, a.group / kG);
          const float sc = fmaxf(m / kFp8Max, kScaleMin);
          const Divisor by = divisor(sc);
          if (j < D) {
            divide(v[p], by);
            store_fp8(a.q + r * a.q_ld, j, D, pack_fp8(v[p]));
            if ((j & (a.group - 1)) == 0) a.scales[r * a.groups + (j >> a.group_shift)] = sc;
          }
        } else {
          top[0] = fmaxf(top[0], m);
        }
      }
    }
    if constexpr (QUANT) {
      if (!a.group) {
        row_reduce<T, 1, true>(top, red_top, turn);
        const float sc = fmaxf(top[0] / kFp8Max, kScaleMin);
        const Divisor by = divisor(sc);
        if (t == 0) a.scales[r] = sc;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const uint32_t j = (uint32_t)(p * T + t) * kG;
          if (j < D) {
            divide(v[p], by);
            store_fp8(a.q + r * a.q_ld, j, D, pack_fp8(v[p]));
          }
        }
      }
    }
  }
}

// Rows of more than 2 groups for each of 1024 threads (D > 16384): the row is
// read again, from L2, for each step that needs the whole of the one before,
// instead of being held (which spilled).  Outputs are written in the last step
// only, each after the same thread's last read of its columns.
template <int DT, bool WHOLE>
__device__ __forceinline__ void wide_sum(const char* x, const char* res, uint32_t j, uint32_t D, float (&v)[kG]) {
  raw_to_f32<DT>(fetch_group<DT, WHOLE>(x, j, D), v);
  if (res) {
    float b[kG];
    raw_to_f32<DT>(fetch_group<DT, WHOLE>(res, j, D), b);
#pragma unroll
    for (int e = 0; e < kG; ++e) v[e] += b[e];
  }
}
template <int DT, bool QUANT, bool WHOLE>
__global__ __launch_bounds__(1024) void k_norm_wide(NormArgs a) {
  constexpr int T = 1024, EB = VecT<DT>::EB;
  __shared__ RowRed<T, 1> red, red_top;
  const uint32_t D = (uint32_t)a.D;
  int turn = 0;
  for (int64_t r = blockIdx.x; r < a.N; r += gridDim.x, turn ^= 1) {
    const char* x = a.x + r * a.x_ld * EB;
    const char* res = a.residual ? a.residual + r * a.r_ld * EB : nullptr;
    float ss[1] = {0.f};
    for (uint32_t j = threadIdx.x * kG; j < D; j += T * kG) {
      float v[kG];
      wide_sum<DT, WHOLE>(x, res, j, D, v);
#pragma unroll
      for (int e = 0; e < kG; ++e) ss[0] = __builtin_fmaf(v[e], v[e], ss[0]);
    }
    row_reduce<T, 1>(ss, red, turn);
    const float rstd = 1.f / sqrtf(ss[0] / (float)D + a.eps);
    float sc = 0.f;
    if (QUANT && !a.group) {
      float top[1] = {0.f};
      for (uint32_t j = threadIdx.x * kG; j < D; j += T * kG) {
        float v[kG], w[kG];
        wide_sum<DT, WHOLE>(x, res, j, D, v);
        load_weight(a.weight, a.wdtype, j, D, w);
#pragma unroll
        for (int e = 0; e < kG; ++e) top[0] = fmaxf(top[0], fabsf(v[e] * rstd * w[e]));
      }
      row_reduce<T, 1, true>(top, red_top, turn);
      sc = fmaxf(top[0] / kFp8Max, kScaleMin);
      if (threadIdx.x == 0) a.scales[r] = sc;
    }
    // every lane takes every step: a group's scale is found across lanes
    for (uint32_t base = 0; base < D; base += T * kG) {
      const uint32_t j = base + threadIdx.x * kG;
      float v[kG], w[kG];
#pragma unroll
      for (int e = 0; e < kG; ++e) v[e] = w[e] = 0.f;
      if (j < D) {
        wide_sum<DT, WHOLE>(x, res, j, D, v);
        if (a.sum) store_group<DT>(a.sum + r * a.sum_ld * EB, j, D, f32_to_raw<DT>(v));
        load_weight(a.weight, a.wdtype, j, D, w);
      }
      float m = 0.f;
#pragma unroll
      for (int e = 0; e < kG; ++e) {
        v[e] = v[e] * rstd * w[e];
        m = fmaxf(m, fabsf(v[e]));
      }
      if constexpr (QUANT) {
        if (a.group) sc = fmaxf(row_max16(m, a.group / kG) / kFp8Max, kScaleMin);
        const Divisor by = divisor(sc);
        if (j < D) {
          divide(v, by);
          store_fp8(a.q + r * a.q_ld, j, D, pack_fp8(v));
          if (a.group && (j & (a.group - 1)) == 0) a.scales[r * a.groups + (j >> a.group_shift)] = sc;
        }
      } else {
        if (j < D) store_group<DT>(a.y + r * a.y_ld * EB, j, D, f32_to_raw<DT>(v));
      }
    }
  }
}

// The gradient.  A workgroup of 1024 threads takes R = 1024 / T rows at a time,
// T threads each, and keeps its share of dw in registers over all its rows; the
// share is added over the R rows in LDS at the end, and a second kernel adds the
// workgroups' shares.  At most one workgroup a CU: each share more is D floats
// written, flushed and read again (1023 x 4096 BF16: 17.6 us with a share per
// row).  PRE: the next rows' loads are issued before this row's sums are
// exchanged, where the registers allow it.
template <int DT, int P>
struct GradRow {
  Raw<DT> s[P], dy[P], dsum[P];
};
template <int DT, int T, int P, bool WHOLE>
__device__ __forceinline__ void fetch_grad_row(const NormGradArgs& a, int64_t r, int t, GradRow<DT, P>& g) {
  constexpr int EB = VecT<DT>::EB;
  const uint32_t D = (uint32_t)a.D;
#pragma unroll
  for (int p = 0; p < P; ++p) g.s[p] = fetch_group<DT, WHOLE>(a.s + r * a.s_ld * EB, (uint32_t)(p * T + t) * kG, D);
#pragma unroll
  for (int p = 0; p < P; ++p) g.dy[p] = fetch_group<DT, WHOLE>(a.dy + r * a.dy_ld * EB, (uint32_t)(p * T + t) * kG, D);
  if (a.dsum) {
#pragma unroll
    for (int p = 0; p < P; ++p)
      g.dsum[p] = fetch_group<DT, WHOLE>(a.dsum + r * a.dsum_ld * EB, (uint32_t)(p * T + t) * kG, D);
  }
}

constexpr int kGradT = 1024;

template <int DT, int T, int P, bool WHOLE>
__global__ __launch_bounds__(kGradT) void k_norm_grad(NormGradArgs a) {
  constexpr int R = kGradT / T;
  constexpr bool PRE = P == 1;
  constexpr int EB = VecT<DT>::EB;
  __shared__ RowRed<T, 2> red[R];
  __shared__ __align__(16) float share[R > 1 ? R : 1][R > 1 ? T * P * kG : 4];
  const int t = (int)threadIdx.x % T;
  const int sub = __builtin_amdgcn_readfirstlane((int)threadIdx.x / T);
  const uint32_t D = (uint32_t)a.D;
  const int64_t step = (int64_t)gridDim.x * R;
  float acc[P][kG], w[P][kG];
  GradRow<DT, P> cur, next;
  int64_t r = (int64_t)blockIdx.x * R + sub;
  if (PRE && r < a.N) fetch_grad_row<DT, T, P, WHOLE>(a, r, t, cur);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const uint32_t j = (uint32_t)(p * T + t) * kG;
#pragma unroll
    for (int e = 0; e < kG; ++e) acc[p][e] = w[p][e] = 0.f;
    if (j < D) load_weight(a.weight, a.wdtype, j, D, w[p]);  // 0 past the row's end
  }
  int turn = 0;
  // the workgroup's rows go together (its threads synchronise); those past the last row only keep step
  for (; r - sub < a.N; r += step, turn ^= 1) {
    const bool live = r < a.N;
    if constexpr (PRE) {
      if (r + step < a.N) fetch_grad_row<DT, T, P, WHOLE>(a, r + step, t, next);
    } else {
      if (live) fetch_grad_row<DT, T, P, WHOLE>(a, r, t, cur);
    }
    float sums[2] = {0.f, 0.f};  // of s^2 and of dy w s
    if (live) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const bool in = (uint32_t)(p * T + t) * kG < D;
        float f[kG], g[kG];
        raw_to_f32<DT>(cur.s[p], f);
        raw_to_f32<DT>(cur.dy[p], g);
#pragma unroll
        for (int e = 0; e < kG; ++e) {
          const float fe = in ? f[e] : 0.f, ge = in ? g[e] : 0.f;
          sums[0] = __builtin_fmaf(fe, fe, sums[0]);
          sums[1] = __builtin_fmaf(ge * w[p][e], fe, sums[1]);
        }
      }
    }
    row_reduce<T, 2>(sums, red[sub], turn);
    if (live) {
      const float rstd = 1.f / sqrtf(sums[0] / (float)D + a.eps);
      const float c = sums[1] / (float)D * rstd;  // mean(dy w n)
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const uint32_t j = (uint32_t)(p * T + t) * kG;
        float f[kG], g[kG], d[kG];
        raw_to_f32<DT>(cur.s[p], f);
        raw_to_f32<DT>(cur.dy[p], g);
        if (a.dsum)
          raw_to_f32<DT>(cur.dsum[p], d);
        else
#pragma unroll
          for (int e = 0; e < kG; ++e) d[e] = 0.f;
#pragma unroll
        for (int e = 0; e < kG; ++e) {
          const float n = f[e] * rstd;
          acc[p][e] = __builtin_fmaf(g[e], n, acc[p][e]);
          d[e] = __builtin_fmaf(__builtin_fmaf(-n, c, g[e] * w[p][e]), rstd, d[e]);
        }
        if (a.dx && j < D) store_group<DT>(a.dx + r * a.dx_ld * EB, j, D, f32_to_raw<DT>(d));
      }
    }
    if constexpr (PRE) cur = next;
  }
  if (!a.dweight) return;
  float* part = a.parts + (int64_t)blockIdx.x * a.D;
  if constexpr (R > 1) {
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        *reinterpret_cast<float4*>(&share[sub][(p * T + t) * kG + 4 * k]) =
            make_float4(acc[p][4 * k], acc[p][4 * k + 1], acc[p][4 * k + 2], acc[p][4 * k + 3]);
    __syncthreads();
    for (uint32_t j = threadIdx.x; j < D; j += kGradT) {
      float v = share[0][j];
#pragma unroll
      for (int k = 1; k < R; ++k) v += share[k][j];
      part[j] = v;
    }
  } else {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t j = (uint32_t)(p * T + t) * kG;
      if (j < D) store_group<CE_F32>(reinterpret_cast<char*>(part), j, D, f32_to_raw<CE_F32>(acc[p]));
    }
  }
}

// The same for D > 16384: the row is read twice, and the workgroup's share of dw is
// kept in LDS (4 D bytes), each thread its own columns.
template <int DT, bool WHOLE>
__global__ __launch_bounds__(1024) void k_norm_grad_wide(NormGradArgs a) {
  constexpr int T = 1024, EB = VecT<DT>::EB;
  __shared__ RowRed<T, 2> red;
  extern __shared__ __align__(16) float share[];  // group g's element e at (g / T) 8 T + e T + g % T
  const uint32_t D = (uint32_t)a.D;
  const int t = (int)threadIdx.x;
  for (uint32_t j = t * kG, at = t; j < D; j += T * kG, at += T * kG)
#pragma unroll
    for (int e = 0; e < kG; ++e) share[at + e * T] = 0.f;
  int turn = 0;
  for (int64_t r = blockIdx.x; r < a.N; r += gridDim.x, turn ^= 1) {
    const char* s = a.s + r * a.s_ld * EB;
    const char* dy = a.dy + r * a.dy_ld * EB;
    float sums[2] = {0.f, 0.f};
    for (uint32_t j = t * kG; j < D; j += T * kG) {
      float f[kG], g[kG], w[kG];
      raw_to_f32<DT>(fetch_group<DT, WHOLE>(s, j, D), f);
      raw_to_f32<DT>(fetch_group<DT, WHOLE>(dy, j, D), g);
      load_weight(a.weight, a.wdtype, j, D, w);
#pragma unroll
      for (int e = 0; e < kG; ++e) {
        sums[0] = __builtin_fmaf(f[e], f[e], sums[0]);
        sums[1] = __builtin_fmaf(g[e] * w[e], f[e], sums[1]);
      }
    }
    row_reduce<T, 2>(sums, red, turn);
    const float rstd = 1.f / sqrtf(sums[0] / (float)D + a.eps);
    const float c = sums[1] / (float)D * rstd;
    for (uint32_t j = t * kG, at = t; j < D; j += T * kG, at += T * kG) {
      float f[kG], g[kG], w[kG], d[kG];
      raw_to_f32<DT>(fetch_group<DT, WHOLE>(s, j, D), f);
      raw_to_f32<DT>(fetch_group<DT, WHOLE>(dy, j, D), g);
      load_weight(a.weight, a.wdtype, j, D, w);
      if (a.dsum)
        raw_to_f32<DT>(fetch_group<DT, WHOLE>(a.dsum + r * a.dsum_ld * EB, j, D), d);
      else
#pragma unroll
        for (int e = 0; e < kG; ++e) d[e] = 0.f;
#pragma unroll
      for (int e = 0; e < kG; ++e) {
        const float n = f[e] * rstd;
        share[at + e * T] = __builtin_fmaf(g[e], n, share[at + e * T]);
        d[e] = __builtin_fmaf(__builtin_fmaf(-n, c, g[e] * w[e]), rstd, d[e]);
      }
      if (a.dx) store_group<DT>(a.dx + r * a.dx_ld * EB, j, D, f32_to_raw<DT>(d));
    }
  }
  if (a.dweight) {
    char* part = reinterpret_cast<char*>(a.parts + (int64_t)blockIdx.x * a.D);
    for (uint32_t j = t * kG, at = t; j < D; j += T * kG, at += T * kG) {
      float f[kG];
#pragma unroll
      for (int e = 0; e < kG; ++e) f[e] = share[at + e * T];
      store_group<CE_F32>(part, j, D, f32_to_raw<CE_F32>(f));
    }
  }
}

// dw[j] (+)= the workgroups' shares: 32 columns per workgroup, thread row k of 32
// adds shares k, k + 32, ... in order, and the rows are added in order.
constexpr int kDwCols = 32, kDwRows = 32;
__global__ __launch_bounds__(kDwCols * kDwRows) void k_norm_dw(const float* parts, int64_t n, int64_t D, float* dw,
                                                               int32_t accumulate) {
  __shared__ float part[kDwRows][kDwCols];
  const int c = (int)threadIdx.x % kDwCols, w = (int)threadIdx.x / kDwCols;
  const int64_t j = (int64_t)blockIdx.x * kDwCols + c;
  float v = 0.f;
  if (j < D) {
#pragma unroll 8
    for (int64_t k = w; k < n; k += kDwRows) v += parts[k * D + j];
  }
  part[w][c] = v;
  __syncthreads();
  if (w == 0 && j < D) {
#pragma unroll
    for (int k = 1; k < kDwRows; ++k) v += part[k][c];
    dw[j] = accumulate ? dw[j] + v : v;
  }
}

// Threads that share a row in the gradient kernel (a row of at most 2 groups
// for each), and its workgroups: as many as the rows fill, at most one a CU.
int grad_threads(int64_t D) {
  const int64_t g = (D + kG - 1) / kG;
  return g <= 128 ? 64 : g <= 256 ? 256 : g <= 512 ? 512 : 1024;
}
constexpr int64_t kGradBlocks = 256;
int64_t grad_blocks(int64_t N, int64_t D) {
  const int64_t rows = kGradT / grad_threads(D), b = (N + rows - 1) / rows;
  return b < kGradBlocks ? b : kGradBlocks;
}

template <int DT, bool QUANT, bool WHOLE, bool NT>
void norm_shape(const NormArgs& a, hipStream_t stream) {
  constexpr int64_t most = 1 << 21;  // a launch holds below 2^32 work-items
  const int64_t g = (a.D + kG - 1) / kG;
  const int64_t rows = a.N < most ? a.N : most;
  const int64_t rows4 = (a.N + 3) / 4 < most ? (a.N + 3) / 4 : most;
#define VCE_NORM(T, P, R) \
  hipLaunchKernelGGL((k_norm<DT, T, P, QUANT, WHOLE, NT>), dim3((uint32_t)(R)), dim3(T < 256 ? 256 : T), 0, stream, a)
  if (g <= 64) VCE_NORM(64, 1, rows4);
  else if (g <= 128) VCE_NORM(64, 2, rows4);
  else if (g <= 256) VCE_NORM(256, 1, rows);
  else if (g <= 512) VCE_NORM(512, 1, rows);
  else if (g <= 1024) VCE_NORM(512, 2, rows);
  else if (g <= 2048) VCE_NORM(1024, 2, rows);
  else hipLaunchKernelGGL((k_norm_wide<DT, QUANT, WHOLE>), dim3((uint32_t)rows), dim3(1024), 0, stream, a);
#undef VCE_NORM
}

template <int DT, bool WHOLE>
void grad_shape(const NormGradArgs& a, hipStream_t stream) {
  const int64_t g = (a.D + kG - 1) / kG;
  const dim3 grid((uint32_t)grad_blocks(a.N, a.D));
#define VCE_GRAD(T, P) hipLaunchKernelGGL((k_norm_grad<DT, T, P, WHOLE>), grid, dim3(kGradT), 0, stream, a)
  if (g <= 64) VCE_GRAD(64, 1);
  else if (g <= 128) VCE_GRAD(64, 2);
  else if (g <= 256) VCE_GRAD(256, 1);
  else if (g <= 512) VCE_GRAD(512, 1);
  else if (g <= 1024) VCE_GRAD(1024, 1);
  else if (g <= 2048) VCE_GRAD(1024, 2);
  else
    hipLaunchKernelGGL((k_norm_grad_wide<DT, WHOLE>), grid, dim3(1024),
                       (size_t)((g + 1023) / 1024 * 1024 * kG) * 4, stream, a);
#undef VCE_GRAD
}

template <int DT, bool QUANT>
void norm_dt(const NormArgs& a, hipStream_t stream) {
  // more than the chip's L2 (8 x 4 MiB) in one output
  const bool nt = a.N * a.D * VecT<DT>::EB > ((int64_t)32 << 20);
  if (a.D % kG == 0)
    nt ? norm_shape<DT, QUANT, true, true>(a, stream) : norm_shape<DT, QUANT, true, false>(a, stream);
  else
    norm_shape<DT, QUANT, false, false>(a, stream);
}
template <int DT>
void grad_dt(const NormGradArgs& a, hipStream_t stream) {
  a.D % kG == 0 ? grad_shape<DT, true>(a, stream) : grad_shape<DT, false>(a, stream);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
  if (a.N == 0) return hipSuccess;
  if (a.dtype == CE_BF16)
    a.q ? norm_dt<CE_BF16, true>(a, stream) : norm_dt<CE_BF16, false>(a, stream);
  else
    a.q ? norm_dt<CE_F32, true>(a, stream) : norm_dt<CE_F32, false>(a, stream);
  return hipGetLastError();
}

size_t norm_grad_workspace(int64_t N, int64_t D) { return (size_t)grad_blocks(N, D) * (size_t)D * 4u; }

hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t stream) {
  hipError_t e = hipSuccess;
  if (a.N > 0) {
    a.dtype == CE_BF16 ? grad_dt<CE_BF16>(a, stream) : grad_dt<CE_F32>(a, stream);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (a.dweight) {
    hipLaunchKernelGGL(k_norm_dw, dim3((uint32_t)((a.D + kDwCols - 1) / kDwCols)), dim3(kDwCols * kDwRows), 0, stream, a.parts,
                       a.N > 0 ? grad_blocks(a.N, a.D) : (int64_t)0, a.D, a.dweight, a.accumulate);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace vce
