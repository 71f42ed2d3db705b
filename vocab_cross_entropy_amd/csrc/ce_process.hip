// Logit processing: penalties for repeated tokens, bias, grammar mask and
// temperature in one pass over the logits, and its gradient.
//
// For row r and column j, with c the occurrences of j in the row's output
// history and `seen` its presence in prompt or output:
//   v = seen ? (x > 0 ? x / theta : x theta) : x
//   z = (v - f c - p [c > 0] + b_j) / T, -inf where the mask's bit is 0
//   dx = dz (seen ? (x > 0 ? 1 / theta : theta) : 1) / T, 0 where masked
// 1 / T is rounded once per row and multiplied in, so z carries one FP32
// rounding more than the division would give (2^-24 relative); the penalty, of
// few columns, is a true division.
//
// Bound: one read and one write of the logits.  What the penalties need from
// the history is a count per column.  A workgroup owns a chunk of one row's
// columns and keeps the chunk's counts in LDS: it reads the row's history
// (from L2: every chunk of the row reads it), adds the tokens that fall into
// its chunk with integer LDS atomics (whose order cannot change the result),
// and then streams its columns once.  Counts take 16 bits with the prompt
// flag in the top one while the history holds at most 32767 tokens, and 32 bits
// beyond.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ce_internal.h"
#include "ce_vec.h"

namespace vce {
namespace {

constexpr int kProcT = 256;
constexpr int kProcSpan = kProcT * kG;  // columns one step of a workgroup covers

constexpr int64_t kProcMaxGrid = 1 << 23;

enum { kHistNone = 0, kHist16 = 1, kHist32 = 2 };

template <int HIST>
struct CountT {
  typedef uint16_t Word;
};
template <>
struct CountT<kHist32> {
  typedef uint32_t Word;
};

template <int DT, int HIST, bool BWD>
__device__ __forceinline__ void process_item(const ProcessArgs& a, int64_t r, uint32_t chunk, char* smem) {
  const int64_t i0 = r / a.d1, i1 = r - i0 * a.d1;
  const int64_t lo = (int64_t)chunk * a.chunk_cols;
  const int64_t hi = lo + a.chunk_cols < a.V ? lo + a.chunk_cols : a.V;
  constexpr int EB = VecT<DT>::EB;
  const char* x = a.x + (i0 * a.s0 + i1 * a.s1) * EB;
  char* z = a.z + (i0 * a.zs0 + i1 * a.zs1) * EB;
  const int tid = (int)threadIdx.x;

  if constexpr (HIST != kHistNone) {
    constexpr int per16 = HIST == kHist16 ? 8 : 4;
    const int words = (int)((hi - lo + per16 - 1) / per16);
    // whole groups are read below: clear the last group's end too
    const int clear = HIST == kHist32 ? (words + 1) & ~1 : words;
    for (int i = tid; i < clear; i += kProcT) reinterpret_cast<u32x4v*>(smem)[i] = u32x4v{0u, 0u, 0u, 0u};
    __syncthreads();
    const int64_t* h = a.hist + i0 * a.hs0 + i1 * a.hs1;
    int64_t n = a.hist_max;
    if (a.hist_len) {
      n = a.hist_len[r];
      n = n < 0 ? 0 : n > a.hist_max ? a.hist_max : n;
    }
    const int64_t np = a.prompt_len ? a.prompt_len[r] : 0;
    const uint64_t first = (uint64_t)(a.vocab_start + lo);
    uint32_t* tab = reinterpret_cast<uint32_t*>(smem);
    for (int64_t i = tid; i < n; i += kProcT) {
      // a token of another chunk or vocabulary shard, or no token at all (negative), wraps to or past the end
      const uint64_t j = (uint64_t)h[i] - first;
      if (j >= (uint64_t)(hi - lo)) continue;
      if constexpr (HIST == kHist16) {
        const int sh = 16 * ((int)j & 1);
        if (i < np)
          atomicOr(&tab[j >> 1], 0x8000u << sh);
        else
          atomicAdd(&tab[j >> 1], 1u << sh);
      } else {
        if (i < np)
          atomicOr(&tab[j], 0x80000000u);
        else
          atomicAdd(&tab[j], 1u);
      }
    }
    __syncthreads();
  }

  const float theta = a.repetition ? a.repetition[r] : 1.f;
  const float fr = a.frequency ? a.frequency[r] : 0.f;
  const float pr = a.presence ? a.presence[r] : 0.f;
  const float rt = a.temperature ? 1.f / a.temperature[r] : 1.f;
  const uint8_t* mask = a.mask ? reinterpret_cast<const uint8_t*>(a.mask + i0 * a.ms0 + i1 * a.ms1) : nullptr;
  const float* bias = a.bias ? a.bias + i0 * a.bs0 + i1 * a.bs1 : nullptr;
  uint8_t* signs = a.signs ? a.signs + r * a.signs_ld : nullptr;

  for (int64_t j = lo + (int64_t)tid * kG; j < hi; j += kProcSpan) {
    float v[kG];
    const Raw<DT> raw = load_group<DT, true>(x, j, a.V);
    raw_to_f32<DT>(raw, v);
    if constexpr (!BWD) {
      if (signs) {
        uint32_t up = 0;
#pragma unroll
        for (int e = 0; e < kG; ++e) up |= (v[e] > 0.f ? 1u : 0u) << e;  // columns past the end hold 0
        signs[j >> 3] = (uint8_t)up;
      }
    }
    if constexpr (HIST != kHistNone) {
      uint32_t c[kG];
      bool any;
      if constexpr (HIST == kHist16) {
        const u32x4v w = reinterpret_cast<const u32x4v*>(smem)[(j - lo) >> 3];
        any = (w.x | w.y | w.z | w.w) != 0u;
#pragma unroll
        for (int e = 0; e < kG; ++e) {
          const uint32_t h16 = (w[e / 2] >> (16 * (e & 1))) & 0xffffu;
          c[e] = (h16 & 0x7fffu) | ((h16 & 0x8000u) << 16);
        }
      } else {
        const u32x4v w0 = reinterpret_cast<const u32x4v*>(smem)[(j - lo) >> 2];
        const u32x4v w1 = reinterpret_cast<const u32x4v*>(smem)[((j - lo) >> 2) + 1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          c[e] = w0[e];
          c[e + 4] = w1[e];
        }
        any = (w0.x | w0.y | w0.z | w0.w | w1.x | w1.y | w1.z | w1.w) != 0u;
      }
      if (any) {
        uint32_t up = 0;
        if constexpr (BWD) up = signs ? signs[j >> 3] : 0u;
#pragma unroll
        for (int e = 0; e < kG; ++e) {
          if (c[e] != 0u) {
            const bool pos = BWD ? (up >> e) & 1u : v[e] > 0.f;
            v[e] = pos ? v[e] / theta : v[e] * theta;
            if constexpr (!BWD) {
              const uint32_t n = c[e] & 0x7fffffffu;
              v[e] = __builtin_fmaf(-fr, (float)n, v[e]) - (n ? pr : 0.f);
            }
          }
        }
      }
    }
    if constexpr (!BWD) {
      if (bias) {
        float b[kG];
        load_f32<CE_F32>(reinterpret_cast<const char*>(bias), j, a.V, b);
#pragma unroll
        for (int e = 0; e < kG; ++e) v[e] += b[e];
      }
    }
#pragma unroll
    for (int e = 0; e < kG; ++e) v[e] *= rt;
    if (mask) {
      const uint32_t m = mask[j >> 3];
      const float off = BWD ? 0.f : -__builtin_inff();
#pragma unroll
      for (int e = 0; e < kG; ++e) v[e] = (m >> e) & 1u ? v[e] : off;
    }
    store_group<DT, true>(z, j, a.V, f32_to_raw<DT>(v));
  }
}

template <int DT, int HIST, bool BWD>
__global__ __launch_bounds__(kProcT) void k_process(ProcessArgs a) {
  extern __shared__ __align__(16) char smem[];
  const int64_t items = a.N * a.chunks;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t r = it / a.chunks;
    if constexpr (HIST != kHistNone) __syncthreads();  // the last item's counts have been read
    process_item<DT, HIST, BWD>(a, r, (uint32_t)(it - r * a.chunks), smem);
  }
}

template <int DT, bool BWD>
hipError_t launch_dt(const ProcessArgs& a, int hist, dim3 grid, hipStream_t stream) {
  const size_t col = (size_t)((a.chunk_cols + 7) & ~(int64_t)7);
  switch (hist) {
    case kHistNone:
      hipLaunchKernelGGL((k_process<DT, kHistNone, BWD>), grid, dim3(kProcT), 0, stream, a);
      break;
    case kHist16:
      hipLaunchKernelGGL((k_process<DT, kHist16, BWD>), grid, dim3(kProcT), col * 2, stream, a);
      break;
    default:
      hipLaunchKernelGGL((k_process<DT, kHist32, BWD>), grid, dim3(kProcT), col * 4, stream, a);
      break;
  }
  return hipGetLastError();
}

}  // namespace

void process_plan(ProcessArgs* a) {
  const int64_t cols = 8192;
  a->chunk_cols = cols;
  a->chunks = (a->V + cols - 1) / cols;
}

hipError_t launch_process(const ProcessArgs& a, bool backward, hipStream_t stream, hipEvent_t ev0, hipEvent_t ev1) {
  hipError_t e = hipSuccess;
  if (ev0 && (e = hipEventRecord(ev0, stream)) != hipSuccess) return e;
  const int hist = !a.hist || a.hist_max == 0 ? kHistNone : a.hist_max <= 32767 ? kHist16 : kHist32;
  // a launch holds below 2^32 work-items, so beyond that a workgroup takes several items
  const int64_t items = a.N * a.chunks;
  const dim3 grid((uint32_t)(items < kProcMaxGrid ? items : kProcMaxGrid));
  if (a.dtype == CE_BF16)
    e = backward ? launch_dt<CE_BF16, true>(a, hist, grid, stream) : launch_dt<CE_BF16, false>(a, hist, grid, stream);
  else
    e = backward ? launch_dt<CE_F32, true>(a, hist, grid, stream) : launch_dt<CE_F32, false>(a, hist, grid, stream);
  if (e != hipSuccess) return e;
  if (ev1) e = hipEventRecord(ev1, stream);
  return e;
}

}  // namespace vce
