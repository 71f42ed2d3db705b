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
// columns: it issues the loads of all its columns, counts the row's tokens that
// fall into the chunk in LDS (integer atomics, whose order cannot change the
// result) while the columns arrive, and then processes and writes them.  Every
// chunk of a row reads the row's history, from L2.  Counts take 16 bits with the
// prompt flag in the top one while the history holds at most 32767 tokens, and 32
// bits beyond.  8192 x 128000 BF16 with the prefixes of 2048 tokens: 738 us, 5.7
// TB/s of the 6.0 that a copy reaches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ce_internal.h"
#include "ce_vec.h"

namespace vce {
namespace {

constexpr int64_t kProcMaxGrid = 1 << 22;

enum { kHistNone = 0, kHist16 = 1, kHist32 = 2 };
constexpr int kHistStep = 4;  // tokens per thread in flight

template <int HIST>
__device__ __forceinline__ void count_token(uint32_t* tab, uint64_t id, uint64_t first, uint32_t cols, bool prompt) {
  // a token of another chunk or vocabulary shard, or no token at all (negative), wraps to or past the end
  const uint64_t j = id - first;
  if (j >= cols) return;
  if constexpr (HIST == kHist16) {
    const int sh = 16 * ((int)j & 1);
    if (prompt)
      atomicOr(&tab[j >> 1], 0x8000u << sh);
    else
      atomicAdd(&tab[j >> 1], 1u << sh);
  } else {
    if (prompt)
      atomicOr(&tab[j], 0x80000000u);
    else
      atomicAdd(&tab[j], 1u);
  }
}

// Which of eight columns have a count, as bits: column 2 k in bit k, column
// 2 k + 1 in bit 16 + k.
template <int HIST>
__device__ __forceinline__ uint32_t seen_columns(const char* tab, uint32_t col) {
  uint32_t seen = 0;
  if constexpr (HIST == kHist16) {
    const u32x4v w = reinterpret_cast<const u32x4v*>(tab)[col >> 3];
    if ((w.x | w.y | w.z | w.w) == 0u) return 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k)  // the top bit of each half that is not 0
      seen |= ((((w[k] & 0x7fff7fffu) + 0x7fff7fffu) | w[k]) & 0x80008000u) >> (15 - k);
  } else {
    const u32x4v w0 = reinterpret_cast<const u32x4v*>(tab)[col >> 2];
    const u32x4v w1 = reinterpret_cast<const u32x4v*>(tab)[(col >> 2) + 1];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      seen |= (w0[2 * k] ? 1u : 0u) << k | (w0[2 * k + 1] ? 1u : 0u) << (16 + k);
      seen |= (w1[2 * k] ? 1u : 0u) << (2 + k) | (w1[2 * k + 1] ? 1u : 0u) << (18 + k);
    }
  }
  return seen;
}
// A column's occurrences in the output (the count without the prompt flag)
template <int HIST>
__device__ __forceinline__ uint32_t occurrences(const char* tab, uint32_t col) {
  if constexpr (HIST == kHist16)
    return reinterpret_cast<const uint16_t*>(tab)[col] & 0x7fffu;
  else
    return reinterpret_cast<const uint32_t*>(tab)[col] & 0x7fffffffu;
}

// FP32: a lane's eight columns are two 16-byte words, and lanes reading their own
// would leave holes that a second access of the same lines fills.  So a wave reads
// (and writes) its 512 columns as two runs of 256, four columns a lane, and
// neighbouring lanes swap halves: the even one ends up with eight columns of the
// first run, the odd one of the second.  It is its own inverse.
__device__ __forceinline__ void swap_halves(u32x4v (&w)[2]) {
  const bool odd = threadIdx.x & 1;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int got = __builtin_amdgcn_update_dpp(0, (int)(odd ? w[0][e] : w[1][e]), kSwap1, 0xf, 0xf, true);
    w[0][e] = odd ? (uint32_t)got : w[0][e];
    w[1][e] = odd ? w[1][e] : (uint32_t)got;
  }
}

// One chunk: U groups of eight columns for each of T threads.
template <int DT, int HIST, bool BWD, int T, int U>
__device__ __forceinline__ void process_item(const ProcessArgs& a, uint32_t r, uint32_t chunk, char* smem) {
  constexpr int EB = VecT<DT>::EB;
  const int64_t i0 = r / (uint32_t)a.d1, i1 = r % (uint32_t)a.d1;
  const uint32_t V = (uint32_t)a.V;
  const uint32_t lo = chunk * (uint32_t)a.chunk_cols;
  const uint32_t hi = V - lo < (uint32_t)a.chunk_cols ? V : lo + (uint32_t)a.chunk_cols;
  const uint32_t tid = threadIdx.x;
  const char* x = a.x + (i0 * a.s0 + i1 * a.s1) * EB;
  char* z = a.z + (i0 * a.zs0 + i1 * a.zs1) * EB;

  // this thread's group in step u, and where its wave's 512 columns start
  const uint32_t lane = tid & 63, wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(tid >> 6));
  const auto start = [=](int u) { return lo + u * T * kG + wave * 512; };
  const auto column = [=](int u) {
    return DT == CE_F32 ? start(u) + (lane & 1) * 256 + (lane >> 1) * kG : lo + (u * T + tid) * kG;
  };
  // FP32: whether the wave reads runs and swaps (all of its columns are there)
  const auto runs = [=](int u) { return DT == CE_F32 && start(u) + 512 <= hi; };
  Raw<DT> raw[U];
  const uint32_t whole = V & ~7u;  // columns in whole groups
  if (whole) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (DT == CE_F32) {
        const uint32_t j = column(u) < whole ? column(u) : 0;
        raw[u].w[0] = fetch_quad<CE_F32>(x, runs(u) ? start(u) + lane * 4 : j);
        raw[u].w[1] = fetch_quad<CE_F32>(x, runs(u) ? start(u) + 256 + lane * 4 : j + 4);
      } else {
        raw[u] = fetch_whole<DT>(x, column(u), whole);
      }
    }
  }
  const uint8_t* mask = a.mask ? reinterpret_cast<const uint8_t*>(a.mask + i0 * a.ms0 + i1 * a.ms1) : nullptr;
  uint8_t* signs = a.signs ? a.signs + (int64_t)r * a.signs_ld : nullptr;
  // the groups' mask bits and signs, a byte each, go out with the columns (4096 x 32000 BF16: 107 against 125 us, the
  // gradient 106 against 141; FP32 195 against 200 and 197 against 211)
  uint32_t allowed[U], up[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t j = column(u), at = (j < hi ? j : lo) >> 3;
    allowed[u] = mask ? mask[at] : 0u;
    up[u] = BWD && HIST != kHistNone && signs ? signs[at] : 0u;
  }
  const float theta = a.repetition ? a.repetition[r] : 1.f;
  const float fr = a.frequency ? a.frequency[r] : 0.f;
  const float pr = a.presence ? a.presence[r] : 0.f;
  const float rt = a.temperature ? 1.f / a.temperature[r] : 1.f;
  const float* bias = a.bias ? a.bias + i0 * a.bs0 + i1 * a.bs1 : nullptr;

  if constexpr (HIST != kHistNone) {
    const int64_t* h = a.hist + i0 * a.hs0 + i1 * a.hs1;
    uint32_t n = (uint32_t)a.hist_max;
    if (a.hist_len) {
      const int32_t len = a.hist_len[r];
      n = len < 0 ? 0u : min((uint32_t)len, n);
    }
    const int32_t plen = a.prompt_len ? a.prompt_len[r] : 0;
    const uint32_t np = plen < 0 ? 0u : (uint32_t)plen;
    // the chunk's counts, in whole groups
    const uint32_t words = (hi - lo + kG - 1) / kG * (HIST == kHist16 ? 1 : 2);
    for (uint32_t i = tid; i < words; i += T) reinterpret_cast<u32x4v*>(smem)[i] = u32x4v{0u, 0u, 0u, 0u};
    uint32_t* tab = reinterpret_cast<uint32_t*>(smem);
    const uint64_t first = (uint64_t)a.vocab_start + lo;
    for (uint32_t base = 0; base < n; base += kHistStep * T) {
      uint64_t id[kHistStep];
#pragma unroll
      for (int k = 0; k < kHistStep; ++k) {
        const uint32_t i = base + tid + k * T;
        id[k] = (uint64_t)h[i < n ? i : n - 1];  // without a branch, so that all are in flight
      }
      if (base == 0) __syncthreads();  // the table is clear
#pragma unroll
      for (int k = 0; k < kHistStep; ++k) {
        const uint32_t i = base + tid + k * T;
        if (i < n) count_token<HIST>(tab, id[k], first, hi - lo, i < np);
      }
    }
    __syncthreads();
  }

#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t j = column(u);
    if constexpr (DT == CE_F32) {
      if (runs(u)) swap_halves(raw[u].w);
    }
    if (j >= hi) continue;
    fix_tail<DT>(raw[u], x, j, whole, V);
    float v[kG];
    raw_to_f32<DT>(raw[u], v);
    if constexpr (!BWD) {
      if (signs) {
        uint32_t bits = 0;
#pragma unroll
        for (int e = 0; e < kG; ++e) bits |= (v[e] > 0.f ? 1u : 0u) << e;  // columns past the end hold 0
        signs[j >> 3] = (uint8_t)bits;
      }
    }
    if constexpr (HIST != kHistNone) {
      // one seen column of each lane at a time: many waves have a lane with one, few lanes have two
      uint32_t seen = seen_columns<HIST>(smem, j - lo);
      while (seen) {
        const uint32_t bit = (uint32_t)__builtin_ctz(seen);
        seen &= seen - 1;
        const uint32_t e = (bit & 15u) * 2 + (bit >> 4);
        float t = v[0];
#pragma unroll
        for (uint32_t k = 1; k < kG; ++k) t = e == k ? v[k] : t;
        const bool pos = BWD ? (up[u] >> e) & 1u : t > 0.f;
        t = pos ? t / theta : t * theta;
        if constexpr (!BWD) {
          const uint32_t n = occurrences<HIST>(smem, j - lo + e);
          t = __builtin_fmaf(-fr, (float)n, t) - (n ? pr : 0.f);
        }
#pragma unroll
        for (uint32_t k = 0; k < kG; ++k) v[k] = e == k ? t : v[k];
      }
    }
    if constexpr (!BWD) {
      if (bias) {
        float b[kG];
        load_f32<CE_F32>(reinterpret_cast<const char*>(bias), j, V, b);
#pragma unroll
        for (int e = 0; e < kG; ++e) v[e] += b[e];
      }
    }
#pragma unroll
    for (int e = 0; e < kG; ++e) v[e] *= rt;
    if (mask) {
      const float off = BWD ? 0.f : -__builtin_inff();
#pragma unroll
      for (int e = 0; e < kG; ++e) v[e] = (allowed[u] >> e) & 1u ? v[e] : off;
    }
    Raw<DT> out = f32_to_raw<DT>(v);
    if constexpr (DT == CE_F32) {
      if (runs(u)) {
        swap_halves(out.w);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          __builtin_nontemporal_store(out.w[h], reinterpret_cast<u32x4_a4*>(z + (start(u) + h * 256 + lane * 4) * 4));
        continue;
      }
    }
    store_group<DT, true>(z, j, V, out);
  }
}

template <int DT, int HIST, bool BWD, int T, int U>
__global__ __launch_bounds__(T) void k_process(ProcessArgs a) {
  __shared__ __align__(16) char smem[HIST == kHistNone ? 16 : T * U * kG * (HIST == kHist16 ? 2 : 4)];
  // (32-bit divisions: 64-bit ones delay the first load by hundreds of cycles)
  const uint32_t chunks = (uint32_t)a.chunks, items = (uint32_t)a.N * chunks;
  for (uint32_t it = blockIdx.x; it < items; it += gridDim.x) {
    const uint32_t r = it / chunks;
    if constexpr (HIST != kHistNone) __syncthreads();  // the last item's counts have been read
    // a row's chunks in an order that shifts from row to row: workgroups go to the 8 XCDs in turn, and with 8 chunks a
    // row one XCD would get the chunk of the frequent tokens of every row (8192 x 128000 BF16: 858 us)
    process_item<DT, HIST, BWD, T, U>(a, r, (it + r % chunks) % chunks, smem);
    if (items - it <= gridDim.x) break;
  }
}

// Chunk shapes (threads, groups per thread); process_plan chooses
struct ProcShape {
  int t, u;
};
constexpr ProcShape kProcMany = {256, 4}, kProcSome = {512, 4}, kProcFew = {256, 1};

template <int DT, int HIST, bool BWD>
hipError_t launch_shape(const ProcessArgs& a, dim3 grid, hipStream_t stream) {
#define VCE_PROC(S) hipLaunchKernelGGL((k_process<DT, HIST, BWD, S.t, S.u>), grid, dim3(S.t), 0, stream, a)
  if (a.shape == 0) VCE_PROC(kProcMany);
  else if (a.shape == 1) VCE_PROC(kProcSome);
  else VCE_PROC(kProcFew);
#undef VCE_PROC
  return hipGetLastError();
}
template <int DT, bool BWD>
hipError_t launch_dt(const ProcessArgs& a, int hist, dim3 grid, hipStream_t stream) {
  return hist == kHistNone ? launch_shape<DT, kHistNone, BWD>(a, grid, stream)
         : hist == kHist16 ? launch_shape<DT, kHist16, BWD>(a, grid, stream)
                           : launch_shape<DT, kHist32, BWD>(a, grid, stream);
}

}  // namespace

void process_plan(ProcessArgs* a) {
  // Many rows: 8192-column chunks by 256 threads, the fastest stream (8192 x 128000 BF16: 741 us, 818 by 512 threads
  // on 16384 columns; around the limit of 8192 items either is ahead by up to a tenth).  Some: 512 threads, which count a
  // long history in half the steps and read it less often (64 x 128000 FP32 with up to 4096 tokens: 16.2 us, 20.0 in
  // 2048-column chunks).  The limit of 512 items is on the high side: with a history, 256 items and more are faster by
  // 512 threads too (63 x 128000 FP32: 19.7 against 16.1 us), without one they are not (126 x 50257 FP32: 10.3 against
  // 11.1).  Few, or of few columns: 2048-column chunks, for workgroups enough and few idle threads (5600 x 500 BF16: 19
  // us, 36 by 512 threads).
  const auto items = [a](ProcShape s) {
    const int64_t cols = (int64_t)s.t * s.u * kG;
    return a->N * ((a->V + cols - 1) / cols);
  };
  const bool one_chunk = a->V <= kProcMany.t * kProcMany.u * kG;  // a row of it
  a->shape = a->V <= kProcFew.t * kProcFew.u * kG                 ? 2
             : items(kProcMany) >= (one_chunk ? 512 : 8192)       ? 0
             : items(kProcSome) >= 512                            ? 1
                                                                  : 2;
  const ProcShape s = a->shape == 0 ? kProcMany : a->shape == 1 ? kProcSome : kProcFew;
  const int64_t most = (int64_t)s.t * s.u * kG;
  a->chunks = (a->V + most - 1) / most;
  a->chunk_cols = ((a->V + a->chunks - 1) / a->chunks + kG - 1) / kG * kG;  // even shares of whole groups
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
