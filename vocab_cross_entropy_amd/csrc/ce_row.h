// Device helpers of the kernels that hold a chunk of one row's logits in
// registers (token log-probabilities, distillation): 16-byte loads at any
// element alignment, maxima, reductions over a workgroup, and the words that the
// chunks of a row exchange.
//
// The exchange is ce_fwd_bwd_fused's: 64-bit words in the workspace, the call's
// tag in the high half and a payload in the low one, written and read with
// relaxed agent-scope atomics.  The tag is the low half of the workspace's epoch,
// which the last workgroup of a call advances, so that words of earlier calls (or
// of another entry point on the same workspace) never pass for this call's and
// nothing is cleared between calls or replays of a captured graph.  Workgroups
// are dispatched in index order and a row's chunks are consecutive, so a chunk
// waits only for workgroups that run or start as soon as a running one ends;
// every wait is bounded.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ce_internal.h"
#include "ce_vec.h"

namespace vce {

constexpr float kLog2e = 1.44269504088896340736f;  // rounded to FP32
constexpr float kLn2f = 0.69314718055994530942f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// A 16-byte vector of logits: E columns.
template <int DT>
struct LogitT;
template <>
struct LogitT<CE_BF16> {
  static constexpr int E = 8, EB = 2;
  static constexpr uint32_t kNegInf = 0xff80ff80u;  // a word of -inf
  typedef u32x4_a2 Word;
};
template <>
struct LogitT<CE_F32> {
  static constexpr int E = 4, EB = 4;
  static constexpr uint32_t kNegInf = 0xff800000u;
  typedef u32x4_a4 Word;
};

template <int DT>
__device__ __forceinline__ void unpack_vec(const u32x4v& v, float (&f)[LogitT<DT>::E]) {
  if constexpr (DT == CE_BF16) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(v[k] << 16);
      f[2 * k + 1] = __uint_as_float(v[k] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = __uint_as_float(v[k]);
  }
}
template <int DT>
__device__ __forceinline__ u32x4v pack_vec(const float (&f)[LogitT<DT>::E]) {
  u32x4v v;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (DT == CE_BF16)
      v[k] = pack2_bf16(f[2 * k], f[2 * k + 1]);
    else
      v[k] = __float_as_uint(f[k]);
  }
  return v;
}
template <int DT>
__device__ __forceinline__ float load_logit(const char* row, int64_t j) {
  if constexpr (DT == CE_BF16)
    return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[j] << 16);
  else
    return reinterpret_cast<const float*>(row)[j];
}
template <int DT>
__device__ __forceinline__ void store_logit(char* row, int64_t j, float g) {
  if constexpr (DT == CE_BF16)
    reinterpret_cast<uint16_t*>(row)[j] = (uint16_t)(pack2_bf16(g, 0.f) & 0xffffu);
  else
    reinterpret_cast<float*>(row)[j] = g;
}

// Register barrier, no instruction: a later sweep unpacks the vector again instead of keeping its floats.
__device__ __forceinline__ void relaunch(u32x4v& v) { asm volatile("" : "+v"(v)); }

// Exponents (x - m) log2 e / T come from one fused multiply-add against m2 = fl(m log2 e / T), whose rounding is
// then taken out of the sums.  Where |m2| exceeds this bound (a row masked with -1e9, or with the type's lowest value) that
// rounding is too large, or m2 not FP32: the vectors hold x - m instead.  It is exact wherever 2^(x - m) is not 0: BF16
// logits beyond 2^8 differ by whole numbers of few bits, FP32 ones by what FP32 holds.
constexpr float kNear = 1024.f;
template <int DT, int P>
__device__ __forceinline__ void subtract(u32x4v (&v)[P], float m) {
#pragma unroll
  for (int j = 0; j < P; ++j) {
    relaunch(v[j]);
    float f[LogitT<DT>::E];
    unpack_vec<DT>(v[j], f);
#pragma unroll
    for (int e = 0; e < LogitT<DT>::E; ++e) f[e] -= m;
    v[j] = pack_vec<DT>(f);
    relaunch(v[j]);
  }
}

// One v_max3_f32 (fmaxf would quiet each operand first).  A quiet NaN loses; a signalling one can take the operands
// before it along.  The sums carry either: where one is NaN, maxima say nothing.
__device__ __forceinline__ float max3_hw(float a, float b, float c) {
  float d;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "v"(c));
  return d;
}
// the largest of m and the vector's columns
template <int DT>
__device__ __forceinline__ float largest(const u32x4v& v, float m) {
  float f[LogitT<DT>::E];
  unpack_vec<DT>(v, f);
#pragma unroll
  for (int k = 0; k < LogitT<DT>::E; k += 2) m = max3_hw(m, f[k], f[k + 1]);
  return m;
}

// The chunk's columns first, first + 1, ... of a vector that is not whole; -inf for those that are not there.
template <int DT>
__device__ __forceinline__ u32x4v partial_vec(const char* chunk, uint32_t first, uint32_t cols) {
  constexpr uint32_t kNone = LogitT<DT>::kNegInf;
  u32x4v v = {kNone, kNone, kNone, kNone};
#pragma unroll
  for (int e = 0; e < LogitT<DT>::E - 1; ++e) {
    if (first + e >= cols) continue;
    if constexpr (DT == CE_BF16) {
      const uint32_t h = reinterpret_cast<const uint16_t*>(chunk)[first + e];
      v[e / 2] = e & 1 ? (v[e / 2] & 0xffffu) | h << 16 : (v[e / 2] & 0xffff0000u) | h;
    } else {
      v[e] = reinterpret_cast<const uint32_t*>(chunk)[first + e];
    }
  }
  return v;
}

// A register chosen at run time (laundered, or the compiler chooses an address and puts the array into scratch memory).
template <int P>
__device__ __forceinline__ u32x4v pick(const u32x4v (&v)[P], uint32_t j) {
  u32x4v w = v[0];
#pragma unroll
  for (int i = 1; i < P; ++i) {
    u32x4v other = v[i];
    relaunch(other);
    if ((uint32_t)i == j) w = other;
  }
  return w;
}

// A chunk of `cols` columns as T x P vectors: vector j * T + tid in slot j of
// thread tid.  load_chunk issues the loads of the whole vectors, none behind a
// branch: slots past them load the chunk's first one.  finish_chunk, the first use of
// the slots, puts in the columns of a last vector that is not whole, and with FILL -inf where there is no column.
template <int DT, int T, int P>
__device__ __forceinline__ void load_chunk(const char* chunk, uint32_t cols, u32x4v (&v)[P]) {
  typedef typename LogitT<DT>::Word Word;
  const uint32_t whole = cols / LogitT<DT>::E;
  if (whole == 0) return;
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const uint32_t i = j * T + threadIdx.x;
    v[j] = __builtin_nontemporal_load(reinterpret_cast<const Word*>(chunk + (i < whole ? i : 0u) * 16u));
  }
}
template <int DT, int T, int P, bool FILL>
__device__ __forceinline__ void finish_chunk(const char* chunk, uint32_t cols, u32x4v (&v)[P]) {
  constexpr int E = LogitT<DT>::E;
  constexpr uint32_t kNone = LogitT<DT>::kNegInf;
  const uint32_t tid = threadIdx.x, whole = cols / E;
  if constexpr (FILL) {
#pragma unroll
    for (int j = 0; j < P; ++j) {
      if ((uint32_t)(j + 1) * T <= whole) continue;  // the same for the whole workgroup
      if (j * T + tid >= whole) v[j] = u32x4v{kNone, kNone, kNone, kNone};
    }
  }
  if (cols % E != 0 && tid == whole % T) {
    const u32x4v w = partial_vec<DT>(chunk, whole * E, cols);
#pragma unroll
    for (int j = 0; j < P; ++j) {
      u32x4v mine = w;
      relaunch(mine);  // (as in pick)
      if ((uint32_t)j == whole / T) v[j] = mine;
    }
  }
}

// A chunk of `cols` columns from load_chunk's slots, `of(vector)` for each vector, written non-temporally; columns
// that are not there are left out.
template <int DT, int T, int P, typename Of>
__device__ __forceinline__ void store_chunk(char* chunk, uint32_t cols, u32x4v (&v)[P], Of of) {
  typedef typename LogitT<DT>::Word Word;
  constexpr int E = LogitT<DT>::E;
  uint32_t tid = threadIdx.x;
  asm volatile("" : "+v"(tid));  // the offsets are formed here, not kept from the loads
  const uint32_t whole = cols / E;
#pragma unroll
  for (int j = 0; j < P; ++j) {
    relaunch(v[j]);
    const uint32_t i = j * T + tid;
    const u32x4v w = of(v[j]);
    if (i < whole) __builtin_nontemporal_store(w, reinterpret_cast<Word*>(chunk + i * 16u));
  }
  if (cols % E != 0 && tid == whole % T) {
    const u32x4v w = of(pick<P>(v, whole / T));
#pragma unroll
    for (int e = 0; e < E - 1; ++e) {
      if (whole * E + e >= cols) continue;
      if constexpr (DT == CE_BF16)
        reinterpret_cast<uint16_t*>(chunk)[whole * E + e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
      else
        reinterpret_cast<uint32_t*>(chunk)[whole * E + e] = w[e];
    }
  }
}

// ---- reductions, in a fixed order

template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ float dpp_or_own(float v) {  // lanes without a source, and rows outside ROWS, read their own
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(v), __float_as_int(v), CTRL, ROWS, 0xf, false));
}
// the largest over the wave, of any sign, uniform
__device__ __forceinline__ float wave_largest(float v) {
  v = fmaxf(v, dpp_or_own<kSwap1>(v));
  v = fmaxf(v, dpp_or_own<kSwap2>(v));
  v = fmaxf(v, dpp_or_own<kHalfMirror>(v));
  v = fmaxf(v, dpp_or_own<kMirror>(v));
  v = fmaxf(v, dpp_or_own<kBcast15, 0xa>(v));
  v = fmaxf(v, dpp_or_own<kBcast31, 0xc>(v));
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
// the bits set in any lane, uniform
__device__ __forceinline__ uint32_t wave_or(uint32_t v) {
  v |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kSwap1, 0xf, 0xf, true);
  v |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kSwap2, 0xf, 0xf, true);
  v |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kHalfMirror, 0xf, 0xf, true);
  v |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kMirror, 0xf, 0xf, true);
  v |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kBcast15, 0xa, 0xf, true);
  v |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kBcast31, 0xc, 0xf, true);
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
// the same of 64-bit values (a shuffle goes through LDS, twice for a double)
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ double dpp64(double v, double none) {  // `none` for lanes without a source, and outside ROWS
  typedef int i2 __attribute__((ext_vector_type(2)));
  const i2 w = __builtin_bit_cast(i2, v), o = __builtin_bit_cast(i2, none);
  const i2 r = {__builtin_amdgcn_update_dpp(o.x, w.x, CTRL, ROWS, 0xf, false),
                __builtin_amdgcn_update_dpp(o.y, w.y, CTRL, ROWS, 0xf, false)};
  return __builtin_bit_cast(double, r);
}
__device__ __forceinline__ double last_lane64(double v) {
  typedef int i2 __attribute__((ext_vector_type(2)));
  const i2 w = __builtin_bit_cast(i2, v);
  const i2 r = {__builtin_amdgcn_readlane(w.x, 63), __builtin_amdgcn_readlane(w.y, 63)};
  return __builtin_bit_cast(double, r);
}
__device__ __forceinline__ double wave_sum64(double v) {
  v += dpp64<kSwap1>(v, 0.0);
  v += dpp64<kSwap2>(v, 0.0);
  v += dpp64<kHalfMirror>(v, 0.0);
  v += dpp64<kMirror>(v, 0.0);
  v += dpp64<kBcast15, 0xa>(v, 0.0);
  v += dpp64<kBcast31, 0xc>(v, 0.0);
  return last_lane64(v);
}
__device__ __forceinline__ int wave_count64(int v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// ---- the exchange

constexpr uint32_t kWaitLimit = 1u << 22;  // polls of one lane, about 128 cycles each

__device__ __forceinline__ void put_word(unsigned long long* p, uint32_t tag, uint32_t payload) {
  __hip_atomic_store(p, ((unsigned long long)tag << 32) | payload, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ unsigned long long peek_word(const unsigned long long* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// The payload of *p once it carries the tag; `w` is a first reading of it.  False
// where the wait was given up.  `spins` is the lane's over all of its waits.
__device__ __forceinline__ bool await_word(const unsigned long long* p, uint32_t tag, unsigned long long w,
                                           uint32_t& spins, uint32_t* payload) {
  while ((uint32_t)(w >> 32) != tag) {
    if (++spins > kWaitLimit) return false;
    __builtin_amdgcn_s_sleep(2);
    w = peek_word(p);
  }
  *payload = (uint32_t)w;
  return true;
}

// A word that nothing writes during the launch, by a scalar load: it takes no place in the order of the vector loads.
template <typename T>
__device__ __forceinline__ T load_uniform(const T* p) {
  typedef const __attribute__((address_space(4))) T* Const;
  return *(Const)p;
}

// A call's view of its workspace: the tag, whether ce_workspace_init prepared it
// for this many bytes, and the test hook (a chunk whose words stay unpublished).
// Scalar loads: nothing writes the record before the call's last workgroup ends.
struct WsView {
  uint32_t tag;
  bool ok;
  unsigned long long withhold;
};
__device__ __forceinline__ WsView view_workspace(const WsHeader* hdr, unsigned long long bytes) {
  const unsigned long long* const rec = &hdr->magic;  // magic, init_bytes, epoch, withhold
  WsView v;
  v.tag = (uint32_t)load_uniform(rec + 2);
  v.ok = (load_uniform(rec) == kWsMagic) & (load_uniform(rec + 1) >= bytes);
  v.withhold = load_uniform(rec + 3);
  return v;
}
__device__ __forceinline__ bool withheld(const WsView& ws, int64_t r, int k) {
  return ws.withhold == ((((unsigned long long)r + 1u) << 8) | (unsigned)k);
}
// The next call's tag; the caller has seen a word of every row that this call's
// workgroups have read the epoch.
__device__ __forceinline__ void next_epoch(WsHeader* hdr) {
  unsigned long long next = hdr->epoch + 1;
  if ((uint32_t)next == 0u) ++next;
  __hip_atomic_store(&hdr->epoch, next, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

}  // namespace vce
