// Device helpers shared by the kernels around the loss (logit processing,
// embedding, RMS norm): groups of eight columns at any element alignment, and
// sums over a wave or a workgroup.
//
// A row is walked in groups of eight columns that start at multiples of eight
// whatever the row's address, so that per-column side data (mask bits, count
// words, scale groups) lines up with the groups.  gfx950 serves 16-byte global
// accesses at any alignment, so a row that starts off a 16-byte boundary takes
// the same instructions as an aligned one, with more cache lines per access.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ce.h"

namespace vce {

constexpr int kG = 8;  // columns per group

typedef unsigned u32x4v __attribute__((ext_vector_type(4)));
// the same 16 bytes at element alignment
typedef u32x4v u32x4_a2 __attribute__((aligned(2)));
typedef u32x4v u32x4_a4 __attribute__((aligned(4)));

template <int DT>
struct VecT;
template <>
struct VecT<CE_BF16> {
  static constexpr int EB = 2;
  static constexpr int NV = 1;  // 16-byte words per group
  typedef u32x4_a2 Word;
};
template <>
struct VecT<CE_F32> {
  static constexpr int EB = 4;
  static constexpr int NV = 2;
  typedef u32x4_a4 Word;
};

// eight columns as loaded
template <int DT>
struct Raw {
  u32x4v w[VecT<DT>::NV];
};

// Four columns at element alignment, as FP32.  A wave whose lanes take four FP32
// columns each covers 1 KiB without holes, where groups of eight leave every other
// 16 bytes to a second access of the same lines.
template <int DT>
__device__ __forceinline__ void quad_to_f32(const u32x4v& w, float (&f)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    f[k] = __uint_as_float(DT == CE_F32 ? w[k] : k & 1 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
}
template <int DT, bool NT = false>
__device__ __forceinline__ u32x4v fetch_quad(const char* row, uint32_t j) {
  if constexpr (DT == CE_F32) {
    const u32x4_a4* p = reinterpret_cast<const u32x4_a4*>(row + j * 4);
    if constexpr (NT) return __builtin_nontemporal_load(p);
    else return *p;
  } else {
    typedef unsigned u32x2v __attribute__((ext_vector_type(2)));
    typedef u32x2v u32x2_a2 __attribute__((aligned(2)));
    const u32x2_a2* p = reinterpret_cast<const u32x2_a2*>(row + j * 2);
    u32x2v v;
    if constexpr (NT) v = __builtin_nontemporal_load(p);
    else v = *p;
    return u32x4v{v.x, v.y, 0u, 0u};
  }
}
// the columns of a row's last quad that are there, zeros for the others
template <int DT>
__device__ __forceinline__ u32x4v partial_quad(const char* row, uint32_t j, uint32_t cols) {
  u32x4v r = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 3; ++e)
    if (j + e < cols) {
      if constexpr (DT == CE_F32)
        r[e] = reinterpret_cast<const uint32_t*>(row)[j + e];
      else
        r[e / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(row)[j + e] << (16 * (e & 1));
    }
  return r;
}
template <bool NT = false>
__device__ __forceinline__ void store_quad(float* row, uint32_t j, uint32_t cols, const float (&f)[4]) {
  if (j + 4 <= cols) {
    const u32x4v w = {__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
    u32x4_a4* p = reinterpret_cast<u32x4_a4*>(row + j);
    if constexpr (NT) __builtin_nontemporal_store(w, p);
    else *p = w;
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (j + e < cols) row[j + e] = f[e];
  }
}

__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  f2 in = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(in, b2));
}

template <int DT>
__device__ __forceinline__ void raw_to_f32(const Raw<DT>& r, float (&f)[kG]) {
  if constexpr (DT == CE_BF16) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(r.w[0][k] << 16);
      f[2 * k + 1] = __uint_as_float(r.w[0][k] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int k = 0; k < kG; ++k) f[k] = __uint_as_float(r.w[k / 4][k % 4]);
  }
}

template <int DT>
__device__ __forceinline__ Raw<DT> f32_to_raw(const float (&f)[kG]) {
  Raw<DT> r;
  if constexpr (DT == CE_BF16) {
#pragma unroll
    for (int k = 0; k < 4; ++k) r.w[0][k] = pack2_bf16(f[2 * k], f[2 * k + 1]);
  } else {
#pragma unroll
    for (int k = 0; k < kG; ++k) r.w[k / 4][k % 4] = __float_as_uint(f[k]);
  }
  return r;
}

// Columns j .. j + 7 of a row of `cols` columns; those past the row's end read
// as zero and are never touched in memory.  NT sets the non-temporal bit, for
// data that is touched once.  Columns are uint32_t (a row is below 4 GiB): with a
// uniform row pointer an access is then one scalar base and one offset register.
template <int DT, bool NT = false>
__device__ __forceinline__ Raw<DT> load_group(const char* row, uint32_t j, uint32_t cols) {
  typedef typename VecT<DT>::Word Word;
  Raw<DT> r;
  if (j + kG <= cols) {
#pragma unroll
    for (int k = 0; k < VecT<DT>::NV; ++k) {
      const Word* p = reinterpret_cast<const Word*>(row + j * VecT<DT>::EB) + k;
      if constexpr (NT)
        r.w[k] = __builtin_nontemporal_load(p);
      else
        r.w[k] = *p;
    }
  } else {
#pragma unroll
    for (int k = 0; k < VecT<DT>::NV; ++k) r.w[k] = u32x4v{0u, 0u, 0u, 0u};
    // a loop over the elements that are there, with every index a constant
    // (registers cannot be indexed)
#pragma unroll
    for (int e = 0; e < kG - 1; ++e) {
      if (j + e < cols) {
        if constexpr (DT == CE_BF16)
          r.w[0][e / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(row)[j + e] << (16 * (e & 1));
        else
          r.w[e / 4][e % 4] = reinterpret_cast<const uint32_t*>(row)[j + e];
      }
    }
  }
  return r;
}

// The same in two steps, for many loads in flight: fetch_whole reads a group of
// the first `whole` columns (cols rounded down to groups; at least one group),
// lanes past them some other one, so that no load stands behind a branch;
// fix_tail then reads the row's partial group where a lane has it.  Lanes past
// the row hold other columns, theirs to drop.
template <int DT, bool NT = false>
__device__ __forceinline__ Raw<DT> fetch_whole(const char* row, uint32_t j, uint32_t whole) {
  typedef typename VecT<DT>::Word Word;
  Raw<DT> r;
  const Word* p = reinterpret_cast<const Word*>(row + (j < whole ? j : 0) * VecT<DT>::EB);
#pragma unroll
  for (int k = 0; k < VecT<DT>::NV; ++k) {
    if constexpr (NT)
      r.w[k] = __builtin_nontemporal_load(p + k);
    else
      r.w[k] = p[k];
  }
  return r;
}
template <int DT>
__device__ __forceinline__ void fix_tail(Raw<DT>& r, const char* row, uint32_t j, uint32_t whole, uint32_t cols) {
  if (j >= whole && j < cols) r = load_group<DT>(row, j, cols);
}
// fetch_whole for a kernel instance whose rows have no partial group (WHOLE), load_group otherwise
template <int DT, bool WHOLE>
__device__ __forceinline__ Raw<DT> fetch_group(const char* row, uint32_t j, uint32_t cols) {
  if constexpr (WHOLE)
    return fetch_whole<DT>(row, j, cols);
  else
    return load_group<DT>(row, j, cols);
}

template <int DT, bool NT = false>
__device__ __forceinline__ void store_group(char* row, uint32_t j, uint32_t cols, const Raw<DT>& r) {
  typedef typename VecT<DT>::Word Word;
  if (j + kG <= cols) {
#pragma unroll
    for (int k = 0; k < VecT<DT>::NV; ++k) {
      Word* p = reinterpret_cast<Word*>(row + j * VecT<DT>::EB) + k;
      if constexpr (NT)
        __builtin_nontemporal_store(r.w[k], p);
      else
        *p = r.w[k];
    }
  } else {
#pragma unroll
    for (int e = 0; e < kG - 1; ++e) {
      if (j + e < cols) {
        if constexpr (DT == CE_BF16)
          reinterpret_cast<uint16_t*>(row)[j + e] = (uint16_t)(r.w[0][e / 2] >> (16 * (e & 1)));
        else
          reinterpret_cast<uint32_t*>(row)[j + e] = r.w[e / 4][e % 4];
      }
    }
  }
}

template <int DT, bool NT = false>
__device__ __forceinline__ void load_f32(const char* row, uint32_t j, uint32_t cols, float (&f)[kG]) {
  raw_to_f32<DT>(load_group<DT, NT>(row, j, cols), f);
}

// Sums and maxima across lanes by DPP (a lane reads a neighbour's register in
// the add itself; a shuffle goes through LDS, about 60 cycles a step).  The
// steps' order is fixed.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ float dpp(float v) {  // lanes without a source, and rows outside ROWS, read 0
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xf, true));
}
constexpr int kSwap1 = 0xB1, kSwap2 = 0x4E;        // quad_perm [1, 0, 3, 2] and [2, 3, 0, 1]
constexpr int kHalfMirror = 0x141, kMirror = 0x140;  // of 8 and of 16 lanes
constexpr int kBcast15 = 0x142, kBcast31 = 0x143;    // the last lane of a row of 16, of the lower half, to the next

__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<kSwap1>(v);
  v += dpp<kSwap2>(v);
  v += dpp<kHalfMirror>(v);
  v += dpp<kMirror>(v);
  v += dpp<kBcast15, 0xa>(v);
  v += dpp<kBcast31, 0xc>(v);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
// the largest of values >= 0 over 4, 8 or 16 neighbouring lanes (in each of them), and over the wave
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, dpp<kSwap1>(v));
  return fmaxf(v, dpp<kSwap2>(v));
}
__device__ __forceinline__ float row_max16(float v, int lanes) {
  v = quad_max(v);
  if (lanes > 4) v = fmaxf(v, dpp<kHalfMirror>(v));
  if (lanes > 8) v = fmaxf(v, dpp<kMirror>(v));
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
  v = row_max16(v, 16);
  v = fmaxf(v, dpp<kBcast15, 0xa>(v));
  v = fmaxf(v, dpp<kBcast31, 0xc>(v));
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

}  // namespace vce
