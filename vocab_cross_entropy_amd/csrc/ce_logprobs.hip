// Token log-probabilities: of given tokens, the entropy and the K likeliest
// alternatives of every row, from one read of the logits; and their gradient.
//
// With m = max_j x_j and D = sum_j exp(x_j - m):
//   log p_t = (x_t - m) - log D
//   H       = log D - sum_j exp(x_j - m) (x_j - m) / D
//   dx_v    = sum_i g_i [v = t_i] - p_v (sum_i g_i + dH (log p_v + H))
//
// One column at the maximum is counted apart, D = 1 + R, so that log D = log1p(R) and
// 1 - p_max = R / D: log-probabilities and entropies near 0, and the gradient of a token
// whose probability is near 1, keep their digits.  Every thread sums its columns relative
// to its own running maximum; the sum of the one thread that owns the row's maximum, which
// may have lost R's digits beside the 1, is formed again at the end without that column.
// Exponentials are base 2 on the hardware's v_exp_f32, against m2 = fl(m log2 e); each batch's
// sums are brought from m2 to the exact m log2 e.
//
// Bound: the read of the logits (the gradient: and its write).  With many rows a
// workgroup takes a row; with few, a row is cut into chunks, and what each chunk finds (m, R,
// the entropy's sum, its K largest keys) goes to the row's last chunk by tagged words.
// A chunk is read in batches of T x P vectors, each batch a sample of the whole chunk (every
// nb-th KiB of it), so that what the first one shows holds for the rest.
//
// The K largest without sorting: the K-th largest of the threads' running maxima,
// found with ballots, is a bound that at least K columns reach and few others do (K threads
// have one each).  Vectors that reach the bound of their time go to LDS; it is raised after
// the first, second, fourth, eighth ... batch.  At the end their columns that reach the
// last bound, about 1.3 K of them, are ranked by counting.  Where too many reach it (constant
// rows, runs of equal values) the K-th value is found exactly by further sweeps over the chunk, and of
// its ties the lowest columns are taken.  Keys order by value, then by column, so nothing
// depends on scheduling.
//
// 8192 x 128000 BF16 with the entropy 343 us, 6.11 TB/s; with 1, 20, 64 and 128 alternatives 344, 352, 367 and 398.
// 2048 x 32000 BF16 with 64: 37 us, where 22 would be its read: five workgroups a CU (93 registers, 27 KB of LDS each;
// held to the registers of six they spill, 45 us) for the eight that each has.  One row of 128000 BF16: 8.8 us, with 20 alternatives 12: latency.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ce_internal.h"
#include "ce_row.h"

namespace vce {
namespace {

constexpr int kTop = kLogprobMaxList;  // most alternatives, and most given tokens, of a row
constexpr int kStatWords = 4;          // m, R, whether m was counted (1, or 0 of a chunk of -inf), the entropy's sum
constexpr float kFar = -1000.f;        // 2^kFar is 0; exponents of masked columns (-inf) stop here where they are a factor
typedef unsigned long long Key;        // order << 32 | ~column; 0: none
typedef Key KeyPair __attribute__((ext_vector_type(2)));

// Values in order as unsigned numbers; +0 and -0 alike, NaN below everything, 0 nothing at all.
template <int DT>
__device__ __forceinline__ uint32_t order_of(float f) {
  const uint32_t b = __float_as_uint(f + 0.f);
  uint32_t o = (int32_t)b < 0 ? ~b : b | 0x80000000u;
  if constexpr (DT == CE_BF16) o >>= 16;
  return f != f ? 1u : o;
}
template <int DT>
__device__ __forceinline__ float value_of(uint32_t o) {
  if (o == 1u) return __uint_as_float(0x7fc00000u);
  if constexpr (DT == CE_BF16) o = o & 0x8000u ? o << 16 : o << 16 | 0xffffu;
  return __uint_as_float((int32_t)o < 0 ? o & 0x7fffffffu : ~o);
}
template <int DT>
constexpr int kOrderBits = DT == CE_BF16 ? 16 : 32;
// bits of it that a bound may leave out (FP32: a relative step of 2^-13)
template <int DT>
constexpr int kLowBits = DT == CE_BF16 ? 0 : 10;
__device__ __forceinline__ Key key_of(uint32_t order, uint32_t column) { return (Key)order << 32 | (uint32_t)~column; }

// A value that at least K of the wave's 64 G numbers reach and as few as possible more, to within the lowest LOW
// bits (0 where fewer than K are not 0): found bit by bit, two at a time, below the bits that all of them share.
template <int LOW, int G>
__device__ __forceinline__ uint32_t reached_by(uint32_t K, const uint32_t (&g)[G]) {
  const auto count = [&](uint32_t c) {
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < G; ++i) n += (uint32_t)__builtin_popcountll(__ballot(g[i] >= c));
    return n;
  };
  const uint32_t one = (uint32_t)__builtin_amdgcn_readfirstlane((int)g[0]);
  uint32_t differ = 0;
#pragma unroll
  for (int i = 0; i < G; ++i) differ |= g[i] ^ one;
  differ = wave_or(differ);
  int b = differ ? 32 - __builtin_clz(differ) : 0;  // the numbers differ below bit b only
  b = (b - LOW + 1) / 2 * 2 + LOW;
  if (b <= LOW) return one >> LOW << LOW;
  uint32_t t = b < 32 ? one >> b << b : 0u;
#pragma unroll 1
  for (b -= 2; b >= LOW; b -= 2) {
    const uint32_t c1 = t + (1u << b), c2 = t + (2u << b), c3 = t + (3u << b);
    const uint32_t n1 = count(c1), n2 = count(c2), n3 = count(c3);
    t = n3 >= K ? c3 : n2 >= K ? c2 : n1 >= K ? c1 : t;
  }
  return t;
}

// The same of n numbers in LDS, by the wave that wrote them.  Slower than with a few in registers.
template <int DT>
__device__ __forceinline__ uint32_t reached_by(uint32_t K, const uint32_t* g, uint32_t n) {
  const uint32_t lane = threadIdx.x & 63;
  uint32_t t = 0;
#pragma unroll 1
  for (int b = kOrderBits<DT> - 2; b >= kLowBits<DT>; b -= 2) {
    const uint32_t step = 1u << b;
    uint32_t n1 = 0, n2 = 0, n3 = 0;
#pragma unroll 2
    for (uint32_t i = 0; i < n; i += 64) {
      const uint32_t o = i + lane < n ? g[i + lane] : 0u;
      n1 += (uint32_t)__builtin_popcountll(__ballot(o >= t + step));
      n2 += (uint32_t)__builtin_popcountll(__ballot(o >= t + 2 * step));
      n3 += (uint32_t)__builtin_popcountll(__ballot(o >= t + 3 * step));
    }
    t += n3 >= K ? 3 * step : n2 >= K ? 2 * step : n1 >= K ? step : 0u;
  }
  return t;
}

// The same of group maxima, `g(i)` a lane's i-th of G: of 64, 128 or 256 groups, at least twice K, made of them.  About
// 1.4 K columns reach it then (K = 32 of 64: 44, 64 of 128: 89); more groups take more ballots than they save.
template <int DT, int G, typename Group>
__device__ __forceinline__ uint32_t bound_of(uint32_t K, Group g) {
  const auto of = [&](auto groups) {
    constexpr int N = decltype(groups)::value;
    uint32_t top[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      top[i] = g(i);
#pragma unroll
      for (int k = N; k < G; k += N) {
        const uint32_t o = g(i + k);
        top[i] = o > top[i] ? o : top[i];
      }
    }
    return reached_by<kLowBits<DT>, N>(K, top);
  };
  if (K <= 32) return of(std::integral_constant<int, 1>{});
  if (K <= 64) return of(std::integral_constant<int, 2>{});
  return of(std::integral_constant<int, 4>{});
}

template <int T>
__device__ __forceinline__ uint32_t block_count(uint32_t c, uint32_t* sh) {
  c = (uint32_t)wave_count64((int)c);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = c;
  __syncthreads();
  uint32_t n = 0;
#pragma unroll
  for (int i = 0; i < T / 64; ++i) n += sh[i];
  return n;
}

// The K largest keys of a chunk, exactly, where a bound `t` let too many through, or may have let too few (NaN, which
// maxima pass over): the K-th largest value over all columns (the bound itself where fewer than K exceed it), every column
// above it, and its ties from the lowest column on.  Leaves K keys in cand[]; a chunk of fewer columns, keys of order 0 too.
// Rare, so it is kept short: every sweep reads the chunk again.  Column 0 of the chunk is the row's column lo.
// With `if_signalling` nothing is done, and false returned, for a chunk without a signalling NaN.  (64 x 128000 FP32 with a
// NaN in every row, 5 alternatives: 24 us, 17 without any; 152 where every NaN is answered by the search.)
template <int DT, int T>
__device__ __forceinline__ bool exact_largest(const char* chunk, uint32_t lo, uint32_t cols, uint32_t K, uint32_t t,
                                              bool if_signalling, Key* cand, uint32_t* n_cand, uint32_t* sh) {
  typedef typename LogitT<DT>::Word Word;
  constexpr int E = LogitT<DT>::E;
  const uint32_t tid = threadIdx.x;
  // the orders of vector i's columns, 0 for those that are not there
  const auto orders = [&](const u32x4v& v, uint32_t i, uint32_t (&o)[E]) {
    float f[E];
    unpack_vec<DT>(v, f);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = i * E + e < cols ? order_of<DT>(f[e]) : 0u;
  };
  const uint32_t whole = cols / E;
  const auto whole_vec = [&](uint32_t i) -> u32x4v { return *reinterpret_cast<const Word*>(chunk + (i < whole ? i : 0u) * 16u); };
  const u32x4v rest = partial_vec<DT>(chunk, whole * E, cols);
  if (if_signalling) {
    uint32_t found = 0;
#pragma unroll 1
    for (uint32_t i = tid; i <= whole; i += T) {
      float f[E];
      unpack_vec<DT>(i < whole ? whole_vec(i) : rest, f);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint32_t bits = __float_as_uint(f[e]);
        found |= (bits & 0x7fc00000u) == 0x7f800000u && (bits & 0x3fffffu);
      }
    }
    if (block_count<T>(found, sh) == 0) return false;
  }
  // how many columns reach c, c + step and c + 2 step
  const auto count = [&](uint32_t c, uint32_t step, uint32_t (&n)[3]) {
    n[0] = n[1] = n[2] = 0;
    const auto add = [&](const u32x4v& v, uint32_t i) {
      uint32_t o[E];
      orders(v, i, o);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        n[0] += o[e] >= c;
        n[1] += o[e] >= c + step;
        n[2] += o[e] >= c + 2 * step;
      }
    };
#pragma unroll 1
    for (uint32_t base = 0; base < whole; base += 4 * T) {
      u32x4v v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = whole_vec(base + k * T + tid);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (base + k * T + tid < whole) add(v[k], base + k * T + tid);
    }
    if (tid == 0) add(rest, whole);
#pragma unroll
    for (int k = 0; k < 3; ++k) n[k] = block_count<T>(n[k], sh);
  };
  // the bound where at least K columns reach it and fewer are above it; else from the top on, two bits a sweep
  uint32_t n[3], above = 0;
#pragma unroll 1
  for (int b = kOrderBits<DT>; b >= -2; b -= 2) {
    if (b == kOrderBits<DT> || b < 0) {
      count(t, 1, n);
      above = n[1];
      if (b < 0 || (n[0] >= K && above < K)) break;
      t = 0;
    } else {
      count(t + (1u << b), 1u << b, n);
      t += n[2] >= K ? 3u << b : n[1] >= K ? 2u << b : n[0] >= K ? 1u << b : 0u;
    }
  }
  if (tid == 0) *n_cand = 0;
  __syncthreads();
  uint32_t have = above;
#pragma unroll 1
  for (uint32_t base = 0; base * E < cols; base += T) {  // columns rise with base, then with the thread, then within the vector
    const uint32_t i = base + tid;
    uint32_t o[E], mine = 0;
    orders(i < whole ? whole_vec(i) : rest, i, o);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      mine += o[e] == t;
      if (o[e] > t) cand[atomicAdd(n_cand, 1u)] = key_of(o[e], lo + i * E + e);
    }
    if (have >= K) continue;  // the same for the whole workgroup
    uint32_t upto = mine;     // inclusive over the wave's lanes
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t u = (uint32_t)__shfl_up((int)upto, d);
      upto += (tid & 63) >= (uint32_t)d ? u : 0u;
    }
    __syncthreads();
    if ((tid & 63) == 63) sh[tid >> 6] = upto;
    __syncthreads();
    uint32_t at = have + upto - mine;
#pragma unroll
    for (int w = 0; w < T / 64; ++w) {
      at += (uint32_t)w < tid >> 6 ? sh[w] : 0u;
      have += sh[w];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (o[e] == t && at < K) cand[at] = key_of(t, lo + i * E + e);
      at += o[e] == t;
    }
  }
  __syncthreads();
  if (tid == 0) *n_cand = K;
  __syncthreads();
  return true;
}

// How many of these lanes come before this one.
__device__ __forceinline__ uint32_t lanes_below(unsigned long long lanes) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(lanes >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)lanes, 0u));
}

// Collected keys: each wave's in a segment of its own, in LDS, with zeros behind them to the next multiple of eight.
template <int W, int SEG>
struct Segments {
  static constexpr int kStride = SEG + 8;
  Key* keys;
  uint32_t* n;      // [W]
  uint32_t* ranks;  // [W * SEG]

  // Adds the keys of the lanes that have one; `have` counts the wave's (beyond SEG they are dropped).
  __device__ __forceinline__ void add(bool mine, Key key, uint32_t& have) const {
    const unsigned long long lanes = __ballot(mine);
    if (lanes == 0) return;
    const uint32_t at = have + lanes_below(lanes);
    if (mine && at < (uint32_t)SEG) keys[(threadIdx.x >> 6) * kStride + at] = key;
    have += (uint32_t)__builtin_popcountll(lanes);
  }
  __device__ __forceinline__ void close(uint32_t have) const {
    const uint32_t lane = threadIdx.x & 63, kept = have < (uint32_t)SEG ? have : (uint32_t)SEG;
    if (lane < 8) keys[(threadIdx.x >> 6) * kStride + kept + lane] = 0;
    if (lane == 0) n[threadIdx.x >> 6] = have;
    for (uint32_t i = threadIdx.x; i < W * SEG; i += W * 64) ranks[i] = 0;
  }
  // the i-th key of all segments
  __device__ __forceinline__ Key at(uint32_t i) const {
    uint32_t base = 0;
#pragma unroll
    for (int w = 0; w < W - 1; ++w) {
      const bool past = i >= n[w] && base == (uint32_t)w * kStride;
      i -= past ? n[w] : 0u;
      base += past ? kStride : 0u;
    }
    return keys[base + i];
  }
  // put(rank, key) for each of the keys: every wave counts, for all keys, the larger ones in its own segment
  template <typename Put>
  __device__ __forceinline__ void rank(uint32_t total, Put put) const {
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const KeyPair* const own = reinterpret_cast<const KeyPair*>(keys + wave * kStride);
    const uint32_t count = n[wave];
#pragma unroll 1
    for (uint32_t base = 0; base < total; base += 64) {
      const uint32_t i = base + lane;
      const Key key = i < total ? at(i) : ~0ull;
      uint32_t r = 0;
#pragma unroll 1
      for (uint32_t q = 0; q < count; q += 8) {
        KeyPair o[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] = own[q / 2 + c];
#pragma unroll
        for (int c = 0; c < 4; ++c) r += (o[c].x > key) + (o[c].y > key);
      }
      if (r) atomicAdd(&ranks[i], r);
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < total; i += W * 64) put(ranks[i], at(i));
  }
};

// Vectors that a wave can keep.  A bound lets 1.4 K of them by over as many batches as it was found from, 45 a wave of
// four for K = 128, and raising it leaves as many of those before.
__host__ __device__ constexpr uint32_t hit_room(int32_t K) { return 64u + (uint32_t)K * 5u / 4u; }

// (Six waves a SIMD of the shape with few loads in flight: 8192 x 4096 FP32, 20 alternatives, 53 us; with the compiler's 81
// registers, five, 60.  The shape with more would spill.)
template <int DT, int T, int P, bool TOP, bool ENT>
__global__ __launch_bounds__(T) __attribute__((amdgpu_waves_per_eu(T == 256 && P == 2 ? 6 : 1, 8))) void k_logprobs(LogprobArgs a) {
  typedef typename LogitT<DT>::Word Word;
  constexpr int E = LogitT<DT>::E, EB = LogitT<DT>::EB, W = T / 64;
  constexpr int TK = (kTop + T - 1) / T;  // given tokens a thread
  constexpr bool kSplit = W > 1;          // one wave only ever takes a whole row
  constexpr int kRound = 1024 / T;        // keys a thread takes into one round of merging
  // A wave's vectors that have reached a bound, and the columns that reach the last one; later the row's keys
  constexpr int kSeg = W > 1 ? 1024 / W : 320;
  static_assert(kSeg >= 64 * (kSplit ? kRound : 0) && kSeg >= kTop, "what the segments hold");
  __shared__ float sh_max[W];
  __shared__ float sh_sum[W][2];
  __shared__ uint32_t sh_own[W];
  __shared__ float st[kSplit ? kMaxChunks : 1][kStatWords];
  __shared__ uint32_t sh_cnt[W], n_seg[W], n_cand;
  __shared__ uint32_t thread_top[TOP && W > 1 ? T : 1], sh_bound;
  __shared__ uint32_t ranks[TOP ? W * kSeg : 1];
  extern __shared__ __align__(16) char hit_mem[];  // for each wave, hit_room(K) vectors, and where they come from
  __shared__ __align__(32) Key seg_keys[TOP ? W * Segments<W, kSeg>::kStride : 1];
  __shared__ Key top[TOP ? kTop : 1];  // the row's keys
  const Segments<W, kSeg> seg{seg_keys, n_seg, ranks};

  const uint32_t tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const uint32_t room = hit_room(a.K);
  u32x4v* const hit = reinterpret_cast<u32x4v*>(hit_mem) + wave * room;
  uint32_t* const hit_vec = reinterpret_cast<uint32_t*>(hit_mem + (size_t)W * room * 16) + wave * room;
  const uint32_t C = kSplit ? (uint32_t)a.chunks : 1u, K = TOP ? (uint32_t)a.K : 0u;
  const uint32_t in_launch = kSplit ? blockIdx.x / C : blockIdx.x;
  const int64_t r = a.row0 + in_launch;
  const uint32_t k = blockIdx.x - in_launch * C;
  const bool last = k == C - 1;  // the row's last chunk brings it together
  WsView ws{0u, true, 0ull};
  if (C > 1) ws = view_workspace(a.hdr, a.ws_bytes);
  const int64_t i0 = (uint32_t)r / (uint32_t)a.d1, i1 = (uint32_t)r % (uint32_t)a.d1;  // (64-bit divisions delay the first load)
  const char* const row = a.x + (i0 * a.s0 + i1 * a.s1) * EB;
  const uint32_t lo = k * (uint32_t)a.chunk_cols;
  const uint32_t cols = (uint32_t)a.V - lo < (uint32_t)a.chunk_cols ? (uint32_t)a.V - lo : (uint32_t)a.chunk_cols;
  const char* const chunk = row + (size_t)lo * EB;
  // Vectors: `whole` of them, and one of cols % E columns.  Lines of 64 vectors; batch b has every nb-th from the b-th on.
  const uint32_t whole = cols / E, vecs = (cols + E - 1) / E;
  const uint32_t nb = (vecs + T * P - 1) / (T * P);
  const auto vector_at = [&](uint32_t b, uint32_t j, uint32_t w, uint32_t l) { return ((j * W + w) * nb + b) * 64 + l; };

  // ---- the given tokens' ids go out first, and their logits after the first batch
  const int64_t* const ids = a.ids ? a.ids + i0 * a.is0 + i1 * a.is1 : nullptr;
  int64_t id[TK];
  float xt[TK];
#pragma unroll
  for (int i = 0; i < TK; ++i) {
    id[i] = last && (int)(i * T + tid) < a.M ? ids[i * T + tid] : -1;
    xt[i] = 0.f;
  }

  float m = -INFINITY;       // this thread's maximum
  float s0 = 0.f, s1 = 0.f;  // its sums of 2^u and of 2^u u, u = (x - m) log2 e
  // the sums relative to a larger maximum (kFar: 2^kFar is 0, and 0 times an infinity would be NaN)
  const auto move_sums = [&](float to) {
    const float d = m > -INFINITY ? fmaxf((m - to) * kLog2e, kFar) : kFar;
    const float w = exp2_hw(d);
    if constexpr (ENT) s1 = __builtin_fmaf(d, s0, s1) * w;
    s0 *= w;
  };
  bool low = true;                      // no bound, or -inf
  float least = -INFINITY;              // the bound
  uint32_t bound = 0, hits = 0;
  // the bound from the running maxima of all threads, by one wave; two barriers
  const auto raise_bound = [&](auto meanwhile) {
    thread_top[tid] = tid < vecs ? order_of<DT>(m) : 0u;
    __syncthreads();
    if (wave == 0) {
      const uint32_t t = bound_of<DT, W>(K, [&](int i) { return thread_top[i * 64 + lane]; });
      if (lane == 0) sh_bound = t;
    }
    meanwhile();
    __syncthreads();
    bound = sh_bound;
  };
  const auto set_least = [&] {
    low = bound <= order_of<DT>(-INFINITY);
    least = low ? -INFINITY : value_of<DT>(bound);
  };
  // the wave's hits that still reach the bound, moved up
  const auto prune = [&] {
    uint32_t kept = 0;
    for (uint32_t i = 0; i < hits; i += 64) {
      const uint32_t at = i + lane < hits ? i + lane : i;
      const u32x4v v = hit[at];
      const uint32_t from = hit_vec[at];
      const float top = largest<DT>(v, -INFINITY);
      const bool mine = i + lane < hits && (low ? top > -INFINITY : top >= least);
      const unsigned long long lanes = __ballot(mine);
      if (mine) {
        hit[kept + lanes_below(lanes)] = v;
        hit_vec[kept + lanes_below(lanes)] = from;
      }
      kept += (uint32_t)__builtin_popcountll(lanes);
    }
    hits = kept;
  };
#pragma unroll 1
  for (uint32_t b = 0; b < nb; ++b) {
    u32x4v v[P];
    if (whole > 0) {
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const uint32_t i = vector_at(b, j, wave, lane);
        v[j] = __builtin_nontemporal_load(reinterpret_cast<const Word*>(chunk + (i < whole ? i : 0u) * 16u));
      }
    }
    if (b == 0) {
#pragma unroll
      for (int i = 0; i < TK; ++i)
        if (id[i] >= 0 && id[i] < a.V) xt[i] = load_logit<DT>(row, id[i]);
    }
#pragma unroll
    for (int j = 0; j < P; ++j) {
      constexpr uint32_t kNone = LogitT<DT>::kNegInf;
      if (vector_at(b, j, wave, 63) < whole) continue;  // the same for the whole wave
      if (vector_at(b, j, wave, lane) >= whole) v[j] = u32x4v{kNone, kNone, kNone, kNone};
    }
    if (vecs > whole && (whole >> 6) % nb == b) {  // the vector that is not whole
      const uint32_t slot = (whole >> 6) / nb;
      if (slot % W == wave && (whole & 63) == lane) {
        const u32x4v w = partial_vec<DT>(chunk, whole * E, cols);
#pragma unroll
        for (int j = 0; j < P; ++j) {
          u32x4v mine = w;
          relaunch(mine);  // (as in pick)
          if ((uint32_t)j == slot / W) v[j] = mine;
        }
      }
    }

    // ---- maxima; the sums so far go over to a new one
    float vm[P], top_m = m;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      vm[j] = largest<DT>(v[j], -INFINITY);
      top_m = fmaxf(top_m, vm[j]);
    }
    if (top_m > m) {
      move_sums(top_m);
      m = top_m;
    }

    // ---- vectors that reach the bound
    if constexpr (TOP) {
      if constexpr (W > 1) {
        if (((b + 1) & b) == 0) {  // b = 0, 1, 3, 7 ...
          raise_bound([] {});
          set_least();
          if (hits > 64 && hits <= room) prune();
        }
      } else {  // one batch: of the vectors' maxima, or of quarter vectors' where K takes nearly all of those (65536 x 1000
                // BF16, K = 128: 381 us, 778 by sweeps; K = 100, 125 vectors: 293, 322)
        if (P == 4 && vecs * 4 <= K * 5) {
          static_assert(kTop * 5 * sizeof(uint32_t) <= sizeof seg_keys, "the quarters' maxima");
          u32x4v* const quarters = reinterpret_cast<u32x4v*>(seg_keys);
#pragma unroll
          for (int j = 0; j < P; ++j) {
            const uint32_t i = vector_at(b, j, wave, lane);
            relaunch(v[j]);
            float f[E];
            unpack_vec<DT>(v[j], f);
            u32x4v o;
#pragma unroll
            for (int q = 0; q < 4; ++q) o[q] = order_of<DT>(fmaxf(f[q * (E / 4)], f[q * (E / 4) + E / 4 - 1]));
            if (i < vecs) quarters[i] = o;
          }
          bound = reached_by<DT>(K, reinterpret_cast<const uint32_t*>(quarters), vecs * 4);
        } else {
          bound = bound_of<DT, P>(K, [&](int j) { return vector_at(b, j, wave, lane) < vecs ? order_of<DT>(vm[j]) : 0u; });
        }
        set_least();
      }
#pragma unroll
      for (int j = 0; j < P; ++j) {
        // (under a bound of -inf the columns above it; -inf's own come in at the end)
        const bool mine = low ? vm[j] > -INFINITY : vm[j] >= least;
        const unsigned long long lanes = __ballot(mine);
        if (lanes == 0) continue;
        const uint32_t at = hits + lanes_below(lanes);
        if (mine && at < room) {
          hit[at] = v[j];
          hit_vec[at] = vector_at(b, j, wave, lane);
        }
        hits += (uint32_t)__builtin_popcountll(lanes);
      }
    }

    // ---- sums
    float from = m == -INFINITY ? 0.f : m * kLog2e;
    if (fabsf(from) > kNear) {
      subtract<DT, P>(v, m);
      from = 0.f;
    }
    float t0 = 0.f, t1 = 0.f, h = 0.f;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      relaunch(v[j]);
      float f[E];
      unpack_vec<DT>(v[j], f);
#pragma unroll
      for (int c = 0; c < E; c += 2) {
        const float u = __builtin_fmaf(f[c], kLog2e, -from), w = __builtin_fmaf(f[c + 1], kLog2e, -from);
        const float eu = exp2_hw(u), ew = exp2_hw(w);
        t0 += eu;
        t1 += ew;
        if constexpr (ENT) {
          h = __builtin_fmaf(eu, fmaxf(u, kFar), h);
          h = __builtin_fmaf(ew, fmaxf(w, kFar), h);
        }
      }
    }
    {
      // from m2 to m log2 e: the terms are too large by 2^d, d = m log2 e - m2
      const float d = from != 0.f ? __builtin_fmaf(m, kLog2e, -from) : 0.f, grow = __builtin_fmaf(-d, kLn2f, 1.f);
      t0 += t1;
      s0 = __builtin_fmaf(t0, grow, s0);
      if constexpr (ENT) s1 = __builtin_fmaf(__builtin_fmaf(-d, t0, h), grow, s1);
    }
  }

  // ---- the chunk's maximum and the first thread that has it
  {
    const float wm = wave_largest(m);
    const unsigned long long owners = __ballot(m == wm);
    if (lane == 0) {
      sh_max[wave] = wm;
      sh_own[wave] = wave * 64 + (uint32_t)__builtin_ctzll(owners | 1ull << 63);
    }
  }
  float M;
  const auto sums_of_chunk = [&] {
    M = sh_max[0];
    uint32_t owner = sh_own[0];
#pragma unroll
    for (int i = 1; i < W; ++i) {
      owner = sh_max[i] > M ? sh_own[i] : owner;
      M = fmaxf(M, sh_max[i]);
    }
    move_sums(M);
    if (M != -INFINITY && tid == owner) s0 = s1 = 0.f;
    if (wave == W - 1 && M != -INFINITY) {  // the owner's vectors again, without one column at the maximum
      bool out = false;                 // it has been left out
      for (uint32_t base = 0; base < nb * P; base += 64) {
        const uint32_t s = base + lane, i = vector_at(s % nb, s / nb, owner >> 6, owner & 63);
        float f[E];
        unpack_vec<DT>(s < nb * P && i < whole ? *reinterpret_cast<const Word*>(chunk + i * 16u)
                       : s < nb * P            ? partial_vec<DT>(chunk, i * E, cols)
                                               : partial_vec<DT>(chunk, cols, cols),
                       f);
        bool mine = false;
#pragma unroll
        for (int c = 0; c < E; ++c) mine |= f[c] == M;
        const unsigned long long lanes = __ballot(mine);
        bool leave = !out && mine && lanes_below(lanes) == 0;
        out |= lanes != 0;
#pragma unroll
        for (int c = 0; c < E; ++c) {
          const float u = (f[c] - M) * kLog2e;
          const bool skip = leave && f[c] == M;
          if (skip) leave = false;
          const float e = skip ? 0.f : exp2_hw(u);
          s0 += e;
          if constexpr (ENT) s1 = __builtin_fmaf(e, fmaxf(u, kFar), s1);
        }
      }
    }
  };
  if constexpr (TOP && W > 1) {
    if (((nb - 1) & nb) != 0) {  // the last batch did not raise it
      raise_bound(sums_of_chunk);
      set_least();
    } else {
      __syncthreads();
      sums_of_chunk();
    }
  } else {
    __syncthreads();
    sums_of_chunk();
  }
  s0 = wave_sum(s0);
  if constexpr (ENT) s1 = wave_sum(s1);
  if (lane == 0) {
    sh_sum[wave][0] = s0;
    sh_sum[wave][1] = s1;
  }

  // the chunk's sums, later the row's: `one` column counted apart
  float one = M == -INFINITY ? 0.f : 1.f, rest = 0.f;
  s1 = 0.f;
  const auto sums_of_waves = [&] {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      rest += sh_sum[i][0];
      s1 += sh_sum[i][1];
    }
  };

  // ---- the K largest: the hits' columns, a lane each
  if constexpr (TOP) {
    uint32_t have = 0;
    if (hits > room) {
      have = kSeg + 1;
      hits = 0;
    }
    for (uint32_t i = 0; i < hits * E; i += 64) {
      const uint32_t at = i + lane < hits * E ? i + lane : 0u;
      const float f = load_logit<DT>(reinterpret_cast<const char*>(hit), at);
      const uint32_t c = hit_vec[at / E] * E + at % E;
      seg.add(i + lane < hits * E && c < cols && (low ? f > -INFINITY : f >= least), key_of(order_of<DT>(f), lo + c), have);
    }
    if (low) {  // fewer than K threads have more than -inf: of the first K columns enough are -inf to fill up with
      for (uint32_t c = tid; c - lane < (K < cols ? K : cols); c += T) {
        const bool in = c < (K < cols ? K : cols);
        seg.add(in && load_logit<DT>(chunk, in ? c : 0) == -INFINITY, key_of(order_of<DT>(-INFINITY), lo + c), have);
      }
    }
    seg.close(have);
    __syncthreads();
    uint32_t reach = 0, most = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      reach += n_seg[i];
      most = n_seg[i] > most ? n_seg[i] : most;
    }
    sums_of_waves();
    const bool missed = most > (uint32_t)kSeg || reach < (cols < K ? cols : K);
    if (missed || rest != rest) {  // (a signalling NaN may have hidden maxima, and with them columns, from the bound)
      if (exact_largest<DT, T>(chunk, lo, cols, K, low ? order_of<DT>(-INFINITY) : bound, !missed, seg_keys, &n_cand, sh_cnt)) {
        if (tid < W) n_seg[tid] = tid == 0 ? n_cand : 0u;
        if (tid < 8 * W) seg_keys[(tid / 8) * Segments<W, kSeg>::kStride + (tid < 8 ? n_cand : 0u) + tid % 8] = 0;
        __syncthreads();
      }
    }
  } else {
    __syncthreads();
    sums_of_waves();
  }

  if (C > 1) {
    const uint32_t words = kStatWords + 2 * K;
    unsigned long long* const slot = a.slots + ((size_t)r * C + k) * words;
    const bool keep = withheld(ws, r, (int)k);
    if (tid == 0 && !keep) {
      put_word(slot + 0, ws.tag, __float_as_uint(M));
      put_word(slot + 1, ws.tag, __float_as_uint(rest));
      put_word(slot + 2, ws.tag, __float_as_uint(one));
      put_word(slot + 3, ws.tag, __float_as_uint(s1));
    }
    if constexpr (TOP) {
      uint32_t n = 0;
#pragma unroll
      for (int i = 0; i < W; ++i) n += n_seg[i];
      const auto publish = [&](uint32_t rank, Key key) {
        if (rank >= K || keep) return;
        put_word(slot + kStatWords + 2 * rank, ws.tag, (uint32_t)key);
        put_word(slot + kStatWords + 2 * rank + 1, ws.tag, (uint32_t)(key >> 32));
      };
      seg.rank(n, publish);
      for (uint32_t i = n + tid; i < K; i += T) publish(i, 0);
    }
    if (!last) return;

    // ---- the row's last chunk collects, with the first readings of all words in flight together
    uint32_t spins = 0;
    bool ok = ws.ok;
    const unsigned long long* const slots = a.slots + (size_t)r * C * words;
    constexpr int kStatReads = (kMaxChunks * kStatWords + T - 1) / T;
    unsigned long long stat[kStatReads], first[TOP ? 2 * kRound : 1];
    const auto stat_word = [&](int i) {
      const uint32_t at = i * T + tid;
      return slots + (size_t)(at / kStatWords) * words + at % kStatWords;
    };
#pragma unroll
    for (int i = 0; i < kStatReads; ++i) stat[i] = i * T + tid < C * kStatWords ? peek_word(stat_word(i)) : 0ull;
    const uint32_t spread = lane * W + wave;  // neighbouring keys go to different waves
    // the chunks' first keys, then their second ...: the threads' largest are then the T best placed
    const auto key_word = [&](uint32_t at) { return slots + (size_t)(at % C) * words + kStatWords + at / C * 2; };
    if constexpr (TOP) {
#pragma unroll
      for (int i = 0; i < kRound; ++i) {
        const uint32_t at = i * T + spread;
        first[2 * i] = at < C * K ? peek_word(key_word(at)) : 0ull;
        first[2 * i + 1] = at < C * K ? peek_word(key_word(at) + 1) : 0ull;
      }
    }
#pragma unroll
    for (int i = 0; i < kStatReads; ++i) {
      if (i * T + tid >= C * kStatWords) continue;
      uint32_t w = 0x7fc00000u;
      ok &= await_word(stat_word(i), ws.tag, stat[i], spins, &w);
      st[(i * T + tid) / kStatWords][(i * T + tid) % kStatWords] = __uint_as_float(w);
    }
    if constexpr (TOP) {
      // Rounds until the last keys taken, one of each chunk, are all behind K others: so are those that follow them.  (One
      // row of 128000 BF16, 128 alternatives: one round of nine, 21 us; 41 with all.)
      uint32_t done = 0, held = 0;  // keys taken, K of each chunk; keys of earlier rounds
      bool more = true;
      while (done < C * K && more) {
        Key key[kRound], last = 0;  // the largest of the thread's that are last of their chunk's
        uint32_t best = 0;
        const uint32_t end = done + kRound * T - held < C * K ? done + kRound * T - held : C * K;
#pragma unroll
        for (int i = 0; i < kRound; ++i) {
          const uint32_t at = i * T + spread, from = done + at - held;
          key[i] = 0;
          if (at < held) {
            key[i] = top[at];
          } else if (from < C * K) {
            const unsigned long long* const p = key_word(from);
            uint32_t k0 = 0, k1 = 0;
            bool got = await_word(p, ws.tag, done ? peek_word(p) : first[2 * i], spins, &k0);
            got &= await_word(p + 1, ws.tag, done ? peek_word(p + 1) : first[2 * i + 1], spins, &k1);
            ok &= got;
            key[i] = got ? (Key)k1 << 32 | k0 : 0ull;
            if (from + C >= end) last = key[i] > last ? key[i] : last;
          }
          const uint32_t o = (uint32_t)(key[i] >> 32);
          best = o > best ? o : best;
        }
        done = end;
        held = K;
        thread_top[tid] = best;
        __syncthreads();  // (and every thread has ranked the chunk's candidates, or read `top`)
        uint32_t least_order = 0;
        if (C * K > 192) {  // fewer are ranked sooner than a bound is found
          if (wave == 0) {
            const uint32_t t = bound_of<DT, W>(K, [&](int i) { return thread_top[i * 64 + lane]; });
            if (lane == 0) sh_bound = t;
          }
          __syncthreads();
          least_order = sh_bound;
        }
        uint32_t have = 0;
#pragma unroll
        for (int i = 0; i < kRound; ++i)
          seg.add((uint32_t)(key[i] >> 32) >= least_order && key[i] != 0ull, key[i], have);
        seg.close(have);
        for (uint32_t i = tid; i < K; i += T) top[i] = 0ull;  // a word that never came leaves a place empty
        __syncthreads();
        uint32_t n = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) n += n_seg[i];
        seg.rank(n, [&](uint32_t rank, Key key) {
          if (rank < K) top[rank] = key;
        });
        __syncthreads();
        more = __syncthreads_or(last != 0ull && last >= top[K - 1]);
      }
    }
    ok = __syncthreads_and(ok);
    if (!ok && tid == 0) atomicOr(&a.hdr->status, ws.ok ? 1u : 2u);
    // lane c of every wave takes chunk c; the first with the row's maximum counts one column of it apart
    const bool has = lane < C;
    const float mc = has ? st[lane][0] : -INFINITY;
    M = wave_largest(mc);
    const bool some = has && mc != -INFINITY;
    const unsigned long long best = __ballot(some && mc == M);
    const float dm = some ? fmaxf((mc - M) * kLog2e, kFar) : 0.f, w = exp2_hw(dm);
    const float rc = has ? st[lane][1] : 0.f, sc = some ? st[lane][3] : 0.f;
    const bool apart = some && mc == M && lanes_below(best) == 0;
    // (a chunk of -inf has the sum 0, or the NaN of a NaN)
    rest = wave_sum(apart ? rc : some ? (rc + 1.f) * w : rc);
    if constexpr (ENT) s1 = wave_sum(some ? __builtin_fmaf(dm, rc + 1.f, sc) * w : 0.f);
    one = best ? 1.f : 0.f;
    if (!ok) rest = __uint_as_float(0x7fc00000u);
    if (TOP && !ok) {
      for (uint32_t i = tid; i < K; i += T) top[i] = 0ull;
      __syncthreads();
    }
  } else if constexpr (TOP) {
    // one chunk: its ranks are the row's (K is at most the number of columns)
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) n += n_seg[i];
    seg.rank(n, [&](uint32_t rank, Key key) {
      if (rank < K) top[rank] = key;
    });
    __syncthreads();
  }

  // ---- the row's outputs (+inf has no distribution either)
  if (M == INFINITY) rest = __uint_as_float(0x7fc00000u);
  const float logd = one == 1.f ? log1pf(rest) : logf(rest);
#pragma unroll
  for (int i = 0; i < TK; ++i) {
    const int at = i * T + tid;
    if (at < a.M) {
      const int64_t t = id[i];
      float lp = (xt[i] - M) - logd;
      if (t < 0 || t >= a.V) lp = __uint_as_float(0x7fc00000u);
      if (t == a.ignore_idx) lp = 0.f;
      a.logp[r * a.M + at] = lp;
    }
  }
  if constexpr (TOP) {
    for (uint32_t i = tid; i < K; i += T) {
      const Key key = top[i];
      const float f = value_of<DT>((uint32_t)(key >> 32));
      a.top_ids[r * K + i] = key ? (int64_t)(uint32_t)~(uint32_t)key : -1;
      a.top_logp[r * K + i] = key ? (f - M) - logd : __uint_as_float(0x7fc00000u);
    }
  }
  if (tid == 0) {
    const float D = rest + one;
    const float h = ENT ? __builtin_fmaf(-kLn2f, s1 / D, logd) : 0.f;
    if (ENT) a.entropy[r] = h;
    if (a.lse) a.lse[r] = M + logd;
    if (a.stats) reinterpret_cast<float4*>(a.stats)[r] = make_float4(M, logd, rest / D, h);
  }

  // ---- the last row's workgroup ends the call once every row has been brought together
  if (C > 1) {
    if (r != a.N - 1) {
      if (tid == 0) put_word(a.done + r, ws.tag, 0u);
      return;
    }
    uint32_t spins = 0, w;
    bool ok = true;
    for (int64_t base = 0; base < r; base += 4 * T) {
      unsigned long long first[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t at = base + i * T + tid;
        first[i] = peek_word(a.done + (at < r ? at : 0));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t at = base + i * T + tid;
        ok = ok && await_word(a.done + (at < r ? at : 0), ws.tag, first[i], spins, &w);
      }
    }
    if (!ok) atomicOr(&a.hdr->status, 1u);
    __syncthreads();
    if (tid == 0) next_epoch(a.hdr);
  }
}

// The gradient: a chunk's vectors, all loaded at once, each written where it was
// read from or elsewhere; the few columns of given tokens are written again by one
// thread a token, with every gradient that names the column added up in order.
// Bound: HBM.  8192 x 128000 BF16 with the entropy's 706 us, 5.94 TB/s; 1024 x 32003 FP32, 5 tokens, 46 us, 5.7 TB/s.
template <int DT, bool ENT>
__global__ __launch_bounds__(kLogprobBwdT) void k_logprobs_bwd(LogprobGradArgs a) {
  constexpr int T = kLogprobBwdT, P = kLogprobBwdP, E = LogitT<DT>::E, EB = LogitT<DT>::EB, W = T / 64;
  static_assert(T >= 2 * kTop, "a thread for every token of both lists");
  __shared__ int64_t sid[T];
  __shared__ float sg[T];
  __shared__ float sh[W];
  const uint32_t tid = threadIdx.x, C = (uint32_t)a.chunks;
  const uint32_t in_launch = blockIdx.x / C, k = blockIdx.x - in_launch * C;
  const int64_t r = a.row0 + in_launch;
  const int64_t i0 = (uint32_t)r / (uint32_t)a.d1, i1 = (uint32_t)r % (uint32_t)a.d1;  // (64-bit divisions delay the first load)
  const char* const row = a.x + (i0 * a.s0 + i1 * a.s1) * EB;
  char* const out = a.out + (i0 * a.os0 + i1 * a.os1) * EB;
  const uint32_t lo = k * (uint32_t)a.chunk_cols;
  const uint32_t cols = (uint32_t)a.V - lo < (uint32_t)a.chunk_cols ? (uint32_t)a.V - lo : (uint32_t)a.chunk_cols;

  const uint32_t M = (uint32_t)a.M, L = M + (uint32_t)a.K;
  int64_t id = -1;
  float g = 0.f;
  if (tid < M) {
    id = a.ids[i0 * a.is0 + i1 * a.is1 + tid];
    g = a.dlogp[r * M + tid];
  } else if (tid < L) {
    id = a.top_ids[r * a.K + (tid - M)];
    g = a.dtop[r * a.K + (tid - M)];
  }
  const float4 s = reinterpret_cast<const float4*>(a.stats)[r];  // m, log D, 1 - p_max, H
  const float dh = ENT ? a.dentropy[r] : 0.f;
  u32x4v v[P];
  load_chunk<DT, T, P>(row + (size_t)lo * EB, cols, v);
  finish_chunk<DT, T, P, false>(row + (size_t)lo * EB, cols, v);

  const bool counts = tid < L && (tid >= M || id != a.ignore_idx);  // an alternative may well be that column
  const bool valid = id >= 0 && id < a.V;
  const bool mine = counts && valid && id >= lo && id < (int64_t)lo + cols;
  if (!counts) g = 0.f;
  if (counts && !valid) g = __uint_as_float(0x7fc00000u);  // the row's gradient is NaN
  float xt = mine ? load_logit<DT>(row, id) : 0.f;
  float G = g;
  if (L > 1) {
    sid[tid] = mine ? id : -1;
    sg[tid] = g;
    G = wave_sum(g);
    if ((tid & 63) == 0) sh[tid >> 6] = G;
    __syncthreads();
    G = sh[0];
#pragma unroll
    for (int i = 1; i < W; ++i) G += sh[i];
  } else if (L == 1) {
    if (tid == 0) sh[0] = g;
    __syncthreads();
    G = sh[0];
  }

  float top = s.x;
  if (fabsf(top * kLog2e) > kNear && fabsf(top) < INFINITY) {
    subtract<DT, P>(v, top);
    xt -= top;
    top = 0.f;
  }
  // p = 2^(x log2 e - c), c = (m + log D) log2 e in two parts; the second matters to FP32's rounding and to log p
  // near 0, which the entropy's gradient takes
  constexpr bool kTwo = DT == CE_F32 || ENT;
  const double c = ((double)top + (double)s.y) * (double)kLog2e;
  const float c_hi = (float)c, c_lo = kTwo ? (float)(c - (double)c_hi) : 0.f;
  const float slope = ENT ? __builtin_fmaf(dh, s.w, G) : G, bend = ENT ? dh * kLn2f : 0.f;
  const auto exponent = [&](float x) {
    const float t = __builtin_fmaf(x, kLog2e, -c_hi);
    return kTwo ? t - c_lo : t;
  };
  store_chunk<DT, T, P>(out + (size_t)lo * EB, cols, v, [&](const u32x4v& x) {
    float f[E];
    unpack_vec<DT>(x, f);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float t = exponent(f[e]), p = exp2_hw(t);
      if constexpr (ENT)  // p = 0 of a masked column takes the 0, not its log's infinity
        f[e] = -p * __builtin_fmaf(fmaxf(t, kFar), bend, slope);
      else
        f[e] = -p * slope;
    }
    return pack_vec<DT>(f);
  });
  if (L == 0) return;
  __syncthreads();
  if (mine) {
    float own = g;
    if (L > 1) {
      own = 0.f;
      for (uint32_t i = 0; i < L; ++i) own += sid[i] == id ? sg[i] : 0.f;
    }
    // own - p (G + ...) without a cancellation at p near 1: own (1 - p) - p (G - own + ...)
    const float t = exponent(xt), p = exp2_hw(t);
    const float q = xt == top && s.z < 0.5f ? s.z : 1.f - p;
    const float others = L > 1 ? G - own : 0.f;
    const float h = ENT ? dh * __builtin_fmaf(fmaxf(t, kFar), kLn2f, s.w) : 0.f;
    store_logit<DT>(out, id, __builtin_fmaf(own, q, -p * (others + h)));
  }
}

// Shapes (threads, vectors a thread and batch); logprob_plan chooses
constexpr FusedShape kShapes[] = {{64, 4}, {64, 8}, {256, 2}, {256, 8}};

template <int DT, int T, int P>
void launch_flags(const LogprobArgs& a, dim3 grid, hipStream_t stream) {
  const uint32_t lds = a.K > 0 ? hit_room(a.K) * (T / 64) * 20u : 0u;
#define VCE_LP(TOP, ENT) hipLaunchKernelGGL((k_logprobs<DT, T, P, TOP, ENT>), grid, dim3(T), lds, stream, a)
  if (a.K > 0) {
    if (a.entropy) VCE_LP(true, true);
    else VCE_LP(true, false);
  } else {
    if (a.entropy) VCE_LP(false, true);
    else VCE_LP(false, false);
  }
#undef VCE_LP
}
template <int DT>
void launch_shape(const LogprobArgs& a, dim3 grid, hipStream_t stream) {
  if (a.shape == 0) launch_flags<DT, kShapes[0].threads, kShapes[0].vecs>(a, grid, stream);
  else if (a.shape == 1) launch_flags<DT, kShapes[1].threads, kShapes[1].vecs>(a, grid, stream);
  else if (a.shape == 2) launch_flags<DT, kShapes[2].threads, kShapes[2].vecs>(a, grid, stream);
  else launch_flags<DT, kShapes[3].threads, kShapes[3].vecs>(a, grid, stream);
}

int64_t vec_cols(int32_t dtype) { return dtype == CE_BF16 ? 8 : 4; }
int64_t shape_cols(int s, int32_t dtype) { return (int64_t)kShapes[s].threads * kShapes[s].vecs * vec_cols(dtype); }
// even shares of whole vectors
int64_t share_cols(int64_t V, int64_t chunks, int64_t vec) { return ((V + chunks - 1) / chunks + vec - 1) / vec * vec; }

}  // namespace

int64_t logprob_max_cols(int32_t dtype) { return (int64_t)1 << (dtype == CE_BF16 ? 20 : 19); }

void logprob_plan(int64_t N, int64_t V, int32_t dtype, int32_t* shape, int64_t* chunks, int64_t* chunk_cols) {
  // Many rows, or short ones: a workgroup a row, a batch of its shape or more; few long ones: chunks of a batch at least, for
  // two workgroups a CU, or four of the smaller shape.  us with the entropy, with 20 and with 128 alternatives:
  //   64 x 128000 FP32 in 8 chunks 13.6, 22.2, 30.4; in 4: 15.8, 23.9, 32.9; in 16: 13.9, 21.6, 30.6
  //   700 x 128000 BF16 a row 39.6, 43.8, 53.1; in two 44.1, 54.5, 79.5
  //   300 x 128000 BF16 in two 25.6, 32.7, 43.2; a row 28.4, 34.4, 42.4
  //   300 x 32003 FP32, four batches, a row 15.1, 20.3, 26.7; in two 16.4, 23.1, 30.8
  //   one row of 128000 BF16, 20 alternatives: 12 in 32 chunks of the smaller shape, 14 in 8 to 16 larger ones
  // K has no part in it, so that what is asked for beside changes no log-probability.
  const auto batches = [=](int s) { return (V + shape_cols(s, dtype) - 1) / shape_cols(s, dtype); };
  const auto chunks_for = [=](int s, int64_t groups) {
    const int64_t want = (groups + N - 1) / (N > 0 ? N : 1), most = batches(s) < kMaxChunks ? batches(s) : kMaxChunks;
    return want < most ? want : most;
  };
  *chunks = 1;
  if (batches(1) == 1) {  // a wave a row (22369 x 3000 BF16 with the entropy: 43 us, 72 by 256 threads)
    *shape = batches(0) == 1 ? 0 : 1;
  } else if (N >= 512 || (N >= 256 && batches(3) <= 4)) {
    *shape = batches(2) <= 2 ? 2 : 3;
  } else if (N * batches(3) >= 256) {
    *shape = 3;
    *chunks = chunks_for(3, 512);
  } else {
    *chunks = chunks_for(2, 1024);
    *shape = batches(2) <= *chunks ? 2 : 3;
  }
  *chunk_cols = share_cols(V, *chunks, vec_cols(dtype));
  *chunks = (V + *chunk_cols - 1) / *chunk_cols;  // whole vectors can leave the last share empty
}

size_t logprob_workspace(int64_t N, int64_t V, int32_t dtype, int32_t K) {
  int32_t shape;
  int64_t chunks, cols;
  logprob_plan(N, V, dtype, &shape, &chunks, &cols);
  if (chunks == 1 || N == 0) return 0;
  const size_t words = kStatWords + 2 * (size_t)K;
  return chunk_words_at(N) + (size_t)N * chunks * words * 8;
}

hipError_t launch_logprobs(LogprobArgs a, void* ws, hipStream_t stream, hipEvent_t ev0, hipEvent_t ev1) {
  hipError_t e = hipSuccess;
  if (ev0 && (e = hipEventRecord(ev0, stream)) != hipSuccess) return e;
  if (a.chunks > 1) {
    a.hdr = static_cast<WsHeader*>(ws);
    a.done = reinterpret_cast<unsigned long long*>(static_cast<char*>(ws) + row_words_at(a.N));
    a.slots = reinterpret_cast<unsigned long long*>(static_cast<char*>(ws) + chunk_words_at(a.N));
    a.ws_bytes = logprob_workspace(a.N, a.V, a.dtype, a.K);
  }
  const int64_t rows = kMaxGridItems / a.chunks;  // a launch
  for (a.row0 = 0; a.row0 < a.N; a.row0 += rows) {
    const int64_t n = a.N - a.row0 < rows ? a.N - a.row0 : rows;
    const dim3 grid((uint32_t)(n * a.chunks));
    if (a.dtype == CE_BF16) launch_shape<CE_BF16>(a, grid, stream);
    else launch_shape<CE_F32>(a, grid, stream);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (ev1) e = hipEventRecord(ev1, stream);
  return e;
}

hipError_t launch_logprobs_bwd(LogprobGradArgs a, hipStream_t stream, hipEvent_t ev0, hipEvent_t ev1) {
  hipError_t e = hipSuccess;
  if (ev0 && (e = hipEventRecord(ev0, stream)) != hipSuccess) return e;
  const int64_t most = (int64_t)kLogprobBwdT * kLogprobBwdP * vec_cols(a.dtype);
  a.chunks = (a.V + most - 1) / most;
  a.chunk_cols = share_cols(a.V, a.chunks, vec_cols(a.dtype));
  a.chunks = (a.V + a.chunk_cols - 1) / a.chunk_cols;
  const int64_t rows = kMaxGridItems / a.chunks > 0 ? kMaxGridItems / a.chunks : 1;
  for (a.row0 = 0; a.row0 < a.N; a.row0 += rows) {
    const int64_t n = a.N - a.row0 < rows ? a.N - a.row0 : rows;
    const dim3 grid((uint32_t)(n * a.chunks)), block(kLogprobBwdT);
    if (a.dtype == CE_BF16) {
      if (a.dentropy) hipLaunchKernelGGL((k_logprobs_bwd<CE_BF16, true>), grid, block, 0, stream, a);
      else hipLaunchKernelGGL((k_logprobs_bwd<CE_BF16, false>), grid, block, 0, stream, a);
    } else {
      if (a.dentropy) hipLaunchKernelGGL((k_logprobs_bwd<CE_F32, true>), grid, block, 0, stream, a);
      else hipLaunchKernelGGL((k_logprobs_bwd<CE_F32, false>), grid, block, 0, stream, a);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (ev1) e = hipEventRecord(ev1, stream);
  return e;
}

}  // namespace vce
