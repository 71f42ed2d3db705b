// Token log-probabilities: of given tokens, the entropy and the K likeliest
// alternatives of every row, from one read of the logits; and their gradient.
//
// With m = max_j x_j and D = sum_j exp(x_j - m):
//   log p_t = (x_t - m) - log D
//   H       = log D - sum_j exp(x_j - m) (x_j - m) / D
//   dx_v    = sum_i g_i [v = t_i] - p_v (sum_i g_i + dH (log p_v + H))
//
// D's largest term is 1, and it is counted apart from the others' sum R: a row with
// one column at the maximum has log D = log1p(R) and 1 - p_max = R / (1 + R), so
// log-probabilities and entropies near 0, and the gradient of a token whose
// probability is near 1, keep their digits.  Exponentials are base 2 on the hardware's
// v_exp_f32, against m2 = fl(m log2 e); the sums are brought from m2 to the exact m log2 e
// at the end.
//
// Bound: the read of the logits (the gradient: and its write).  A workgroup holds
// a chunk of one row in registers, loaded at once.  What each chunk finds (m, R, the
// entropy's sum, its K largest keys) goes to the row's last chunk by tagged words.
//
// The K largest of a chunk without sorting it: the K-th largest of its threads'
// maxima, found bit by bit with ballots, is a bound that at least K columns reach and
// few others do; the columns that reach it are collected in LDS and ranked by counting.
// Where too many reach it (constant rows, masked ones: all -inf) the exact K-th
// value is found the same way over all columns, and of its ties the lowest columns are
// taken.  Keys order by value, then by column, so nothing depends on scheduling.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ce_internal.h"
#include "ce_row.h"

namespace vce {
namespace {

constexpr int kTop = kLogprobMaxList;  // most alternatives, and most given tokens, of a row
constexpr int kCand = 1024;            // candidates of a chunk that LDS holds
constexpr int kMerge = 1024;           // keys merged at a time
constexpr int kLocalBits = 15;         // a chunk has at most 2^15 columns
constexpr uint32_t kLocalMask = (1u << kLocalBits) - 1;
constexpr int kStatWords = 4;          // m, R, columns at the maximum, the entropy's sum
static_assert(kMerge / kTop >= 2, "a merge takes the list so far and at least one more");

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

// A chunk's key: order, then the lower column.  BF16's fits 32 bits and one exchange word.
template <int DT>
struct KeyT;
template <>
struct KeyT<CE_BF16> {
  typedef uint32_t Key;
  static constexpr int kWords = 1;
};
template <>
struct KeyT<CE_F32> {
  typedef unsigned long long Key;
  static constexpr int kWords = 2;
};
template <int DT>
__device__ __forceinline__ typename KeyT<DT>::Key chunk_key(uint32_t order, uint32_t local) {
  return (typename KeyT<DT>::Key)order << kLocalBits | (kLocalMask - local);
}
// A row's key: order << 32 | ~column.
template <int DT>
__device__ __forceinline__ unsigned long long row_key(typename KeyT<DT>::Key k, uint32_t lo) {
  if (k == 0) return 0ull;
  const uint32_t local = kLocalMask - ((uint32_t)k & kLocalMask);
  return (unsigned long long)(k >> kLocalBits) << 32 | (uint32_t)~(lo + local);
}

// The largest t whose bits are found from the top such that count(t) >= K (0: none).
template <int BITS, typename Count>
__device__ __forceinline__ uint32_t kth_largest(uint32_t K, Count count) {
  uint32_t t = 0;
#pragma unroll 1
  for (int b = BITS - 1; b >= 0; --b) {
    const uint32_t c = t | 1u << b;
    if (count(c) >= K) t = c;
  }
  return t;
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

// The K largest keys of a chunk of at least K columns, exactly, where a bound `t` that
// `reach` columns reach let too many through, or too few (NaN, which maxima pass over): the
// K-th largest value over all columns (the bound itself where fewer than K exceed it),
// every column above it, and its ties from the lowest column on.  Leaves K keys in cand[].
template <int DT, int T, int P>
__device__ __forceinline__ void exact_largest(const u32x4v (&v)[P], uint32_t cols, uint32_t K, uint32_t t,
                                              uint32_t reach, typename KeyT<DT>::Key* cand, uint32_t* n_cand,
                                              uint32_t* sh) {
  constexpr int E = LogitT<DT>::E;
  const uint32_t tid = threadIdx.x;
  const auto count = [&](uint32_t at_least) {
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      u32x4v w = v[j];
      relaunch(w);  // the orders are formed again in each round, not kept in registers
      float f[E];
      unpack_vec<DT>(w, f);
#pragma unroll
      for (int e = 0; e < E; ++e) c += (j * T + tid) * E + e < cols && order_of<DT>(f[e]) >= at_least;
    }
    return block_count<T>(c, sh);
  };
  uint32_t above = count(t + 1);
  if (above >= K || reach < K) {
    t = kth_largest<kOrderBits<DT>>(K, count);
    above = count(t + 1);
  }
  if (tid == 0) *n_cand = 0;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < P; ++j) {
    float f[E];
    unpack_vec<DT>(v[j], f);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint32_t c = (j * T + tid) * E + e, o = order_of<DT>(f[e]);
      if (c < cols && o > t) cand[atomicAdd(n_cand, 1u)] = chunk_key<DT>(o, c);
    }
  }
  uint32_t have = above;
#pragma unroll
  for (int j = 0; j < P; ++j) {  // columns rise with j, then with the thread, then within the vector
    if (have >= K) continue;     // the same for the whole workgroup
    float f[E];
    unpack_vec<DT>(v[j], f);
    uint32_t mine = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) mine += (j * T + tid) * E + e < cols && order_of<DT>(f[e]) == t;
    uint32_t upto = mine;  // inclusive over the wave's lanes
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t u = (uint32_t)__shfl_up((int)upto, o);
      upto += (tid & 63) >= (uint32_t)o ? u : 0u;
    }
    __syncthreads();
    if ((tid & 63) == 63) sh[tid >> 6] = upto;
    __syncthreads();
    uint32_t at = have + upto - mine, all = 0;
#pragma unroll
    for (int i = 0; i < T / 64; ++i) {
      at += (uint32_t)i < tid >> 6 ? sh[i] : 0u;
      all += sh[i];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint32_t c = (j * T + tid) * E + e;
      if (c < cols && order_of<DT>(f[e]) == t) {
        if (at < K) cand[at] = chunk_key<DT>(t, c);
        ++at;
      }
    }
    have += all;
  }
  if (tid == 0) *n_cand = K;
  __syncthreads();
}

// Descending lists of K keys (0: none) in `a`, nl of them, merged to one; `b` is room for as many.
// Returns where it is.  The caller's writes of `a` are visible.
template <int T>
__device__ unsigned long long* merge_lists(unsigned long long* a, unsigned long long* b, uint32_t nl, uint32_t K) {
  while (nl > 1) {
    for (uint32_t i = threadIdx.x; i < nl * K; i += T) {
      const uint32_t l = i / K, at = i - l * K, other = l ^ 1u;
      const unsigned long long key = a[i];
      uint32_t rank = at;
      if (other < nl) {
        const unsigned long long* o = a + other * K;
        uint32_t lo = 0, hi = K;  // how many of the other list's keys are larger
        while (lo < hi) {
          const uint32_t mid = (lo + hi) >> 1;
          if (o[mid] > key) lo = mid + 1;
          else hi = mid;
        }
        rank += lo;
      }
      if (rank < K) b[(l >> 1) * K + rank] = key;
    }
    __syncthreads();
    unsigned long long* const t = a;
    a = b;
    b = t;
    nl = (nl + 1) >> 1;
  }
  return a;
}

// What a row comes to, the same in every thread.
struct RowSum {
  float m, logd;
  float rest;    // sum of exp(x - m) but for one column at the maximum
  float s1;      // sum of exp(x - m) (x - m) log2 e
  float at_max;  // columns counted as exactly 1
};
// (at_max - 1 further columns at the maximum are counted in D beside rest)
__device__ __forceinline__ float log_of_sum(const RowSum& s) {
  return s.at_max == 1.f ? log1pf(s.rest) : logf(s.rest + s.at_max);
}

template <int DT, int T, int P, bool TOP, bool ENT>
__global__ __launch_bounds__(T) void k_logprobs(LogprobArgs a) {
  typedef typename KeyT<DT>::Key Key;
  constexpr int E = LogitT<DT>::E, EB = LogitT<DT>::EB, W = T / 64;
  constexpr int KW = KeyT<DT>::kWords;
  constexpr int TK = (kTop + T - 1) / T;  // given tokens a thread
  __shared__ float sh_max[W];
  __shared__ float sh_sum[W][4];
  __shared__ float st[kMaxChunks][kStatWords];
  __shared__ uint32_t sh_cnt[W];
  __shared__ uint32_t lane_top[TOP ? T : 1];
  __shared__ uint32_t n_cand;
  __shared__ __align__(16) unsigned long long keys[TOP ? 2 * kMerge : 1];  // candidates, later the lists
  Key* const cand = reinterpret_cast<Key*>(keys);
  static_assert(kCand * sizeof(Key) <= 2 * kMerge * 8, "candidates fit");

  const uint32_t tid = threadIdx.x, wave = tid >> 6;
  const uint32_t C = (uint32_t)a.chunks, K = TOP ? (uint32_t)a.K : 0u;
  const uint32_t in_launch = blockIdx.x / C;
  const int64_t r = a.row0 + in_launch;
  const uint32_t k = blockIdx.x - in_launch * C;
  const bool last = k == C - 1;  // the row's last chunk brings it together
  WsView ws{0u, true, 0ull};
  if (C > 1) ws = view_workspace(a.hdr, a.ws_bytes);
  const int64_t i0 = r / a.d1, i1 = r - i0 * a.d1;
  const char* const row = a.x + (i0 * a.s0 + i1 * a.s1) * EB;
  const uint32_t lo = k * (uint32_t)a.chunk_cols;
  const uint32_t cols = (uint32_t)a.V - lo < (uint32_t)a.chunk_cols ? (uint32_t)a.V - lo : (uint32_t)a.chunk_cols;

  // ---- the given tokens' ids go out first, then the chunk, then the tokens' logits
  const int64_t* const ids = a.ids ? a.ids + i0 * a.is0 + i1 * a.is1 : nullptr;
  int64_t id[TK];
#pragma unroll
  for (int i = 0; i < TK; ++i) id[i] = last && (int)(i * T + tid) < a.M ? ids[i * T + tid] : -1;
  u32x4v v[P];
  load_chunk<DT, T, P>(row + (size_t)lo * EB, cols, v);
  float xt[TK];
#pragma unroll
  for (int i = 0; i < TK; ++i) xt[i] = id[i] >= 0 && id[i] < a.V ? load_logit<DT>(row, id[i]) : 0.f;
  if (TOP && tid == 0) n_cand = 0;

  // ---- maxima
  float vm[P], m = -INFINITY;
#pragma unroll
  for (int j = 0; j < P; ++j) {
    vm[j] = largest<DT>(v[j], -INFINITY);
    m = fmaxf(m, vm[j]);
  }
  if constexpr (TOP && W > 1) lane_top[tid] = tid * E < cols ? order_of<DT>(m) : 0u;
  m = wave_largest(m);
  if ((tid & 63) == 0) sh_max[wave] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < W; ++i) m = fmaxf(m, sh_max[i]);
  const float m2 = m == -INFINITY ? 0.f : m * kLog2e;

  // ---- sums: a vector that reaches the maximum leaves one such column out
  float s0 = 0.f, s1 = 0.f, at_max = 0.f;
#pragma unroll
  for (int j = 0; j < P; ++j) {
    relaunch(v[j]);
    float f[E], e[E];
    unpack_vec<DT>(v[j], f);
    float t = 0.f, h = 0.f;
    const auto exponent = [&](int c) { return __builtin_fmaf(f[c], kLog2e, -m2); };
    // (2^-1000 is 0, and 0 times a masked column's -inf would be NaN)
    const auto bent = [&](int c) { return e[c] * fmaxf(exponent(c), -1000.f); };
#pragma unroll
    for (int c = 0; c < E; ++c) {
      e[c] = exp2_hw(exponent(c));
      if constexpr (ENT) h += bent(c);
    }
#pragma unroll
    for (int c = 0; c < E; c += 2) t += e[c] + e[c + 1];
    if (vm[j] == m && m != -INFINITY) {
      int own = E - 1;
#pragma unroll
      for (int c = E - 1; c >= 0; --c) own = f[c] == m ? c : own;
      t = h = 0.f;
#pragma unroll
      for (int c = 0; c < E; ++c) {
        t += c == own ? 0.f : e[c];
        if constexpr (ENT) h += c == own ? 0.f : bent(c);
      }
      at_max += 1.f;
    }
    s0 += t;
    if constexpr (ENT) s1 += h;
  }
  s0 = wave_sum(s0);
  at_max = wave_sum(at_max);
  if constexpr (ENT) s1 = wave_sum(s1);
  if ((tid & 63) == 0) {
    sh_sum[wave][0] = s0;
    sh_sum[wave][1] = at_max;
    sh_sum[wave][2] = s1;
  }

  // ---- the K largest
  if constexpr (TOP) {
    constexpr int G = W > 1 ? W : P;  // group maxima a lane: threads' or, in one wave, vectors'
    uint32_t g[G];
#pragma unroll
    for (int i = 0; i < G; ++i) {
      if constexpr (W > 1) g[i] = lane_top[i * 64 + (tid & 63)];
      else g[i] = (i * T + tid) * E < cols ? order_of<DT>(vm[i]) : 0u;
    }
    const uint32_t bound = kth_largest<kOrderBits<DT>>(K, [&](uint32_t c) {
      uint32_t n = 0;
#pragma unroll
      for (int i = 0; i < G; ++i) n += (uint32_t)__builtin_popcountll(__ballot(g[i] >= c));
      return n;
    });
#pragma unroll
    for (int j = 0; j < P; ++j) {
      if (order_of<DT>(vm[j]) < bound) continue;
      float f[E];
      unpack_vec<DT>(v[j], f);
#pragma unroll
      for (int c = 0; c < E; ++c) {
        const uint32_t o = order_of<DT>(f[c]), local = (j * T + tid) * E + c;
        if (o >= bound && local < cols) {
          const uint32_t at = atomicAdd(&n_cand, 1u);
          if (at < (uint32_t)kCand) cand[at] = chunk_key<DT>(o, local);
        }
      }
    }
    __syncthreads();
    const uint32_t reach = n_cand;
    if (reach > (uint32_t)kCand || reach < (cols < K ? cols : K))
      exact_largest<DT, T, P>(v, cols, K, bound, reach, cand, &n_cand, sh_cnt);
  } else {
    __syncthreads();
  }
  s0 = at_max = s1 = 0.f;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    s0 += sh_sum[i][0];
    at_max += sh_sum[i][1];
    s1 += sh_sum[i][2];
  }
  RowSum sum;
  {
    // from m2 to m log2 e: the terms are too large by 2^d, d = m log2 e - m2
    const float d = m == -INFINITY || m == INFINITY ? 0.f : __builtin_fmaf(m, kLog2e, -m2);
    const float grow = __builtin_fmaf(-d, kLn2f, 1.f);
    sum.m = m;
    sum.rest = s0 * grow;
    sum.at_max = at_max;
    sum.s1 = (s1 - d * s0) * grow;
  }

  unsigned long long* top = keys;
  if (C > 1) {
    const uint32_t words = kStatWords + K * KW;
    unsigned long long* const slot = a.slots + ((size_t)r * C + k) * words;
    const bool keep = withheld(ws, r, (int)k);
    if (tid == 0 && !keep) {
      put_word(slot + 0, ws.tag, __float_as_uint(sum.m));
      put_word(slot + 1, ws.tag, __float_as_uint(sum.rest));
      put_word(slot + 2, ws.tag, __float_as_uint(sum.at_max));
      put_word(slot + 3, ws.tag, __float_as_uint(sum.s1));
    }
    if constexpr (TOP) {
      const uint32_t n = n_cand;
      for (uint32_t i = tid; i < (n > K ? n : K); i += T) {
        Key key = 0;
        uint32_t rank = i;
        if (i < n) {
          key = cand[i];
          rank = 0;
          for (uint32_t q = 0; q < n; ++q) rank += cand[q] > key;
        }
        if (rank < K && !keep) {
          put_word(slot + kStatWords + rank * KW, ws.tag, (uint32_t)key);
          if constexpr (KW == 2) put_word(slot + kStatWords + rank * KW + 1, ws.tag, (uint32_t)(key >> 32));
        }
      }
    }
    if (!last) return;

    // ---- the row's last chunk collects
    uint32_t spins = 0;
    bool ok = ws.ok;
    const unsigned long long* const slots = a.slots + (size_t)r * C * words;
    for (uint32_t i = tid; i < C * kStatWords; i += T) {
      const unsigned long long* p = slots + (size_t)(i / kStatWords) * words + i % kStatWords;
      uint32_t w = 0x7fc00000u;
      ok &= await_word(p, ws.tag, peek_word(p), spins, &w);
      st[i / kStatWords][i % kStatWords] = __uint_as_float(w);
    }
    if constexpr (TOP) {
      const uint32_t most = (uint32_t)kMerge / K;  // lists at a time
      uint32_t done = 0, held = 0;                 // chunks taken, lists in front (the result so far)
      unsigned long long* b = keys + kMerge;
      __syncthreads();  // every thread has ranked its candidates
      while (done < C) {
        const uint32_t take = C - done < most - held ? C - done : most - held;
        for (uint32_t i = tid; i < take * K; i += T) {
          const uint32_t c = done + i / K;
          const unsigned long long* p = slots + (size_t)c * words + kStatWords + (i % K) * KW;
          const unsigned long long w0 = peek_word(p), w1 = KW == 2 ? peek_word(p + KW - 1) : 0ull;
          uint32_t k0 = 0, k1 = 0;
          bool got = await_word(p, ws.tag, w0, spins, &k0);
          if constexpr (KW == 2) got &= await_word(p + 1, ws.tag, w1, spins, &k1);
          ok &= got;
          const Key key = KW == 2 ? (Key)((unsigned long long)k1 << 32 | k0) : (Key)k0;
          top[(held + i / K) * K + i % K] = got ? row_key<DT>(key, c * (uint32_t)a.chunk_cols) : 0ull;
        }
        __syncthreads();
        unsigned long long* const out = merge_lists<T>(top, b, held + take, K);
        b = out == top ? b : top;
        top = out;
        done += take;
        held = 1;
      }
    }
    ok = __syncthreads_and(ok);
    if (!ok && tid == 0) atomicOr(&a.hdr->status, ws.ok ? 1u : 2u);
    // lane c of every wave takes chunk c
    const uint32_t c = tid & 63;
    const bool has = c < C;
    const float mc = has ? st[c][0] : -INFINITY;
    m = wave_largest(mc);
    const bool some = has && mc != -INFINITY, best = some && mc == m;
    const float dm = some ? (mc - m) * kLog2e : 0.f, w = exp2_hw(dm);
    const float rc = some ? st[c][1] : 0.f, nc = some ? st[c][2] : 0.f, sc = some ? st[c][3] : 0.f;
    // a chunk whose maximum is NaN (it holds nothing else) carries it in its sum
    const float carry = has && mc == -INFINITY && st[c][1] != st[c][1] ? st[c][1] : 0.f;
    sum.m = m;
    sum.rest = wave_sum((best ? rc : (rc + nc) * w) + carry);
    sum.at_max = wave_sum(best ? nc : 0.f);
    if constexpr (ENT) sum.s1 = wave_sum(some ? __builtin_fmaf(dm, rc + nc, sc) * w : 0.f);
    if (!ok) sum.rest = __uint_as_float(0x7fc00000u);
    if (TOP && !ok) {
      for (uint32_t i = tid; i < K; i += T) top[i] = 0ull;
      __syncthreads();
    }
  } else if constexpr (TOP) {
    // one chunk: its ranks are the row's (K is at most the number of columns)
    const uint32_t n = n_cand;
    uint32_t rank[(kCand + T - 1) / T];
    Key key[(kCand + T - 1) / T];
#pragma unroll
    for (int i = 0; i < (kCand + T - 1) / T; ++i) {
      const uint32_t at = i * T + tid;
      rank[i] = K;
      if (i * T < (int)n && at < n) {
        key[i] = cand[at];
        rank[i] = 0;
        for (uint32_t q = 0; q < n; ++q) rank[i] += cand[q] > key[i];
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < (kCand + T - 1) / T; ++i)
      if (rank[i] < K) keys[rank[i]] = row_key<DT>(key[i], 0u);
    __syncthreads();
  }

  // ---- the row's outputs (+inf has no distribution either)
  if (sum.m == INFINITY) sum.rest = __uint_as_float(0x7fc00000u);
  sum.logd = log_of_sum(sum);
  const float logd = sum.logd;
#pragma unroll
  for (int i = 0; i < TK; ++i) {
    const int at = i * T + tid;
    if (at < a.M) {
      const int64_t t = id[i];
      float lp = (xt[i] - sum.m) - logd;
      if (t < 0 || t >= a.V) lp = __uint_as_float(0x7fc00000u);
      if (t == a.ignore_idx) lp = 0.f;
      a.logp[r * a.M + at] = lp;
    }
  }
  if constexpr (TOP) {
    for (uint32_t i = tid; i < K; i += T) {
      const unsigned long long key = top[i];
      const float f = value_of<DT>((uint32_t)(key >> 32));
      a.top_ids[r * K + i] = key ? (int64_t)(uint32_t)~(uint32_t)key : -1;
      a.top_logp[r * K + i] = key ? (f - sum.m) - logd : __uint_as_float(0x7fc00000u);
    }
  }
  if (tid == 0) {
    const float D = sum.rest + sum.at_max;
    const float h = ENT ? __builtin_fmaf(-kLn2f, sum.s1 / D, logd) : 0.f;
    if (ENT) a.entropy[r] = h;
    if (a.lse) a.lse[r] = sum.m + logd;
    if (a.stats)
      reinterpret_cast<float4*>(a.stats)[r] =
          make_float4(sum.m, logd, sum.at_max == 1.f ? sum.rest / D : 1.f - 1.f / D, h);
  }

  // ---- the last row's workgroup ends the call once every row has been brought together
  if (C > 1) {
    if (tid == 0) put_word(a.done + r, ws.tag, 0u);
    if (r != a.N - 1) return;
    uint32_t spins = 0, w;
    bool ok = true;
    for (int64_t base = 0; base < a.N; base += 4 * T) {
      unsigned long long first[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t at = base + i * T + tid;
        first[i] = peek_word(a.done + (at < a.N ? at : 0));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t at = base + i * T + tid;
        ok = ok && await_word(a.done + (at < a.N ? at : 0), ws.tag, first[i], spins, &w);
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
  const int64_t i0 = r / a.d1, i1 = r - i0 * a.d1;
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

  const bool counts = tid < L && id != a.ignore_idx;
  const bool valid = id >= 0 && id < a.V;
  const bool mine = counts && valid && id >= lo && id < (int64_t)lo + cols;
  if (!counts) g = 0.f;
  if (counts && !valid) g = __uint_as_float(0x7fc00000u);  // the row's gradient is NaN
  const float xt = mine ? load_logit<DT>(row, id) : 0.f;
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

  // p = 2^(x log2 e - c), c = (m + log D) log2 e in two parts; the second matters to FP32's rounding and to log p
  // near 0, which the entropy's gradient takes
  constexpr bool kTwo = DT == CE_F32 || ENT;
  const double c = ((double)s.x + (double)s.y) * (double)kLog2e;
  const float c_hi = (float)c, c_lo = kTwo ? (float)(c - (double)c_hi) : 0.f;
  const float slope = ENT ? __builtin_fmaf(dh, s.w, G) : G, bend = ENT ? dh * kLn2f : 0.f;
  const auto exponent = [&](float x) {
    const float t = __builtin_fmaf(x, kLog2e, -c_hi);
    return kTwo ? t - c_lo : t;
  };
#pragma unroll
  for (int j = 0; j < P; ++j) {
    float f[E];
    unpack_vec<DT>(v[j], f);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float t = exponent(f[e]), p = exp2_hw(t);
      if constexpr (ENT)  // p = 0 of a masked column takes the 0, not its log's infinity
        f[e] = -p * __builtin_fmaf(fmaxf(t, -1000.f), bend, slope);
      else
        f[e] = -p * slope;
    }
    store_vec<DT>(out + (size_t)lo * EB, cols, j * T + tid, pack_vec<DT>(f));
  }
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
    const float q = xt == s.x && s.z < 0.5f ? s.z : 1.f - p;
    const float others = L > 1 ? G - own : 0.f;
    const float h = ENT ? dh * __builtin_fmaf(fmaxf(t, -1000.f), kLn2f, s.w) : 0.f;
    store_logit<DT>(out, id, __builtin_fmaf(own, q, -p * (others + h)));
  }
}

// Chunk shapes (threads, vectors a thread); logprob_plan chooses
constexpr FusedShape kShapes[] = {{64, 4}, {256, 2}, {256, 8}};

template <int DT, int T, int P>
void launch_flags(const LogprobArgs& a, dim3 grid, hipStream_t stream) {
#define VCE_LP(TOP, ENT) hipLaunchKernelGGL((k_logprobs<DT, T, P, TOP, ENT>), grid, dim3(T), 0, stream, a)
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
  else launch_flags<DT, kShapes[2].threads, kShapes[2].vecs>(a, grid, stream);
}

int64_t vec_cols(int32_t dtype) { return dtype == CE_BF16 ? 8 : 4; }
int64_t shape_cols(int s, int32_t dtype) { return (int64_t)kShapes[s].threads * kShapes[s].vecs * vec_cols(dtype); }
// even shares of whole vectors
int64_t share_cols(int64_t V, int64_t chunks, int64_t vec) { return ((V + chunks - 1) / chunks + vec - 1) / vec * vec; }

}  // namespace

int64_t logprob_max_cols(int32_t dtype) { return shape_cols(2, dtype) * kMaxChunks; }

void logprob_plan(int64_t N, int64_t V, int32_t dtype, int32_t* shape, int64_t* chunks, int64_t* chunk_cols) {
  const auto pieces = [=](int s) { return (V + shape_cols(s, dtype) - 1) / shape_cols(s, dtype); };
  *shape = V <= shape_cols(0, dtype) ? 0 : N * pieces(2) < 256 && pieces(1) <= kMaxChunks ? 1 : 2;
  *chunks = pieces(*shape);
  *chunk_cols = share_cols(V, *chunks, vec_cols(dtype));
  *chunks = (V + *chunk_cols - 1) / *chunk_cols;  // whole vectors can leave the last share empty
}

size_t logprob_workspace(int64_t N, int64_t V, int32_t dtype, int32_t K) {
  int32_t shape;
  int64_t chunks, cols;
  logprob_plan(N, V, dtype, &shape, &chunks, &cols);
  if (chunks == 1 || N == 0) return 0;
  const size_t words = kStatWords + (size_t)K * (dtype == CE_BF16 ? 1 : 2);
  return kWsHeaderBytes + (size_t)N * 8 + (size_t)N * chunks * words * 8;
}

hipError_t launch_logprobs(LogprobArgs a, void* ws, hipStream_t stream, hipEvent_t ev0, hipEvent_t ev1) {
  hipError_t e = hipSuccess;
  if (ev0 && (e = hipEventRecord(ev0, stream)) != hipSuccess) return e;
  if (a.chunks > 1) {
    a.hdr = static_cast<WsHeader*>(ws);
    a.done = reinterpret_cast<unsigned long long*>(static_cast<char*>(ws) + kWsHeaderBytes);
    a.slots = a.done + a.N;
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
