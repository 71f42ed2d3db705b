// Distillation from a teacher's top logits: the loss of every row and its gradient,
// one read of the student's logits and one write of the gradient.
//
// Row of logits x, temperature T, the teacher's K entries (column c_k, value t_k):
//   q = softmax(x / T)
//   p_k = softmax_k(t / T), and nothing is left (r = 0), or p_k = exp(t_k), r = max(0, 1 - sum_k p_k)
//   loss = T^2 (sum_k p_k (log p_k - log q_ck) + r (log r - log q_o)),  q_o = sum of q over unnamed columns
//   dx_v = s T (q_v S - P_v - [v unnamed] q_v r / q_o),   S = sum_k p_k + r, P_v = sum of p_k with c_k = v
//
// The sum of the exponentials is taken over the unnamed columns alone (the named ones
// are set to -inf in their registers, found by a bitmap of the chunk in LDS), relative to
// their own maximum; the named ones, a few, are added in 64 bits.  So q_o keeps its digits
// where the named columns hold nearly everything, and so does q_c - p_c, whose terms
// are both near 1 there: the largest term of the row is the same number in q_c and in the sum.
// All that is per entry or per row is 64-bit, by one wave, while the others wait; their loads are under way then.
//
// Bound: one read and one write of the logits.  A chunk of a row stays in a
// workgroup's registers between its sums and its gradient, and a row's chunks exchange
// eight words each through the workspace, as in ce_fwd_bwd_fused (whose chunk shapes these are).
// The loss alone is brought together by a row's last chunk, and no other waits.  A call among others, 8192 x 128000
// BF16 with 64 entries: 696 us, 6.03 TB/s of the logits' bytes; 2048 x 32000 BF16 with 20 and lengths: 56 us, 4.7 TB/s, two
// of them the rows' count; the loss alone of 1024 x 128000 BF16, 56 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ce_internal.h"
#include "ce_row.h"

namespace vce {
namespace {

// what a chunk tells: its largest unnamed logit m and the sum of the unnamed columns; a reference for its named ones (a
// logit: the largest of all that the chunk has), their sum, and that of p times their exponents, both 64-bit, in two words
// each; sums are relative to powers of two near m and the reference.  (Less would show where a student is near its teacher
// and the loss is a small difference: log2 e / T in FP32 alone moves a loss of 2e-7 by up to 6e-4 of it and its gradient by
// 2e-3, one of 2e-9 by 4e-3 and 2e-2.  The eighth word is empty: 64 bytes a chunk, one word a lane for eight chunks.
// 8192 x 128000 BF16, 696 us: with seven words 6 us more, with nine 25 to 60, with weights by 64-bit exponentials in place
// of powers of two 10.)
enum { kMax, kRest, kRef, kSum, kCross = kSum + 2, kEmpty = kCross + 2, kWords };
constexpr int kEntries = kDistillMaxTop / 64;  // entries a lane of the wave that handles them
constexpr double kLn2d = 0.693147180559945309417, kLog2eD = 1.442695040888963407360;

typedef uint32_t Words2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void put64(uint32_t* w, double v) {
  const Words2 b = __builtin_bit_cast(Words2, v);
  w[0] = b.x;
  w[1] = b.y;
}
__device__ __forceinline__ double get64(const uint32_t* w) { return __builtin_bit_cast(double, Words2{w[0], w[1]}); }

// 2^x: 2^n times the Taylor series of 2^f, |f| <= 1/2, to (f ln 2)^13 / 13!, 2e-17 of it.  Shorter than the library's,
// whose code takes longer to fetch than to run.
__device__ __forceinline__ double exp2_64(double x) {
  x = x < -1100.0 ? -1100.0 : x;
  const double n = rint(x), y = (x - n) * kLn2d;
  double p = 1.0 / 6227020800.0;
  constexpr double kInv[] = {1.0 / 479001600, 1.0 / 39916800, 1.0 / 3628800, 1.0 / 362880, 1.0 / 40320, 1.0 / 5040,
                             1.0 / 720,       1.0 / 120,      1.0 / 24,      1.0 / 6,      0.5,         1.0, 1.0};
#pragma unroll
  for (int i = 0; i < 13; ++i) p = fma(p, y, kInv[i]);
  return ldexp(p, (int)n);
}
// log2 x, x >= 0 and normal: of the mantissa in [sqrt(1/2), sqrt 2), 2 atanh s with s = (m - 1) / (m + 1), |s| < 0.172,
// to s^21 / 21, 4e-18.
__device__ __forceinline__ double log2_64(double x) {
  double m = __builtin_amdgcn_frexp_mant(x);
  int e = __builtin_amdgcn_frexp_exp(x);
  const bool small = m < 0.70710678118654752;
  m = small ? m + m : m;
  e -= small ? 1 : 0;
  const double s = (m - 1.0) / (m + 1.0), s2 = s * s;
  double p = 1.0 / 21.0;
#pragma unroll
  for (int k = 19; k >= 1; k -= 2) p = fma(p, s2, 1.0 / k);
  return x == 0.0 ? -(double)INFINITY : fma(2.0 * kLog2eD * s, p, (double)e);
}
__device__ __forceinline__ double lane64(double v, int l) {
  typedef int i2 __attribute__((ext_vector_type(2)));
  const i2 w = __builtin_bit_cast(i2, v);
  const i2 r = {__builtin_amdgcn_readlane(w.x, l), __builtin_amdgcn_readlane(w.y, l)};
  return __builtin_bit_cast(double, r);
}

// In a split row the references of sums are powers of two, 2^n with n = rint(x log2 e / T) of a chunk's largest logit x:
// each chunk's is its own, and sums are brought together by exponents alone.  A column's exponent is
// fma(x, log2 e / T, -n), rounded once.  From 2^50 on logits are equal or too far apart to add up, and exponents are their
// differences from the reference, as they are in a row of one chunk.
__device__ __forceinline__ double power_of(float x, double kb) { return rint((double)x * kb); }
__device__ __forceinline__ double above(float x, float ref, double n, double kb) {
  return fabs(n) < 0x1p50 ? fma((double)x, kb, -n) : ((double)x - (double)ref) * kb;
}
__device__ __forceinline__ int steps(double d) { return (int)fmax(d, -2200.0); }  // (d <= 0; NaN is of sums that are 0 or NaN)

template <int T>
__device__ void finish_distill(const DistillArgs& a, uint32_t tag, bool ws_ok) {
  __shared__ double part[T / 64];
  uint32_t spins = 0;
  bool ok = true;
  double acc = 0.0;
  for (int64_t base = 0; base < a.N; base += 4 * T) {
    unsigned long long first[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t at = base + i * T + threadIdx.x;
      first[i] = peek_word(a.row_words + (at < a.N ? at : 0));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t at = base + i * T + threadIdx.x;
      uint32_t w = 0;
      ok = ok && await_word(a.row_words + (at < a.N ? at : 0), tag, first[i], spins, &w);
      acc += at < a.N ? (double)__uint_as_float(w) : 0.0;
    }
  }
  if (!ok) atomicOr(&a.hdr->status, 1u);
  acc = wave_sum64(acc);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = acc;
  ok = __syncthreads_and(ok);
  if (threadIdx.x != 0) return;
  if (a.reduce != CE_REDUCE_NONE) {
    double total = 0.0;
    for (int i = 0; i < T / 64; ++i) total += part[i];
    if (a.reduce == CE_REDUCE_MEAN) total /= (double)(a.n ? *a.n : (int32_t)a.N);
    a.loss[0] = ok && ws_ok ? (float)total : __uint_as_float(0x7fc00000u);
  }
  next_epoch(a.hdr);
}

// (Six waves a SIMD, 80 registers: 515 x 32003 FP32 32 us; left to the compiler, 35.)
// SPLIT: more than one chunk a row.  (One kernel for both: 65536 x 1000 BF16 with 20 logits 265 us, 215 apart.)
template <int DT, int T, int P, bool GRAD, bool SPLIT>
__global__ __launch_bounds__(T) __attribute__((amdgpu_waves_per_eu(6, 8))) void k_distill(DistillArgs a) {
  constexpr int E = LogitT<DT>::E, EB = LogitT<DT>::EB, W = T / 64;
  __shared__ float sh_max[W], sh_sum[W];
  __shared__ __align__(8) uint8_t named[T * 8];  // byte tid * 8 + j: which columns of slot j's vector are named
  __shared__ uint32_t words[kMaxChunks * kWords];
  __shared__ double kept_p[kDistillMaxTop], kept_e[kDistillMaxTop];  // the entries', over the exchange
  __shared__ uint32_t kept_col[kDistillMaxTop];
  __shared__ uint8_t kept_chunk[kDistillMaxTop];
  __shared__ float bc[2];  // the unnamed columns' exponents' offset, and their factor
  const uint32_t tid = threadIdx.x, lane = tid & 63;
  const uint32_t C = SPLIT ? (uint32_t)a.chunks : 1u;
  const uint32_t in_launch = SPLIT ? blockIdx.x / C : blockIdx.x;
  const int64_t r = a.row0 + in_launch;
  const uint32_t k = blockIdx.x - in_launch * C;
  WsView ws{0u, true, 0ull};
  if (a.hdr) ws = view_workspace(a.hdr, a.ws_bytes);
  const bool ends = a.hdr && r == a.N - 1 && k == C - 1;
  const int64_t i0 = (uint32_t)r / (uint32_t)a.d1, i1 = (uint32_t)r % (uint32_t)a.d1;
  const char* const row = a.x + (i0 * a.s0 + i1 * a.s1) * EB;
  char* const out = GRAD ? a.out + (i0 * a.os0 + i1 * a.os1) * EB : nullptr;
  const uint32_t lo = k * (uint32_t)a.chunk_cols;
  const uint32_t cols = (uint32_t)a.V - lo < (uint32_t)a.chunk_cols ? (uint32_t)a.V - lo : (uint32_t)a.chunk_cols;
  int L = a.K;
  if (a.len) {
    L = load_uniform(a.len + r);
    L = L < 0 ? 0 : L > a.K ? a.K : L;
  }
  const auto row_loss = [&](float loss) {  // by one thread of the row
    if (a.reduce == CE_REDUCE_NONE) a.loss[r] = loss;
    if (a.hdr) put_word(a.row_words + r, ws.tag, __float_as_uint(loss));
  };

  if (L == 0) {  // left out: loss 0, gradient 0, the logits not read
    if constexpr (GRAD) {
      u32x4v v[P] = {};
      store_chunk<DT, T, P>(out + (size_t)lo * EB, cols, v, [](const u32x4v&) { return u32x4v{0u, 0u, 0u, 0u}; });
    }
    if (k == 0 && tid == 0) row_loss(0.f);
  } else {
    // ---- wave 0's entries, then the chunk; while it comes in, the bitmap and the teacher's probabilities
    const float up = a.g ? load_uniform(a.g + (a.reduce == CE_REDUCE_NONE ? r : 0)) : 1.f;
    const int32_t count = a.reduce == CE_REDUCE_MEAN && a.n ? load_uniform(a.n) : (int32_t)a.N;
    int64_t id[kEntries];
    float tv[kEntries], xe[kEntries];
    if (tid < 64) {
      const int64_t* ids = a.ids + i0 * a.is0 + i1 * a.is1;
      const char* const t = a.teacher + (i0 * a.ts0 + i1 * a.ts1) * (a.tdtype == CE_BF16 ? 2 : 4);
#pragma unroll
      for (int i = 0; i < kEntries; ++i) {
        const int at = i * 64 + (int)lane;
        id[i] = -1;
        tv[i] = xe[i] = 0.f;
        if (at < L) {
          id[i] = ids[at];
          tv[i] = a.tdtype == CE_BF16 ? load_logit<CE_BF16>(t, at) : load_logit<CE_F32>(t, at);
        }
      }
    }
    u32x4v v[P];
    load_chunk<DT, T, P>(row + (size_t)lo * EB, cols, v);
    reinterpret_cast<uint64_t*>(named)[tid] = 0ull;
    __syncthreads();
    bool here[kEntries], first[kEntries];
    uint32_t col[kEntries];  // of the entries here; others have none
    double p[kEntries], mass = 0.0, plogp = 0.0;
    bool bad = false;
    if (tid < 64) {
#pragma unroll
      for (int i = 0; i < kEntries; ++i) {
        const bool is = i * 64 + (int)lane < L;
        bad |= is && (id[i] < 0 || id[i] >= a.V);
        here[i] = is && id[i] >= lo && id[i] < (int64_t)lo + cols;
        first[i] = false;
        col[i] = ~0u;
        if (here[i]) {
          const uint32_t c = (uint32_t)(id[i] - lo), vec = c / E;
          col[i] = c;
          const uint32_t at = (vec % T) * 8 + vec / T;  // its byte
          const uint32_t bit = 1u << (c % E + 8 * (at & 3));
          first[i] = !(atomicOr(reinterpret_cast<uint32_t*>(named) + (at >> 2), bit) & bit);
          xe[i] = load_logit<DT>(row, id[i]);
        }
      }
    }
    __syncthreads();
    if (tid < 64) {
      double t[kEntries], top = 0.0, logd = 0.0, d = 1.0;
      const bool logits = a.kind == CE_TEACHER_LOGITS;
      if (logits) {
        float largest_t = -INFINITY;
#pragma unroll
        for (int i = 0; i < kEntries; ++i) largest_t = fmaxf(largest_t, i * 64 + (int)lane < L ? tv[i] : -INFINITY);
        top = (double)wave_largest(largest_t) * a.inv_t;
      }
#pragma unroll
      for (int i = 0; i < kEntries; ++i) {
        t[i] = i * 64 + (int)lane < L ? (logits ? (double)tv[i] * a.inv_t : (double)tv[i]) - top : -(double)INFINITY;
        p[i] = i * 64 < L ? exp2_64(t[i] * kLog2eD) : 0.0;
        mass += p[i];
      }
      mass = wave_sum64(mass);
      if (logits) {
        d = mass;
        logd = log2_64(d) * kLn2d;
        mass = d == d && d > 0.0 ? 1.0 : __builtin_nan("");
      }
#pragma unroll
      for (int i = 0; i < kEntries; ++i) {
        p[i] /= d;
        plogp += p[i] == 0.0 ? 0.0 : p[i] * (t[i] - logd);
      }
      plogp = wave_sum64(plogp);
      bad = __any(bad);
    }

    const bool tells = k == (GRAD ? 0 : C - 1);  // brings the row's loss together
    if (SPLIT && tells && tid < 64) {
#pragma unroll
      for (int i = 0; i < kEntries; ++i) {  // (bad columns: the row is NaN whichever chunk they are taken for)
        const uint32_t c = (uint32_t)id[i] / (uint32_t)a.chunk_cols;
        kept_chunk[i * 64 + lane] = (uint8_t)(c < C ? c : 0u);
      }
    }
    float grad[kEntries];  // of the named columns here

    // ---- the unnamed columns: maximum and sum
    finish_chunk<DT, T, P, true>(row + (size_t)lo * EB, cols, v);
    float m = -INFINITY;
    const uint64_t flags = reinterpret_cast<const uint64_t*>(named)[tid];
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const uint32_t b = (uint32_t)(flags >> (8 * j)) & 0xffu;
      if (b) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (!(b >> e & 1u)) continue;
          if constexpr (DT == CE_BF16)
            v[j][e / 2] = e & 1 ? (v[j][e / 2] & 0xffffu) | 0xff800000u : (v[j][e / 2] & 0xffff0000u) | 0xff80u;
          else
            v[j][e] = 0xff800000u;
        }
      }
      m = largest<DT>(v[j], m);
    }
    m = wave_largest(m);
    if (lane == 0) sh_max[tid >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) m = fmaxf(m, sh_max[i]);
    const bool shifted = fabsf(m * a.kb) > kNear && fabsf(m) < INFINITY;
    if (shifted) subtract<DT, P>(v, m);
    const float from = shifted || m == -INFINITY ? 0.f : m * a.kb;
    float grow = 1.f;
    if (tid < 64 && m != -INFINITY) {  // from `from` to the exact m kb, or to the power of two
      const float d = SPLIT ? (float)above(m, m, power_of(m, a.kb64), a.kb64) : 0.f;
      grow = exp2_hw(shifted ? d : d - __builtin_fmaf(m, a.kb, -from));
    }
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      relaunch(v[j]);
      float f[E];
      unpack_vec<DT>(v[j], f);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        s0 += exp2_hw(__builtin_fmaf(f[e], a.kb, -from));
        s1 += exp2_hw(__builtin_fmaf(f[e + 1], a.kb, -from));
      }
    }
    s0 = wave_sum(s0 + s1);
    if (lane == 0) sh_sum[tid >> 6] = s0;
    __syncthreads();

    double loss = 0.0, power = 0.0;
    // ---- wave 0: the named columns here, then the row over its chunks
    if (tid < 64) {
      s0 = sh_sum[0];
#pragma unroll
      for (int i = 1; i < W; ++i) s0 += sh_sum[i];
      s0 *= grow;
      double e[kEntries], sum = 0.0, cross = 0.0;
      bool odd = false;  // NaN or +inf, which have no sum
      float ref = m;
#pragma unroll
      for (int i = 0; i < kEntries; ++i) {
        odd |= here[i] && !(xe[i] < INFINITY);
        ref = fmaxf(ref, here[i] ? xe[i] : -INFINITY);
      }
      ref = wave_largest(ref);
      const double n_ref = SPLIT ? power_of(ref, a.kb64) : INFINITY;  // (one chunk's exponents are differences from M)
#pragma unroll
      for (int i = 0; i < kEntries; ++i) {
        const bool some = here[i] && xe[i] != -INFINITY;
        const double z = some ? above(xe[i], ref, n_ref, a.kb64) : -(double)INFINITY;
        e[i] = __any(some) ? exp2_64(z) : 0.0;
        sum += first[i] ? e[i] : 0.0;
        if (here[i] && p[i] != 0.0) cross += p[i] * z;
      }
      const bool twice = [&] {
        bool again = false;
#pragma unroll
        for (int i = 0; i < kEntries; ++i) again |= here[i] && !first[i];
        return __any(again);
      }();
      sum = wave_sum64(sum);
      cross = wave_sum64(cross);
      if (__any(odd)) sum = __builtin_nan("");
      // lane c: what chunk c tells
      bool ok = true;
      uint32_t w[kWords];
      w[kMax] = __float_as_uint(m);
      w[kRest] = __float_as_uint(s0);
      w[kRef] = __float_as_uint(ref);
      put64(w + kSum, sum);
      put64(w + kCross, cross);
      w[kEmpty] = 0u;
      const auto keep = [&] {
#pragma unroll
        for (int i = 0; i < kEntries; ++i) {
          kept_p[i * 64 + lane] = p[i];
          kept_e[i * 64 + lane] = e[i];
          kept_col[i * 64 + lane] = col[i];
        }
      };
      if (GRAD && !SPLIT) keep();
      if (SPLIT) {
        unsigned long long* const slots = a.slots + (size_t)r * C * kWords;
        if (lane < kWords && !withheld(ws, r, (int)k)) {
          uint32_t mine = w[0];
#pragma unroll
          for (int q = 1; q < kWords; ++q) mine = (int)lane == q ? w[q] : mine;
          put_word(slots + k * kWords + lane, ws.tag, mine);
        }
        if (!GRAD && k != C - 1) return;
        keep();  // the last chunk brings the row's loss together; no other needs it
        uint32_t spins = 0;
        for (uint32_t i = lane; i < C * kWords; i += 64) {
          uint32_t got = 0x7fc00000u;
          ok &= await_word(slots + i, ws.tag, peek_word(slots + i), spins, &got);
          words[i] = got;
        }
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
#pragma unroll
        for (int q = 0; q < kWords; ++q) w[q] = words[(lane < C ? lane : 0u) * kWords + q];
        ok = __all(ok);
      }
      ok = ok && ws.ok;
      if (!ok && lane == 0) atomicOr(&a.hdr->status, ws.ok ? 1u : 2u);
      // the unnamed columns' sum relative to their largest, U, so that it is 0 only where all of them are masked; all of
      // it relative to the row's largest logit, M
      float M = ref, U = m;
      double rest = (double)s0, down = ((double)U - (double)M) * a.kb64, n_M = 0.0, n_U = 0.0, all = sum;
      int up_named = 0;
      if (SPLIT) {
        const bool has = lane < C;
        const float w_max = __uint_as_float(w[kMax]), w_ref = __uint_as_float(w[kRef]);
        M = wave_largest(has ? w_ref : -INFINITY);
        U = wave_largest(has ? w_max : -INFINITY);
        n_M = power_of(M, a.kb64);
        n_U = power_of(U, a.kb64);
        down = n_U - n_M;
        rest = wave_sum64(has ? ldexp((double)__uint_as_float(w[kRest]), steps(power_of(w_max, a.kb64) - n_U)) : 0.0);
        up_named = steps(power_of(w_ref, a.kb64) - n_M);
        all = wave_sum64(has ? ldexp(get64(w + kSum), up_named) : 0.0);
      }
      // their sum and its logarithm are made of the same three factors: of `rest`, 2^whole, and of an FP32 exponential
      down = U == -INFINITY ? 0.0 : fmax(down, -1e30);
      const double whole = rint(down), part = (double)exp2_hw((float)(down - whole));
      const double over = rest * ldexp(part, steps(whole));
      all += over;
      // what the teacher leaves, to the unnamed columns; nothing where none of them can take it: all masked, also by
      // values such as -1e9, next to which their share is 0 in 64 bits
      double left = 0.0;
      if (a.kind == CE_TEACHER_LOGPROBS && over != 0.0) left = fmax(0.0, 1.0 - mass);
      const double S = mass + left;
      // four logarithms at once: of the sum, of what is left, of the unnamed columns' sum's factors
      const double logs = log2_64(lane == 0 ? all : lane == 1 ? left : lane == 2 ? rest : part);
      const double log_all = lane64(logs, 0), log_rest = lane64(logs, 2);
      // the loss but for the named columns' exponents
      loss = plogp + mass * log_all * kLn2d;
      if (left != 0.0) loss += left * (lane64(logs, 1) - (log_rest + (whole + lane64(logs, 3)) - log_all)) * kLn2d;
      if constexpr (!SPLIT) loss -= cross * kLn2d;
      double s = (double)up * a.t;
      if (a.reduce == CE_REDUCE_MEAN) s /= (double)count;
      if (bad || !ok) s = loss = __builtin_nan("");
      if (!SPLIT && lane == 0) row_loss((float)(loss * a.t * a.t));
      power = n_M;
      if constexpr (GRAD) {
        // of an unnamed column: q_v S - left q_v / q_o = (q_o S - left) 2^(z_v - log2 of their sum)
        const double near_u = SPLIT ? log_rest - above(U, U, n_U, a.kb64) : log_rest;
        const double c = rest == 0.0 ? 0.0 : (double)a.kb * ((double)U - (shifted ? (double)m : 0.0)) + near_u;
        const double c_lo = fabsf((float)c) < INFINITY ? c - (double)(float)c : 0.0;  // 2^-c_lo, a few 2^-14 at most, goes to the factor
        if (lane == 0) {
          bc[0] = (float)c;
          bc[1] = (float)(s * (over / all * S - left) * fma(-kLn2d, c_lo, 1.0));
        }
        // the named columns' gradients; entries of the same column add up, in order
        const int up_own = __builtin_amdgcn_readlane(up_named, (int)k);
#pragma unroll
        for (int i = 0; i < kEntries; ++i) {
          const uint32_t c = kept_col[i * 64 + lane];
          double P_i = kept_p[i * 64 + lane];
          if (twice) {
            P_i = 0.0;
            for (int q = 0; q < L; ++q) P_i += kept_col[q] == c ? kept_p[q] : 0.0;
          }
          grad[i] = (float)(s * (ldexp(kept_e[i * 64 + lane], up_own) / all * S - P_i));
        }
      }
    }
    // of p (z - n_M), with the power of each entry's chunk; the other waves write their part of the gradient meanwhile
    const auto tell_loss = [&] {
      const bool has = lane < C;
      double cross = has ? get64(words + lane * kWords + kCross) : 0.0;
#pragma unroll
      for (int i = 0; i < kEntries; ++i) {
        const double p_i = kept_p[i * 64 + lane];
        const float of = __uint_as_float(words[kept_chunk[i * 64 + lane] * kWords + kRef]);
        if (p_i != 0.0) cross += p_i * (power_of(of, a.kb64) - power);
      }
      loss = (loss - wave_sum64(cross) * kLn2d) * (a.t * a.t);
      if (lane == 0) row_loss((float)loss);
    };
    if constexpr (SPLIT && !GRAD) {
      if (tid < 64) tell_loss();
    }
    if constexpr (GRAD) {
      __syncthreads();
      const float c = bc[0], f_un = bc[1];
      if (SPLIT && tells && tid < 64) tell_loss();
      store_chunk<DT, T, P>(out + (size_t)lo * EB, cols, v, [&](const u32x4v& x) {
        float f[E];
        unpack_vec<DT>(x, f);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = exp2_hw(__builtin_fmaf(f[e], a.kb, -c)) * f_un;
        return pack_vec<DT>(f);
      });
      __syncthreads();
      if (tid < 64) {  // over the zeros that were written for the named columns
#pragma unroll
        for (int i = 0; i < kEntries; ++i) {
          const uint32_t c = kept_col[i * 64 + lane];
          if (c != ~0u) store_logit<DT>(out, (int64_t)lo + c, grad[i]);
        }
      }
    }
  }
  if (ends) finish_distill<T>(a, ws.tag, ws.ok);
}

// Rows that have an entry: every row's gradient is over their number.  2048 rows: 2.4 us and more by itself, mostly the
// launch; 1 to 2 of a call.
__global__ __launch_bounds__(1024) void k_distill_count(const int32_t* len, int64_t N, int32_t K, int32_t* n) {
  __shared__ int part[16];
  int c = 0;
  for (int64_t r = threadIdx.x; r < N; r += 1024) c += len ? len[r] > 0 : K > 0;
  c = wave_count64(c);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = c;
  __syncthreads();
  if (threadIdx.x == 0) {
    c = 0;
    for (int i = 0; i < 16; ++i) c += part[i];
    *n = c;
  }
}

template <int DT, int T, int P, bool GRAD>
void launch_distill_chunks(const DistillArgs& a, dim3 grid, hipStream_t stream) {
  if constexpr (P == 8) {  // (a split row's chunks have more than 1365 vectors, and the smaller shapes hold 1024)
    if (a.chunks > 1) {
      hipLaunchKernelGGL((k_distill<DT, T, P, GRAD, true>), grid, dim3(T), 0, stream, a);
      return;
    }
  }
  hipLaunchKernelGGL((k_distill<DT, T, P, GRAD, false>), grid, dim3(T), 0, stream, a);
}
template <int DT, int T, int P>
void launch_distill_shape(const DistillArgs& a, dim3 grid, hipStream_t stream) {
  if (a.out) launch_distill_chunks<DT, T, P, true>(a, grid, stream);
  else launch_distill_chunks<DT, T, P, false>(a, grid, stream);
}
template <int DT>
void launch_distill_dt(const DistillArgs& a, FusedShape s, dim3 grid, hipStream_t stream) {
  if (s.threads == 512) launch_distill_shape<DT, 512, 8>(a, grid, stream);
  else if (s.vecs == 8) launch_distill_shape<DT, 256, 8>(a, grid, stream);
  else if (s.vecs == 4) launch_distill_shape<DT, 256, 4>(a, grid, stream);
  else if (s.vecs == 2) launch_distill_shape<DT, 256, 2>(a, grid, stream);
  else launch_distill_shape<DT, 256, 1>(a, grid, stream);
}

int64_t vec_cols(int32_t dtype) { return dtype == CE_BF16 ? 8 : 4; }

}  // namespace

int64_t distill_max_cols(int32_t dtype) { return (int64_t)4096 * vec_cols(dtype) * kMaxChunks; }

void distill_plan(int64_t V, int32_t dtype, int64_t* chunks, int64_t* chunk_cols) {
  const int64_t E = vec_cols(dtype), vecs = (V + E - 1) / E;
  int64_t n = fused_auto_chunks(dtype, V);
  while ((vecs + n - 1) / n > 4096) ++n;  // that plan leaves the columns around the whole vectors to other lanes
  *chunk_cols = (vecs + n - 1) / n * E;
  *chunks = (V + *chunk_cols - 1) / *chunk_cols;
}

size_t distill_workspace(int64_t N, int64_t V, int32_t dtype) {
  int64_t chunks, cols;
  distill_plan(V, dtype, &chunks, &cols);
  return chunks > 1 ? chunk_words_at(N) + (size_t)N * chunks * kWords * 8 : row_words_at(N) + (size_t)N * 8;
}

hipError_t launch_distill(DistillArgs a, void* ws, int32_t* n_valid, hipStream_t stream, hipEvent_t ev0,
                          hipEvent_t ev1) {
  hipError_t e = hipSuccess;
  WsHeader* const hdr = static_cast<WsHeader*>(ws);
  // n is the number of rows without lengths; with them it is counted first
  if (n_valid || (a.reduce == CE_REDUCE_MEAN && (a.len || a.N == 0))) {
    int32_t* const n = n_valid ? n_valid : &hdr->n_valid;
    hipLaunchKernelGGL(k_distill_count, dim3(1), dim3(1024), 0, stream, a.len, a.N, a.K, n);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    a.n = n;
  }
  if (a.N == 0)  // the mean of no rows is 0/0
    return a.reduce == CE_REDUCE_NONE ? hipSuccess
                                      : launch_mean(nullptr, 0, a.reduce == CE_REDUCE_MEAN ? a.n : nullptr, a.loss, stream);
  if (ev0 && (e = hipEventRecord(ev0, stream)) != hipSuccess) return e;
  if (a.chunks > 1 || a.reduce != CE_REDUCE_NONE) {
    a.hdr = hdr;
    a.row_words = reinterpret_cast<unsigned long long*>(static_cast<char*>(ws) + row_words_at(a.N));
    a.slots = reinterpret_cast<unsigned long long*>(static_cast<char*>(ws) + chunk_words_at(a.N));
    a.ws_bytes = distill_workspace(a.N, a.V, a.dtype);
  }
  const FusedShape shape = fused_shape_for(a.chunk_cols / vec_cols(a.dtype));
  if (a.chunks > 1 && shape.vecs != 8) return hipErrorInvalidConfiguration;
  const int64_t rows = kMaxGridItems / a.chunks;  // a launch
  for (a.row0 = 0; a.row0 < a.N; a.row0 += rows) {
    const int64_t n = a.N - a.row0 < rows ? a.N - a.row0 : rows;
    const dim3 grid((uint32_t)(n * a.chunks));
    if (a.dtype == CE_BF16) launch_distill_dt<CE_BF16>(a, shape, grid, stream);
    else launch_distill_dt<CE_F32>(a, shape, grid, stream);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (ev1) e = hipEventRecord(ev1, stream);
  return e;
}

}  // namespace vce
