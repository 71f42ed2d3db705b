// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out_n = scale W[id_n]
//   dW[v] (+)= scale * sum over { n : id_n = v } of dout_n
//
// Lookup: one read of the rows named and one write of the output.
//
// Gradient: every row of dout is read once and every row of dW that a token
// names is written once (read once too when it is added to).  Few tokens take one
// launch: each token's workgroups look through all ids and, if its own has not
// come before, add up the rows of that id.  With more tokens, to make the sum's
// order fixed and its writes few, they are sorted by id first, ties by position (a
// stable sort of N small keys, little beside the N rows of D values):
//   up to kRankMax tokens whose (id, position) pair fits 32 bits: one launch in
//     which each token's place is the count of smaller pairs (N^2 compares of LDS
//     words, N^2 / 16384 cycles of the whole chip; 8192 tokens added to 128000 x 1024:
//     35.0 us, 39.0 by the radix sort, but 16384 tokens 58.5 against 51.5);
//   more: a stable radix sort, 9 bits at most a pass, in one launch a pass up to
//     kOneMax tokens (every workgroup counts all keys) and three beyond.
// The sorted list is then cut into tiles of equally many tokens, so a token that
// makes up a large share of the batch costs no more than the others.  A
// workgroup adds up the runs of equal ids in its tile in FP32 and writes them to
// dW.  A run of at most a tile's length that crosses a boundary belongs whole to
// the tile where it starts; a longer one leaves one partial sum per tile, and a
// last launch adds those in tile order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ce_internal.h"
#include "ce_vec.h"

namespace vce {
namespace {

constexpr int kT = 256;
constexpr int64_t kMaxBlocks = (int64_t)1 << 23;  // a launch holds below 2^32 work-items

__host__ __device__ __forceinline__ int64_t min64(int64_t a, int64_t b) { return a < b ? a : b; }
__host__ __device__ __forceinline__ int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Lanes that share one row: the smallest power of two that covers its groups, at most a workgroup.
int lanes_log2(int64_t groups) {
  int l = 0;
  while (l < 8 && ((int64_t)1 << l) < groups) ++l;
  return l;
}

template <int DT>
__global__ __launch_bounds__(kT) void k_embed(EmbedArgs a, int lanes_shift) {
  constexpr int EB = VecT<DT>::EB;
  const int lanes = 1 << lanes_shift;
  const int lane = (int)threadIdx.x & (lanes - 1);
  const int64_t per = kT >> lanes_shift;
  const uint32_t D = (uint32_t)a.D;
  for (int64_t n = (int64_t)blockIdx.x * per + ((int)threadIdx.x >> lanes_shift); n < a.N;
       n += (int64_t)gridDim.x * per) {
    const int64_t id = a.ids[n * a.id_stride];
    const uint64_t v = (uint64_t)id - (uint64_t)a.vocab_start;
    char* out = a.out + n * a.out_ld * EB;
    if (v < (uint64_t)a.V) {
      const char* w = a.w + (int64_t)v * a.w_ld * EB;
      if constexpr (DT == CE_F32) {
        // quads, side by side across the lanes: with eight columns a lane every store leaves half of each line to the
        // next one (12385 x 4096: 65 against 47 us)
        const uint32_t whole = D & ~3u, step = (uint32_t)lanes * 4;
        for (uint32_t at = (uint32_t)lane * 4; at < D; at += 2 * step) {
          u32x4v q[2];
          const uint32_t j[2] = {at, at + step};
          if (whole) {
#pragma unroll
            for (int h = 0; h < 2; ++h) q[h] = fetch_quad<DT>(w, j[h] < whole ? j[h] : 0);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (j[h] >= D) continue;
            if (j[h] >= whole) q[h] = partial_quad<DT>(w, j[h], D);
            float f[4];
            quad_to_f32<DT>(q[h], f);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] *= a.scale;
            store_quad<true>(reinterpret_cast<float*>(out), j[h], D, f);
          }
        }
        continue;
      }
      for (uint32_t j = (uint32_t)lane * kG; j < D; j += (uint32_t)lanes * kG) {
        float f[kG];
        load_f32<DT>(w, j, D, f);
#pragma unroll
        for (int e = 0; e < kG; ++e) f[e] *= a.scale;
        store_group<DT, true>(out, j, D, f32_to_raw<DT>(f));
      }
    } else {
      // another shard's id adds nothing here; an id outside the vocabulary is a caller's error
      const float fill = (uint64_t)id < (uint64_t)a.vocab_total ? 0.f : __builtin_nanf("");
      float f[kG];
#pragma unroll
      for (int e = 0; e < kG; ++e) f[e] = fill;
      for (uint32_t j = (uint32_t)lane * kG; j < D; j += (uint32_t)lanes * kG)
        store_group<DT, true>(out, j, D, f32_to_raw<DT>(f));
    }
  }
}

// ---- sorting -------------------------------------------------------------

// The sort key of token n: its row of this shard, or V for a token without a gradient here (the
// padding id, another shard's, or no id at all); those come last.
__device__ __forceinline__ uint32_t key_of(const EmbedGradArgs& a, int64_t id) {
  const uint64_t v = (uint64_t)id - (uint64_t)a.vocab_start;
  return v < (uint64_t)a.V && (a.padding_idx < 0 || id != a.padding_idx) ? (uint32_t)v : (uint32_t)a.V;
}

__device__ __forceinline__ uint32_t token_key(const EmbedGradArgs& a, int64_t n) {
  return key_of(a, a.ids[n * a.id_stride]);
}

int bits_of(int64_t v) {  // of the values 0 .. v
  int b = 1;
  while (b < 63 && ((int64_t)1 << b) <= v) ++b;
  return b;
}

constexpr int64_t kRankMax = 8192;
constexpr int kRankT = 1024;
constexpr int kRankTokens = 32;                    // tokens a workgroup places
constexpr int kRankOwn = 4;                        // of them, tokens a thread counts for
constexpr int kRankSlices = kRankT / (kRankTokens / kRankOwn);  // of the pairs, one a thread

// Place of every token among the pairs (key, position): the count of smaller
// ones.  A workgroup holds all pairs in LDS; 8 threads share a slice of them,
// 4 tokens each, so a 16-byte LDS read serves 16 compares.
__global__ __launch_bounds__(kRankT) void k_rank(EmbedGradArgs a, int pos_bits, uint32_t* skey, uint32_t* sidx) {
  __shared__ __align__(16) uint32_t pair[kRankMax];
  __shared__ uint32_t part[kRankSlices / 8][kRankTokens];
  const uint32_t n = (uint32_t)a.N;
  const uint32_t steps = (n + kRankSlices * 4 - 1) / (kRankSlices * 4);  // 16-byte words per slice
  constexpr int LOADS = (int)(kRankMax / kRankT);
  int64_t id[LOADS];
#pragma unroll
  for (int k = 0; k < LOADS; ++k) {  // without a branch, so that all are in flight
    const uint32_t i = k * kRankT + threadIdx.x;
    id[k] = a.ids[(int64_t)(i < n ? i : n - 1) * a.id_stride];
  }
#pragma unroll
  for (int k = 0; k < LOADS; ++k) {
    const uint32_t i = k * kRankT + threadIdx.x;
    pair[i] = i < n ? (key_of(a, id[k]) << pos_bits) | i : 0xffffffffu;
  }
  __syncthreads();
  constexpr int OWNERS = kRankTokens / kRankOwn;
  const uint32_t own = threadIdx.x % OWNERS, slice = threadIdx.x / OWNERS;
  const uint32_t base = blockIdx.x * kRankTokens;
  uint32_t mine[kRankOwn], less[kRankOwn];
#pragma unroll
  for (int k = 0; k < kRankOwn; ++k) {
    const uint32_t me = base + k * OWNERS + own;
    mine[k] = me < n ? pair[me] : 0u;
    less[k] = 0;
  }
  const u32x4v* p = reinterpret_cast<const u32x4v*>(pair) + slice;
#pragma unroll 4
  for (uint32_t i = 0; i < steps; ++i) {
    const u32x4v q = p[i * kRankSlices];  // a wave's 8 slices read 128 bytes side by side
#pragma unroll
    for (int k = 0; k < kRankOwn; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) less[k] += q[e] < mine[k] ? 1u : 0u;
  }
  // a wave holds 8 slices: add them across its lanes, then the waves' sums in LDS
#pragma unroll
  for (int k = 0; k < kRankOwn; ++k) {
#pragma unroll
    for (int m = OWNERS; m < 64; m <<= 1) less[k] += __shfl_xor(less[k], m, 64);
    if ((threadIdx.x & 63) < OWNERS) part[threadIdx.x >> 6][k * OWNERS + own] = less[k];
  }
  __syncthreads();
  const uint32_t me = base + threadIdx.x;
  if (threadIdx.x < kRankTokens && me < n) {
    uint32_t at = 0;
#pragma unroll
    for (int k = 0; k < kRankSlices / 8; ++k) at += part[k][threadIdx.x];
    skey[at] = pair[me] >> pos_bits;
    sidx[at] = pair[me] & ((1u << pos_bits) - 1u);
  }
}

constexpr int kSortTile = 2048;
constexpr int kMaxDigit = 9;
constexpr int kWaves = kT / 64;

struct SortPass {
  const uint32_t* key_in;  // NULL: the first pass reads the ids
  const uint32_t* idx_in;
  uint32_t* key_out;
  uint32_t* idx_out;
  uint32_t* hist;          // [bins][tiles]
  int64_t tiles;
  int shift, bits;
};

__global__ __launch_bounds__(kT) void k_sort_count(EmbedGradArgs a, SortPass s) {
  __shared__ uint32_t h[1 << kMaxDigit];
  const int bins = 1 << s.bits;
  for (int i = (int)threadIdx.x; i < bins; i += kT) h[i] = 0;
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * kSortTile, hi = min64(lo + kSortTile, a.N);
  uint32_t key[kSortTile / kT];
#pragma unroll
  for (int k = 0; k < kSortTile / kT; ++k) {
    const int64_t n = min64(lo + k * kT + (int)threadIdx.x, hi - 1);
    key[k] = s.key_in ? s.key_in[n] : token_key(a, n);
  }
#pragma unroll
  for (int k = 0; k < kSortTile / kT; ++k)
    if (lo + k * kT + (int)threadIdx.x < hi) atomicAdd(&h[(key[k] >> s.shift) & (bins - 1)], 1u);
  __syncthreads();
  for (int i = (int)threadIdx.x; i < bins; i += kT) s.hist[(int64_t)i * s.tiles + blockIdx.x] = h[i];
}

// Exclusive sums over n counts, in place, by one workgroup.
__global__ __launch_bounds__(1024) void k_sort_scan(uint32_t* h, int64_t n) {
  __shared__ uint32_t wave_total[16];
  uint32_t base = 0;
  const int lane = (int)threadIdx.x & 63, w = (int)threadIdx.x >> 6;
  for (int64_t at = 0; at < n; at += 4096) {
    const int64_t i = at + (int64_t)threadIdx.x * 4;
    uint32_t v[4], sum = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = i + k < n ? h[i + k] : 0u;
      sum += v[k];
    }
    uint32_t scan = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t o = __shfl_up(scan, d, 64);
      if (lane >= d) scan += o;
    }
    __syncthreads();
    if (lane == 63) wave_total[w] = scan;
    __syncthreads();
    uint32_t before = base, all = 0;
    for (int k = 0; k < 16; ++k) {
      if (k < w) before += wave_total[k];
      all += wave_total[k];
    }
    uint32_t run = before + scan - sum;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (i + k < n) h[i + k] = run;
      run += v[k];
    }
    base += all;
  }
}

// Moves a tile's tokens to their places.  Wave w takes the w-th quarter of the
// tile in order; a token's place is its bin's start for this tile (from the
// scan), plus the tokens of that bin in earlier waves, plus those earlier in
// its own wave: equal keys keep their order.
__global__ __launch_bounds__(kT) void k_sort_move(EmbedGradArgs a, SortPass s) {
  __shared__ uint32_t next[kWaves][1 << kMaxDigit];
  const int bins = 1 << s.bits;
  for (int i = (int)threadIdx.x; i < kWaves * bins; i += kT) next[i / bins][i % bins] = 0;
  __syncthreads();
  constexpr int QUARTER = kSortTile / kWaves, ROUNDS = QUARTER / 64;
  const int lane = (int)threadIdx.x & 63, w = (int)threadIdx.x >> 6;
  const int64_t lo = (int64_t)blockIdx.x * kSortTile + w * QUARTER;
  uint32_t key[ROUNDS], idx[ROUNDS];
#pragma unroll
  for (int k = 0; k < ROUNDS; ++k) {
    const int64_t n = min64(lo + k * 64 + lane, a.N - 1);
    key[k] = s.key_in ? s.key_in[n] : token_key(a, n);
    idx[k] = s.idx_in ? s.idx_in[n] : (uint32_t)n;
  }
#pragma unroll
  for (int k = 0; k < ROUNDS; ++k)
    if (lo + k * 64 + lane < a.N) atomicAdd(&next[w][(key[k] >> s.shift) & (bins - 1)], 1u);
  __syncthreads();
  for (int i = (int)threadIdx.x; i < bins; i += kT) {
    uint32_t at = s.hist[(int64_t)i * s.tiles + blockIdx.x];
    for (int k = 0; k < kWaves; ++k) {
      const uint32_t c = next[k][i];
      next[k][i] = at;
      at += c;
    }
  }
  __syncthreads();
  // rounds are kept in step by barriers: a wave reads its bins' next places, then their last lanes move them on
#pragma unroll
  for (int k = 0; k < ROUNDS; ++k) {
    const bool live = lo + k * 64 + lane < a.N;
    const uint32_t bin = (key[k] >> s.shift) & (bins - 1);
    uint64_t same = __ballot(live);
    for (int b = 0; b < s.bits; ++b) {
      const bool bit = (bin >> b) & 1u;
      const uint64_t set = __ballot(bit);
      same &= bit ? set : ~set;
    }
    const uint32_t before = (uint32_t)__popcll(same & (((uint64_t)1 << lane) - 1));
    const uint32_t first = live ? next[w][bin] : 0u;
    __syncthreads();
    if (live) {
      const uint32_t to = first + before;
      s.key_out[to] = key[k];
      s.idx_out[to] = idx[k];
      if (before + 1 == (uint32_t)__popcll(same)) next[w][bin] = to + 1;
    }
    __syncthreads();
  }
}

// A pass over up to kOneMax tokens in one launch: every workgroup counts all
// keys itself, those before its tile apart, so none waits for another.  Its tile
// is one token per thread.
constexpr int kOneT = 1024;
constexpr int64_t kOneMax = 65536;
__global__ __launch_bounds__(kOneT) void k_sort_one(EmbedGradArgs a, SortPass s) {
  constexpr int BINS = 1 << kMaxDigit, W = kOneT / 64;
  // counts before this tile and from it on, in 8 copies side by side: lanes of one bin do not all meet in one word
  constexpr int C = 8;
  __shared__ uint32_t before[BINS * C], rest[BINS * C], next[W][BINS], wave_total[BINS / 64];
  const uint32_t n = (uint32_t)a.N, mask = (1u << s.bits) - 1u;
  const int lane = (int)threadIdx.x & 63, w = (int)threadIdx.x >> 6;
  for (int i = (int)threadIdx.x; i < BINS * C; i += kOneT) before[i] = rest[i] = 0;
  for (int i = (int)threadIdx.x; i < W * BINS; i += kOneT) next[0][i] = 0;
  __syncthreads();
  uint32_t mine = 0;
  const uint32_t tiles = (n + kOneT - 1) / kOneT;
  for (uint32_t t0 = 0; t0 < tiles; t0 += 8) {
    uint32_t key[8];
    if (s.key_in) {
#pragma unroll
      for (uint32_t k = 0; k < 8; ++k) {
        const uint32_t i = (t0 + k) * kOneT + threadIdx.x;
        key[k] = s.key_in[i < n ? i : n - 1];
      }
    } else {
      int64_t id[8];
#pragma unroll
      for (uint32_t k = 0; k < 8; ++k) {
        const uint32_t i = (t0 + k) * kOneT + threadIdx.x;
        id[k] = a.ids[(int64_t)(i < n ? i : n - 1) * a.id_stride];
      }
#pragma unroll
      for (uint32_t k = 0; k < 8; ++k) key[k] = key_of(a, id[k]);
    }
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {
      const uint32_t t = t0 + k;
      if (t == blockIdx.x) mine = key[k];
      if (t * kOneT + threadIdx.x < n)
        atomicAdd(&(t < blockIdx.x ? before : rest)[((key[k] >> s.shift) & mask) * C + (lane & (C - 1))], 1u);
    }
  }
  // this tile: lanes of a wave with the same bin, in order
  const uint32_t at = blockIdx.x * kOneT + threadIdx.x;
  const bool live = at < n;
  const uint32_t bin = (mine >> s.shift) & mask;
  uint64_t same = __ballot(live);
  for (int b = 0; b < s.bits; ++b) {
    const bool bit = (bin >> b) & 1u;
    const uint64_t set = __ballot(bit);
    same &= bit ? set : ~set;
  }
  const uint32_t rank = (uint32_t)__popcll(same & (((uint64_t)1 << lane) - 1));
  if (live && rank == 0) next[w][bin] = (uint32_t)__popcll(same);
  __syncthreads();
  // places: bins before this one, this bin in the tiles before, this bin in the waves before
  uint32_t scan = 0, all = 0, prior = 0;
  if (threadIdx.x < BINS) {
#pragma unroll
    for (int k = 0; k < C; ++k) {
      prior += before[threadIdx.x * C + k];
      all += rest[threadIdx.x * C + k];
    }
    all += prior;
    scan = all;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t o = __shfl_up(scan, d, 64);
      if (lane >= d) scan += o;
    }
    if (lane == 63) wave_total[w] = scan;
  }
  __syncthreads();
  if (threadIdx.x < BINS) {
    uint32_t place = scan - all + prior;
    for (int k = 0; k < w; ++k) place += wave_total[k];
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const uint32_t c = next[k][threadIdx.x];
      next[k][threadIdx.x] = place;
      place += c;
    }
  }
  __syncthreads();
  if (live) {
    const uint32_t to = next[w][bin] + rank;
    s.key_out[to] = mine;
    s.idx_out[to] = s.idx_in ? s.idx_in[at] : at;
  }
}

// ---- sums ----------------------------------------------------------------

constexpr int64_t kTileTokens = 16, kMaxTiles = 4096;

struct SumArgs {
  const uint32_t* skey;
  const uint32_t* sidx;
  float* parts;            // [2 tiles][D]: a tile's share of a long run from the tile before, of one into the next
  uint32_t* starts;        // [tiles] 1 where a long run starts, else 0
  int64_t tiles, tile;     // tokens per tile
  int64_t col_blocks;      // k_embed_sum's units across a row: a unit is a tile's tokens over 512 columns
  bool narrow;
  int lanes_shift;         // k_embed_narrow: lanes of a row
  int64_t fill_blocks;     // workgroups that write the rows no token names (0 when dW is added to)
  bool flat;               // they take dW as one array (fill_flat)
};
constexpr int kFillRows = 8;  // (32: 72 against 68 us on 20011 x 1037 FP32 tokens, 32000 rows)

// Tokens with key `key` that follow one another from position `at` on (UP) or
// from at - 1 down, at most `limit` of them.  UNI: by the lanes of a wave, 64 at a
// time; else by a search of each thread's own.
template <bool UNI, bool UP>
__device__ __forceinline__ uint32_t run_from(const SumArgs& s, uint32_t N, uint32_t at, uint32_t key, uint32_t limit) {
  const uint32_t there = UP ? N - at : at, most = there < limit ? there : limit;
  if constexpr (UNI) {
    const uint32_t lane = threadIdx.x & 63;
    for (uint32_t base = 0; base < most; base += 64) {
      const uint32_t d = base + lane;
      const bool in = d < most && s.skey[UP ? at + d : at - 1 - d] == key;
      const uint64_t all = __ballot(in);
      if (all != ~(uint64_t)0) return base + (uint32_t)__builtin_ctzll(~all);
    }
    return most;
  } else {
    uint32_t lo = 0, hi = most;  // sorted: the matches come first
    while (lo < hi) {
      const uint32_t mid = (lo + hi) >> 1;
      if (s.skey[UP ? at + mid : at - 1 - mid] == key) lo = mid + 1; else hi = mid;
    }
    return lo;
  }
}
// Whether the run across boundary `b` (0 < b < N, both sides of one key) is longer than a tile; *ahead: its tokens
// from b on, where it is not.
template <bool UNI>
__device__ __forceinline__ bool long_run(const SumArgs& s, uint32_t N, uint32_t b, uint32_t key, uint32_t* ahead) {
  const uint32_t tile = (uint32_t)s.tile;
  const uint32_t back = run_from<UNI, false>(s, N, b, key, tile);
  *ahead = run_from<UNI, true>(s, N, b, key, tile);
  return back + *ahead > tile;
}

// Where a tile's work begins and ends: [i0, i1) without the share of a run from the tile before that is short (it is
// that tile's) and with the whole of a short one that it starts; and whether its first and last runs are shares of long
// ones.  Tiles of 16 tokens, with 16 before and after: one load of a wave (5000 x 256 BF16 tokens: 25 against 27 us).
struct TileRuns {
  uint32_t i0, i1;
  bool from_before, goes_on, one_run;
};
__device__ __forceinline__ TileRuns tile_runs(const SumArgs& s, uint32_t N, uint32_t none, int64_t t) {
  TileRuns r;
  r.i0 = (uint32_t)(t * s.tile);
  r.i1 = (uint32_t)min64((int64_t)r.i0 + s.tile, N);
  r.from_before = r.goes_on = false;
  constexpr uint32_t kTT = (uint32_t)kTileTokens;
  static_assert(kTT == 16, "windows of three tiles in a wave's lanes, in 16-bit fields");
  if (s.tile == kTileTokens) {
    const uint32_t len = r.i1 - r.i0;
    const int64_t at = (int64_t)r.i0 - kTT + (threadIdx.x & 63);
    const bool in = (threadIdx.x & 63) < 3 * kTT && at >= 0 && at < (int64_t)N;
    const uint32_t key = s.skey[in ? at : (int64_t)r.i0];
    const uint32_t first = (uint32_t)__builtin_amdgcn_readlane((int)key, kTT);
    const uint32_t last = (uint32_t)__builtin_amdgcn_readlane((int)key, (int)(kTT - 1 + len));
    const uint64_t eq_first = __ballot(in && key == first), eq_last = __ballot(in && key == last);
    const uint32_t back_in = (uint32_t)__popcll(eq_first & 0xffff);
    const uint32_t ahead_in = (uint32_t)__popcll((eq_first >> kTT) & 0xffff);
    const uint32_t back_out = (uint32_t)__popcll((eq_last >> len) & 0xffff);
    const uint32_t ahead_out = (uint32_t)__popcll((eq_last >> (kTT + len)) & 0xffff);
    if (back_in && first != none) {
      r.from_before = back_in + ahead_in > kTT;
      if (!r.from_before) r.i0 += ahead_in;
    }
    if (ahead_out && last != none) {
      r.goes_on = back_out + ahead_out > kTT;
      if (!r.goes_on) r.i1 += ahead_out;
    }
    r.one_run = first == last;
    return r;
  }
  const uint32_t first = s.skey[r.i0], last = s.skey[r.i1 - 1];
  const bool crosses_in = r.i0 > 0 && s.skey[r.i0 > 0 ? r.i0 - 1 : 0] == first && first != none;
  const bool crosses_out = r.i1 < N && s.skey[r.i1 < N ? r.i1 : 0] == last && last != none;
  uint32_t ahead;
  if (crosses_in) {
    r.from_before = long_run<true>(s, N, r.i0, first, &ahead);
    if (!r.from_before) r.i0 += ahead;
  }
  if (crosses_out) {
    r.goes_on = long_run<true>(s, N, r.i1, last, &ahead);
    if (!r.goes_on) r.i1 += ahead;
  }
  r.one_run = first == last;
  return r;
}

// Zeros in the rows v0 .. v0 + kFillRows - 1 of dW whose bit in `named` is not set:
// 16-byte stores from a row's first 16-byte boundary on, single columns before and
// after.  Rows that share cache lines are written with the non-temporal bit (20011
// tokens of 1037 FP32 columns, 32000 rows: 65 against 82 us), whole lines without (2000
// tokens of 4096 columns, 32000 rows: 115 against 117 us).
__device__ __forceinline__ void zero_rows(const EmbedGradArgs& a, int64_t v0, uint32_t named) {
  const uint32_t D = (uint32_t)a.D;
  const u32x4v zero = {0u, 0u, 0u, 0u};
  const bool lines = (((uintptr_t)a.dw | (uintptr_t)(a.dw_ld * 4)) & 127) == 0;
  for (int k = 0; k < kFillRows && v0 + k < a.V; ++k) {
    if ((named >> k) & 1u) continue;
    float* row = a.dw + (v0 + k) * a.dw_ld;
    uint32_t head = (uint32_t)((16 - ((uintptr_t)row & 15)) & 15) / 4;
    head = head < D ? head : D;
    const uint32_t body = (D - head) / 4;
    if (threadIdx.x < head) row[threadIdx.x] = 0.f;
    u32x4v* const p = reinterpret_cast<u32x4v*>(row + head);
    if (lines) {
      for (uint32_t j = threadIdx.x; j < body; j += kT) p[j] = zero;
    } else {
      for (uint32_t j = threadIdx.x; j < body; j += kT) __builtin_nontemporal_store(zero, p + j);
    }
    const uint32_t tail = head + body * 4 + threadIdx.x;
    if (threadIdx.x < 4 && tail < D) row[tail] = 0.f;
  }
}

// The same where dW's rows lie end to end from a 16-byte boundary on: a workgroup takes E values, whatever rows they
// belong to, a quad a thread and step.  For rows of few columns (8 rows a workgroup against 8192 values a workgroup,
// two tables in turn: 3000 tokens in 120000 x 64 columns 63 and 20 us, 30000 in 120000 x 300 93 and 69, in 120000 x 520
// 106 and 98.5, but 20011 in 32000 x 1037 65 and 85, 8192 in 32000 x 4096 131 and 134), and for any with at most 256
// tokens, then 4096 values (3 in 64703 x 4096: 187 and 163 us, 255 in 32000 x 4096 102 and 91; 257 107 and, by 8192
// values, 109).
constexpr int kFlatFew = 4096, kFlat = 8192;
constexpr int64_t kFlatCols = 512;
template <int E>
struct FillShare {
  uint32_t named[E / 32 + 2];  // a bit per row that the share touches
  uint32_t any;
};
bool end_to_end(const EmbedGradArgs& a) { return (a.dw_ld == a.D || a.V == 1) && (uintptr_t)a.dw % 16 == 0; }
// the rows of a share: the first one, and how many
template <int E>
__device__ __forceinline__ uint32_t fill_first(const EmbedGradArgs& a, int64_t block, uint32_t* count) {
  const int64_t e0 = block * E, end = min64(e0 + E, a.V * a.D) - 1;
  const uint32_t r0 = (uint32_t)(e0 / a.D);
  *count = (uint32_t)(end / a.D) - r0 + 1;
  return r0;
}
template <int E>
__device__ __forceinline__ void fill_clear(FillShare<E>& f, uint32_t rows) {
  for (uint32_t i = threadIdx.x; i < (rows + 31) / 32; i += kT) f.named[i] = 0;
  if (threadIdx.x == 0) f.any = 0;
}
template <int E>
__device__ __forceinline__ void fill_name(FillShare<E>& f, uint32_t row) {
  atomicOr(&f.named[row >> 5], 1u << (row & 31));
  f.any = 1;
}
template <int E>
__device__ __forceinline__ void zero_share(const EmbedGradArgs& a, int64_t block, uint32_t r0, const FillShare<E>& f) {
  const int64_t e0 = block * E;
  const uint32_t count = (uint32_t)min64(E, a.V * a.D - e0), D = (uint32_t)a.D;
  float* const p = a.dw + e0;
  const u32x4v zero = {0u, 0u, 0u, 0u};
  const bool any = f.any;
  const auto unnamed = [&](uint32_t row) { return ((f.named[row >> 5] >> (row & 31)) & 1u) == 0; };
  uint32_t col = (uint32_t)(e0 - (int64_t)r0 * a.D) + threadIdx.x * 4, row = col / D;
  col -= row * D;
  const uint32_t step_row = 4 * kT / D, step_col = 4 * kT - step_row * D;
#pragma unroll 4
  for (uint32_t at = threadIdx.x * 4; at < count; at += 4 * kT) {
    if (at + 4 <= count && (!any || (col + 4 <= D && unnamed(row)))) {
      *reinterpret_cast<u32x4v*>(p + at) = zero;
    } else {
      uint32_t r = row, c = col;
      for (uint32_t e = 0; e < 4 && at + e < count; ++e) {
        if (!any || unnamed(r)) p[at + e] = 0.f;
        if (++c == D) {
          c = 0;
          ++r;
        }
      }
    }
    row += step_row;
    col += step_col;
    if (col >= D) {
      col -= D;
      ++row;
    }
  }
}

// The first sorted token with a key of at least v, by a wave: 64 places a step.
__device__ __forceinline__ uint32_t lower_bound(const SumArgs& s, uint32_t N, uint32_t v) {
  uint32_t lo = 0, n = N;  // it is one of lo .. lo + n
  while (n > 0) {
    const uint32_t step = (n + 63) / 64, at = lo + ((threadIdx.x & 63) + 1) * step - 1;  // the last of each part
    const uint64_t less = __ballot(at < lo + n && s.skey[at < N ? at : N - 1] < v);
    const uint32_t parts = (uint32_t)__popcll(less);  // parts that lie wholly before it
    const uint32_t skip = parts * step < n ? parts * step : n;
    lo += skip;
    n = n - skip < step - 1 ? n - skip : step - 1;
  }
  return lo;
}
__device__ __forceinline__ void fill_flat(const EmbedGradArgs& a, const SumArgs& s, int64_t block) {
  __shared__ FillShare<kFlat> f;
  __shared__ uint32_t range[2];
  uint32_t rows;
  const uint32_t r0 = fill_first<kFlat>(a, block, &rows), N = (uint32_t)a.N;
  fill_clear(f, rows);
  if (threadIdx.x < 128) {
    const uint32_t at = lower_bound(s, N, threadIdx.x < 64 ? r0 : r0 + rows);
    if ((threadIdx.x & 63) == 0) range[threadIdx.x >> 6] = at;
  }
  __syncthreads();
  for (uint32_t n = range[0] + threadIdx.x; n < range[1]; n += kT) fill_name(f, s.skey[n] - r0);
  __syncthreads();
  zero_share(a, block, r0, f);
}

// Rows of dW that no token names: a search of the sorted keys for each, zeros where it is not found.
__device__ __forceinline__ void fill_rows(const EmbedGradArgs& a, const SumArgs& s, int64_t block) {
  __shared__ uint32_t named;
  const int64_t v0 = block * kFillRows;
  if (threadIdx.x < 64) {
    const int64_t v = v0 + (int)threadIdx.x;
    uint32_t lo = 0, hi = (uint32_t)a.N;  // the first sorted token with a key of at least v
    while (lo < hi) {
      const uint32_t mid = (lo + hi) >> 1;
      if (s.skey[mid] < (uint32_t)v) lo = mid + 1; else hi = mid;
    }
    const bool found = lo < (uint32_t)a.N && s.skey[lo] == (uint32_t)v;
    const uint64_t all = __ballot(found);
    if (threadIdx.x == 0) named = (uint32_t)all;
  }
  __syncthreads();
  zero_rows(a, v0, named);
}

// Few tokens, no sort: block (n, c) is token n's, for the 512 columns from 512 c
// on.  Every thread compares the keys of M tokens with token n's; the block of an
// id's first token adds up the rows of all of them, a quarter of the batch's
// positions per wave, and the waves' sums in order.
constexpr int64_t kDirectMax = 1024, kDirectBlocks = 4096;
template <int DT, int M>
__global__ __launch_bounds__(kT) void k_embed_direct(EmbedGradArgs a, int64_t col_blocks, int64_t sum_blocks,
                                                     int64_t blocks, bool flat) {
  constexpr int EB = VecT<DT>::EB;
  constexpr int B = 4;
  // word w M + k, bit l: whether token (w M + k) 64 + l has the block's key, so wave w has a quarter in order
  __shared__ uint64_t match[kWaves * M];
  __shared__ float part[kWaves][512];
  __shared__ uint32_t mine, named;
  const uint32_t D = (uint32_t)a.D, whole = D & ~3u, N = (uint32_t)a.N, none = (uint32_t)a.V, t = threadIdx.x;
  const uint32_t lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane((int)(t >> 6));
  int64_t id[M];
#pragma unroll
  for (int k = 0; k < M; ++k) {
    const uint32_t m = (uint32_t)(w * M + k) * 64 + lane;
    id[k] = a.ids[(int64_t)(m < N ? m : N - 1) * a.id_stride];
  }
  uint32_t key[M];
#pragma unroll
  for (int k = 0; k < M; ++k) key[k] = (uint32_t)(w * M + k) * 64 + lane < N ? key_of(a, id[k]) : none;
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    __syncthreads();  // what the last block left in LDS has been read
    if (b >= sum_blocks && flat) {
      constexpr int E = M == 1 ? kFlatFew : kFlat;
      __shared__ FillShare<E> f;
      uint32_t rows;
      const uint32_t r0 = fill_first<E>(a, b - sum_blocks, &rows);
      fill_clear(f, rows);
      __syncthreads();
#pragma unroll
      for (int k = 0; k < M; ++k)
        if (key[k] != none && key[k] - r0 < rows) fill_name(f, key[k] - r0);
      __syncthreads();
      zero_share(a, b - sum_blocks, r0, f);
      continue;
    }
    if (b >= sum_blocks) {
      const uint32_t v0 = (uint32_t)(b - sum_blocks) * kFillRows;
      if (t == 0) named = 0;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < M; ++k)
        if (key[k] != none && key[k] - v0 < (uint32_t)kFillRows) atomicOr(&named, 1u << (key[k] - v0));
      __syncthreads();
      zero_rows(a, v0, named);
      continue;
    }
    const uint32_t n = (uint32_t)b / (uint32_t)col_blocks;  // (sum_blocks is at most kDirectBlocks)
#pragma unroll
    for (int k = 0; k < M; ++k)
      if ((uint32_t)(w * M + k) * 64 + lane == n) mine = key[k];
    __syncthreads();
    const uint32_t own = mine;
#pragma unroll
    for (int k = 0; k < M; ++k) {
      const uint64_t same = __ballot(key[k] == own);
      if (lane == 0) match[w * M + k] = same;
    }
    __syncthreads();
    bool first = own != none;
#pragma unroll
    for (int k = 0; k < kWaves * M; ++k) {
      const uint32_t at = (uint32_t)k * 64;
      const uint64_t before = n >= at + 64 ? ~(uint64_t)0 : n > at ? ((uint64_t)1 << (n - at)) - 1 : 0;
      first = first && (match[k] & before) == 0;
    }
    if (!first) continue;  // (the same for the whole workgroup)
    const uint32_t c = (uint32_t)(b - n * col_blocks) * 512;
    uint32_t j[2];
    j[0] = c + lane * 4;
    j[1] = j[0] + 256;
    float* const dw = a.dw + (int64_t)own * a.dw_ld;
    float old[2] = {0.f, 0.f};  // of columns c + t and c + 256 + t, which this thread writes
    if (a.accumulate) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (c + h * 256 + t < D) old[h] = dw[c + h * 256 + t];
    }
    float acc[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[h][e] = 0.f;
    for (int k = 0; k < M; ++k) {
      const uint64_t found = match[w * M + k];
      // (scalars: the same for all lanes)
      uint64_t bits = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(found >> 32)) << 32 |
                      (uint32_t)__builtin_amdgcn_readfirstlane((int)found);
      while (bits) {
        const int count = min(B, (int)__popcll(bits));
        uint32_t at[B];
#pragma unroll
        for (int i = 0; i < B; ++i) {  // past the last one, the last one again
          at[i] = (uint32_t)((w * M + k) * 64 + __builtin_ctzll(bits));
          if (i + 1 < count) bits &= bits - 1;
        }
        bits &= bits - 1;
        u32x4v row[B][2];
        if (whole) {
#pragma unroll
          for (int i = 0; i < B; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              row[i][h] = fetch_quad<DT>(a.dout + (int64_t)at[i] * a.dout_ld * EB, j[h] < whole ? j[h] : 0);
        }
#pragma unroll
        for (int i = 0; i < B; ++i) {
          if (i < count) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (j[h] >= whole && j[h] < D)
                row[i][h] = partial_quad<DT>(a.dout + (int64_t)at[i] * a.dout_ld * EB, j[h], D);
              float f[4];
              quad_to_f32<DT>(row[i][h], f);
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[h][e] += f[e];
            }
          }
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<float4*>(&part[w][h * 256 + lane * 4]) = make_float4(acc[h][0], acc[h][1], acc[h][2], acc[h][3]);
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t q = h * 256 + t;
      if (c + q < D) {
        float v = part[0][q];
#pragma unroll
        for (int k = 1; k < kWaves; ++k) v += part[k][q];
        dw[c + q] = a.accumulate ? __builtin_fmaf(v, a.scale, old[h]) : v * a.scale;
      }
    }
  }
}

// Whether the direct kernel takes a call.  Its blocks cost 1.5 us a few thousand, where the sort's launches cost 12
// (300 x 4096: 12.6 against 21.6 us; 1000 x 1037: 14.7 and 25.7; 1000 x 4096, 8000 blocks: 31.6 and 24.8), and an id
// that takes up the batch has one block per 512 columns (1000 tokens of one id: 42 us, sorted 20; 2000: 80).
bool direct(int64_t N, int64_t D) { return N <= kDirectMax && N * ceil_div(D, 512) <= kDirectBlocks; }

template <int DT>
hipError_t launch_direct(const EmbedGradArgs& a, hipStream_t stream) {
  const int64_t col_blocks = ceil_div(a.D, 512), sum_blocks = a.N * col_blocks;
  const bool few = a.N <= kT, flat = end_to_end(a) && (few || a.D <= kFlatCols);
  const int64_t fill = flat ? ceil_div(a.V * a.D, few ? kFlatFew : kFlat) : ceil_div(a.V, kFillRows);
  const int64_t blocks = sum_blocks + (a.accumulate ? 0 : fill);
  const dim3 grid((uint32_t)min64(blocks, kMaxBlocks));
  if (few)
    hipLaunchKernelGGL((k_embed_direct<DT, 1>), grid, dim3(kT), 0, stream, a, col_blocks, sum_blocks, blocks, flat);
  else
    hipLaunchKernelGGL((k_embed_direct<DT, 4>), grid, dim3(kT), 0, stream, a, col_blocks, sum_blocks, blocks, flat);
  return hipGetLastError();
}

// The four columns from j on, in two steps so that a load waits for nothing: a row's last, partial quad (and any past
// it) is loaded as the row's last four columns, and its columns are moved to the front when they are used (what is
// behind them is never stored).  SHORT: rows of fewer than four columns.
template <int DT, bool NT, bool SHORT>
__device__ __forceinline__ u32x4v load_quad(const char* row, uint32_t j, uint32_t whole, uint32_t D) {
  if constexpr (SHORT) return partial_quad<DT>(row, j, D);
  else return fetch_quad<DT, NT>(row, j < whole ? j : D - 4);
}
template <int DT, bool SHORT>
__device__ __forceinline__ u32x4v tail_quad(u32x4v w, uint32_t j, uint32_t whole, uint32_t D) {
  if constexpr (!SHORT) {
    const uint32_t n = j < whole ? 0u : D - whole;  // columns of a partial quad
    if constexpr (DT == CE_F32) {
      w.x = n == 1 ? w.w : n == 2 ? w.z : n == 3 ? w.y : w.x;
      w.y = n == 2 ? w.w : n == 3 ? w.z : w.y;
      w.z = n == 3 ? w.w : w.z;
    } else {
      const uint64_t v = ((uint64_t)w.y << 32 | w.x) >> (16 * ((4 - n) & 3));
      w.x = (uint32_t)v;
      w.y = (uint32_t)(v >> 32);
    }
  }
  return w;
}

// A unit's tokens in batches: the batch's rows of dout, and the rows of dW
// that its run ends add to, are all loaded before the first is used.  A lane
// takes two quads of columns, half a unit apart.  A wave holds one unit, so that
// tokens, keys and row addresses are scalars (rows of more than kNarrow columns).
// NT: dout is read with the non-temporal bit, where a wave's loads cover whole
// cache lines (rows on 16-byte boundaries); where lines are shared by two loads it
// has them fetched twice.
template <int DT, bool NT, bool FLAT>
__global__ __launch_bounds__(kT) void k_embed_sum(EmbedGradArgs a, SumArgs s, int64_t sum_blocks) {
  constexpr int EB = VecT<DT>::EB;
  constexpr int B = 4;  // (8 took the registers of a third of the waves: 75 against 71 us)
  const uint32_t D = (uint32_t)a.D, whole = D & ~3u, N = (uint32_t)a.N, none = (uint32_t)a.V;
  for (int64_t b = blockIdx.x; b < sum_blocks + s.fill_blocks; b += gridDim.x) {
    if (b >= sum_blocks) {
      __syncthreads();
      if constexpr (FLAT)
        fill_flat(a, s, b - sum_blocks);
      else
        fill_rows(a, s, b - sum_blocks);
      continue;
    }
    // (32 bits: a unit has 4 KiB of partial sums in the workspace)
    const uint32_t unit = (uint32_t)b * kWaves + (uint32_t)__builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const uint32_t cb = unit % (uint32_t)s.col_blocks;
    const int64_t t = unit / (uint32_t)s.col_blocks;
    uint32_t j[2];
    j[0] = cb * 512 + (threadIdx.x & 63) * 4;
    j[1] = j[0] + 256;
    if (t >= s.tiles) continue;
    const TileRuns run = tile_runs(s, N, none, t);
    const uint32_t i0 = run.i0, i1 = run.i1;
    bool from_before = run.from_before;
    if (j[0] >= D) continue;  // (only here: the lanes look for a run's end together)
    if (j[0] == 0) s.starts[t] = run.goes_on && !(from_before && run.one_run);
    float acc[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[h][e] = 0.f;
    for (uint32_t i = i0; i < i1; i += B) {
      uint32_t key[B + 1], idx[B];
#pragma unroll
      for (int k = 0; k < B; ++k) {
        const uint32_t at = i + k < N ? i + k : N - 1;
        key[k] = s.skey[at];
        idx[k] = s.sidx[at];
      }
      key[B] = i + B < N ? s.skey[i + B] : 0xffffffffu;
      if (key[0] == none) break;  // sorted: nothing with a gradient follows
      u32x4v row[B][2], old[B][2];
#pragma unroll
      for (int k = 0; k < B; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          row[k][h] = load_quad<DT, NT, false>(a.dout + (int64_t)idx[k] * a.dout_ld * EB, j[h], whole, D);
      if (a.accumulate) {
#pragma unroll
        for (int k = 0; k < B; ++k) {
          if (i + k < i1 && key[k] != none && (i + k + 1 >= N || key[k + 1] != key[k])) {  // a run ends here
            const char* dw = reinterpret_cast<const char*>(a.dw + (int64_t)key[k] * a.dw_ld);
#pragma unroll
            for (int h = 0; h < 2; ++h) old[k][h] = load_quad<CE_F32, false, false>(dw, j[h], whole, D);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < B; ++k) {
        if (i + k < i1 && key[k] != none) {
          const bool ends = i + k + 1 >= N || key[k + 1] != key[k];
          float* const dw = a.dw + (int64_t)key[k] * a.dw_ld;
          float* const part = s.parts + (2 * t + (from_before ? 0 : 1)) * a.D;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float f[4];
            quad_to_f32<DT>(tail_quad<DT, false>(row[k][h], j[h], whole, D), f);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[h][e] += f[e];
            if (ends || i + k + 1 == i1) {
              if (from_before || !ends) {
                if (j[h] < D) store_quad(part, j[h], D, acc[h]);
              } else {
                float o[4];
                quad_to_f32<CE_F32>(tail_quad<CE_F32, false>(old[k][h], j[h], whole, D), o);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  o[e] = a.accumulate ? __builtin_fmaf(acc[h][e], a.scale, o[e]) : acc[h][e] * a.scale;
                if (j[h] < D) store_quad<true>(dw, j[h], D, o);
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[h][e] = 0.f;
            }
          }
          if (ends || i + k + 1 == i1) from_before = false;
        }
      }
    }
  }
}

// Rows of at most kNarrow columns: a unit is a sorted token over all columns, a quad a
// lane, and works where a run starts (a short run, or a long one up to its tile's
// end) or where a tile begins inside a long one.  One token's chain of loads is what
// few tokens take, and short code: with a tile a unit and its tokens unrolled, most
// of the time went to fetching instructions (1500 x 16 BF16 tokens: 21 us for this
// launch alone).
constexpr int64_t kNarrow = 128, kFewElems = 7 << 20;
template <int DT, bool SHORT>
__global__ __launch_bounds__(kT) void k_embed_narrow(EmbedGradArgs a, SumArgs s, int64_t sum_blocks) {
  constexpr int EB = VecT<DT>::EB;
  constexpr int B = 4;
  const uint32_t D = (uint32_t)a.D, whole = D & ~3u, N = (uint32_t)a.N, none = (uint32_t)a.V, T = (uint32_t)s.tile;
  for (int64_t b = blockIdx.x; b < sum_blocks + s.fill_blocks; b += gridDim.x) {
    if (b >= sum_blocks) {
      __syncthreads();
      if (s.flat)
        fill_flat(a, s, b - sum_blocks);
      else
        fill_rows(a, s, b - sum_blocks);
      continue;
    }
    const uint32_t unit = (uint32_t)b * (uint32_t)(kT >> s.lanes_shift) + (threadIdx.x >> s.lanes_shift);
    const uint32_t i = unit / (uint32_t)s.col_blocks, cb = unit - i * (uint32_t)s.col_blocks;
    const uint32_t j = cb * 256 + (threadIdx.x & ((1u << s.lanes_shift) - 1)) * 4;
    if (i >= N) continue;
    const uint32_t t = i / T, edge = t * T, end = N - edge < T ? N : edge + T;
    const uint32_t key = s.skey[i], before = s.skey[i ? i - 1 : 0], last = s.skey[end - 1];
    const uint32_t far = s.skey[N - i > T ? i + T : N - 1];
    const bool starts = i == 0 || before != key, inside = !starts && i == edge;
    bool is_long = starts && N - i > T && far == key;
    if (inside) {
      uint32_t ahead;
      is_long = long_run<false>(s, N, i, key, &ahead);
    }
    // the first place of the tile's last run tells the join whether a long one starts
    if (j == 0 && (starts || inside) && key == last) s.starts[t] = key != none && starts && is_long;
    if (key == none || !(starts || (inside && is_long)) || j >= D) continue;
    const uint32_t stop = is_long ? end : N - i < T ? N : i + T;
    float* const to = is_long ? s.parts + (2 * (int64_t)t + (starts ? 1 : 0)) * a.D : a.dw + (int64_t)key * a.dw_ld;
    const bool add = a.accumulate && !is_long;
    u32x4v old = {0u, 0u, 0u, 0u};
    if (a.accumulate) old = load_quad<CE_F32, false, SHORT>(reinterpret_cast<const char*>(to), j, whole, D);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    uint32_t next_key[B], next_idx[B];
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const uint32_t at = i + k < N ? i + k : N - 1;
      next_key[k] = s.skey[at];
      next_idx[k] = s.sidx[at];
    }
    for (uint32_t n = i;;) {
      bool in[B];
      u32x4v row[B];
#pragma unroll
      for (int k = 0; k < B; ++k) {
        in[k] = n + k < stop && next_key[k] == key;
        const int64_t idx = in[k] ? next_idx[k] : next_idx[0];  // past the run, its first row of this step again
        row[k] = load_quad<DT, false, SHORT>(a.dout + idx * a.dout_ld * EB, j, whole, D);
      }
      n += B;
#pragma unroll
      for (int k = 0; k < B; ++k) {
        const uint32_t at = n + k < N ? n + k : N - 1;
        next_key[k] = s.skey[at];
        next_idx[k] = s.sidx[at];
      }
#pragma unroll
      for (int k = 0; k < B; ++k) {
        float f[4];
        quad_to_f32<DT>(tail_quad<DT, SHORT>(row[k], j, whole, D), f);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = in[k] ? acc[e] + f[e] : acc[e];
      }
      if (n >= stop || next_key[0] != key) break;
    }
    float o[4];
    quad_to_f32<CE_F32>(tail_quad<CE_F32, SHORT>(old, j, whole, D), o);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = is_long ? acc[e] : add ? __builtin_fmaf(acc[e], a.scale, o[e]) : acc[e] * a.scale;
    store_quad(to, j, D, o);
  }
}

// The long runs: workgroup x takes those that start in tiles x, x + 64, ... (one
// lane a tile finds them) and adds their partial sums in tile order, an eighth
// of them per wave (256 columns, four a lane).
constexpr int kJoinWaves = 8, kJoinBlocks = 64;
constexpr int kJoinT = 64 * kJoinWaves;
__global__ __launch_bounds__(kJoinT) void k_embed_join(EmbedGradArgs a, SumArgs s) {
  static_assert(kMaxTiles <= (int64_t)kJoinBlocks * 64, "one lane a tile");
  __shared__ float part[kJoinWaves][256];
  const int lane = (int)threadIdx.x & 63, w = (int)threadIdx.x >> 6;
  const uint32_t D = (uint32_t)a.D;
  const int64_t look = blockIdx.x + (int64_t)lane * kJoinBlocks;
  uint64_t found = __ballot(look < s.tiles && s.starts[look < s.tiles ? look : 0] != 0u);
  while (found) {
    const int64_t t = blockIdx.x + (int64_t)__builtin_ctzll(found) * kJoinBlocks;
    found &= found - 1;
    const uint32_t key = s.skey[(t + 1) * s.tile];
    // tiles t + 1 .. t + n - 1 begin with the run's key: one lane a tile
    int64_t n = 1;
    for (int64_t u = t + 1;; u += 64) {
      const bool in = u + lane < s.tiles && s.skey[(u + lane) * s.tile] == key;
      const uint64_t all = __ballot(in);
      n += all == ~(uint64_t)0 ? 64 : __builtin_ctzll(~all);
      if (all != ~(uint64_t)0) break;
    }
    const int64_t per = ceil_div(n, kJoinWaves);
    const int64_t k0 = w * per, k1 = min64(k0 + per, n);
    for (uint32_t c = blockIdx.y * 256; c < D; c += gridDim.y * 256) {
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int64_t k = k0; k < k1; ++k) {
        const float* p = s.parts + (k == 0 ? 2 * t + 1 : 2 * (t + k)) * a.D + c;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] += p[c + e * 64 + lane < D ? e * 64 + lane : 0];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) part[w][e * 64 + lane] = acc[e];
      __syncthreads();
      if (threadIdx.x < 256 && c + threadIdx.x < D) {
        float v = part[0][threadIdx.x];
#pragma unroll
        for (int k = 1; k < kJoinWaves; ++k) v += part[k][threadIdx.x];
        float* d = a.dw + (int64_t)key * a.dw_ld + c + threadIdx.x;
        *d = a.accumulate ? __builtin_fmaf(v, a.scale, *d) : v * a.scale;
      }
      __syncthreads();
    }
  }
}

template <int DT>
void launch_sum(const EmbedGradArgs& a, const SumArgs& s, int64_t sum_blocks, dim3 grid, hipStream_t stream) {
  if (a.D < 4)
    hipLaunchKernelGGL((k_embed_narrow<DT, true>), grid, dim3(kT), 0, stream, a, s, sum_blocks);
  else if (s.narrow)
    hipLaunchKernelGGL((k_embed_narrow<DT, false>), grid, dim3(kT), 0, stream, a, s, sum_blocks);
  else if (s.flat)  // (not in the others: its registers cost 8192 x 4096 BF16, added to, 60 instead of 57 us)
    hipLaunchKernelGGL((k_embed_sum<DT, false, true>), grid, dim3(kT), 0, stream, a, s, sum_blocks);
  else if ((uintptr_t)a.dout % 16 == 0 && a.dout_ld % kG == 0)
    hipLaunchKernelGGL((k_embed_sum<DT, true, false>), grid, dim3(kT), 0, stream, a, s, sum_blocks);
  else
    hipLaunchKernelGGL((k_embed_sum<DT, false, false>), grid, dim3(kT), 0, stream, a, s, sum_blocks);
}

// Workspace: sorted keys and positions (twice for the radix sort's passes), its counts, the partial sums.
struct GradLayout {
  bool rank;
  int key_bits, passes, digit;
  int64_t sort_tiles, tile, tiles;
  size_t keys[2], idx[2], hist, starts, parts, total;
};

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

GradLayout grad_layout(int64_t N, int64_t D, int64_t V) {
  GradLayout g{};
  g.key_bits = bits_of(V);
  g.rank = N <= kRankMax && g.key_bits + bits_of(N - 1) < 32;  // the all-ones pair stays free
  g.passes = g.rank ? 0 : (g.key_bits + kMaxDigit - 1) / kMaxDigit;
  g.digit = g.rank ? 0 : (g.key_bits + g.passes - 1) / g.passes;
  g.sort_tiles = ceil_div(N, kSortTile);
  // tokens per tile: 16, more where that would leave over kMaxTiles tiles (and twice as many partial sums)
  g.tile = ceil_div(N, kMaxTiles);
  if (g.tile < kTileTokens) g.tile = kTileTokens;
  g.tiles = ceil_div(N, g.tile);
  size_t off = 0;
  for (int k = 0; k < (g.rank ? 1 : 2); ++k) {
    g.keys[k] = off;
    off = align256(off + (size_t)N * 4);
    g.idx[k] = off;
    off = align256(off + (size_t)N * 4);
  }
  g.hist = off;
  if (!g.rank) off = align256(off + ((size_t)g.sort_tiles << g.digit) * 4);
  g.starts = off;
  off = align256(off + (size_t)min64(ceil_div(N, kTileTokens), kMaxTiles) * 4);
  g.parts = off;
  // (room for the tiles of any smaller N too: a workspace serves batches up to its own)
  off = align256(off + (size_t)min64(ceil_div(N, kTileTokens), kMaxTiles) * 2 * (size_t)D * 4);
  g.total = off < 256 ? 256 : off;
  return g;
}

}  // namespace

hipError_t launch_embed(const EmbedArgs& a, hipStream_t stream) {
  if (a.N == 0) return hipSuccess;
  const int sh = lanes_log2(ceil_div(a.D, kG));
  const dim3 grid((uint32_t)min64(ceil_div(a.N, kT >> sh), kMaxBlocks));
  if (a.dtype == CE_BF16)
    hipLaunchKernelGGL(k_embed<CE_BF16>, grid, dim3(kT), 0, stream, a, sh);
  else
    hipLaunchKernelGGL(k_embed<CE_F32>, grid, dim3(kT), 0, stream, a, sh);
  return hipGetLastError();
}

size_t embed_grad_workspace(int64_t N, int64_t D, int64_t V) {
  return direct(N, D) ? 256 : grad_layout(N, D, V).total;
}

hipError_t launch_embed_grad(const EmbedGradArgs& a, hipStream_t stream) {
  hipError_t e;
  if (a.N == 0) return a.accumulate ? hipSuccess : launch_fill_f32(a.dw, a.V, a.D, a.dw_ld, stream);
  if (direct(a.N, a.D)) return a.dtype == CE_BF16 ? launch_direct<CE_BF16>(a, stream) : launch_direct<CE_F32>(a, stream);
  const GradLayout g = grad_layout(a.N, a.D, a.V);
  uint32_t* key[2] = {reinterpret_cast<uint32_t*>(a.ws + g.keys[0]), reinterpret_cast<uint32_t*>(a.ws + g.keys[1])};
  uint32_t* idx[2] = {reinterpret_cast<uint32_t*>(a.ws + g.idx[0]), reinterpret_cast<uint32_t*>(a.ws + g.idx[1])};
  int cur = 0;
  if (g.rank) {
    hipLaunchKernelGGL(k_rank, dim3((uint32_t)ceil_div(a.N, kRankTokens)), dim3(kRankT), 0, stream, a,
                       bits_of(a.N - 1), key[0], idx[0]);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  } else {
    for (int p = 0; p < g.passes; ++p) {
      SortPass s;
      s.key_in = p ? key[cur] : nullptr;
      s.idx_in = p ? idx[cur] : nullptr;
      s.key_out = key[p ? cur ^ 1 : 0];
      s.idx_out = idx[p ? cur ^ 1 : 0];
      s.hist = reinterpret_cast<uint32_t*>(a.ws + g.hist);
      s.tiles = g.sort_tiles;
      s.shift = p * g.digit;
      s.bits = g.digit;
      if (p) cur ^= 1;
      if (a.N <= kOneMax) {
        hipLaunchKernelGGL(k_sort_one, dim3((uint32_t)ceil_div(a.N, kOneT)), dim3(kOneT), 0, stream, a, s);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        continue;
      }
      const dim3 grid((uint32_t)g.sort_tiles);
      hipLaunchKernelGGL(k_sort_count, grid, dim3(kT), 0, stream, a, s);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      hipLaunchKernelGGL(k_sort_scan, dim3(1), dim3(1024), 0, stream, s.hist, g.sort_tiles << g.digit);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      hipLaunchKernelGGL(k_sort_move, grid, dim3(kT), 0, stream, a, s);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  SumArgs s;
  s.skey = key[cur];
  s.sidx = idx[cur];
  s.parts = reinterpret_cast<float*>(a.ws + g.parts);
  s.starts = reinterpret_cast<uint32_t*>(a.ws + g.starts);
  s.tiles = g.tiles;
  s.tile = g.tile;
  const bool narrow = a.D <= kNarrow || a.N * a.D <= kFewElems;
  s.narrow = narrow;
  s.lanes_shift = narrow ? (int)min64(lanes_log2(ceil_div(a.D, 4)), 6) : 0;
  s.col_blocks = ceil_div(a.D, narrow ? 256 : 512);
  s.flat = !a.accumulate && end_to_end(a) && a.D <= kFlatCols;
  s.fill_blocks = a.accumulate ? 0 : s.flat ? ceil_div(a.V * a.D, kFlat) : ceil_div(a.V, kFillRows);
  const int64_t sum_blocks =
      narrow ? ceil_div(a.N * s.col_blocks, kT >> s.lanes_shift) : ceil_div(g.tiles * s.col_blocks, kWaves);
  const dim3 grid((uint32_t)min64(sum_blocks + s.fill_blocks, kMaxBlocks));
  if (a.dtype == CE_BF16)
    launch_sum<CE_BF16>(a, s, sum_blocks, grid, stream);
  else
    launch_sum<CE_F32>(a, s, sum_blocks, grid, stream);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (g.tiles > 1) {
    const dim3 jgrid((uint32_t)min64(g.tiles - 1, kJoinBlocks), (uint32_t)min64(ceil_div(a.D, 256), 16));
    hipLaunchKernelGGL(k_embed_join, jgrid, dim3(kJoinT), 0, stream, a, s);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace vce
