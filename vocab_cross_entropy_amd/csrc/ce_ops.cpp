// C ABI of the operators around the loss: logit processing, embedding, RMS norm,
// token log-probabilities and distillation.  Argument checks, then one call of the launcher; every check runs
// before the first HIP call, so a rejected call enqueues nothing.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <initializer_list>

#include <hip/hip_runtime_api.h>

#include "ce.h"
#include "ce_internal.h"

namespace {

ce_status ofail(ce_status s, const char* fmt, ...) {
  char msg[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  vce::set_last_error(msg);
  return s;
}

ce_status launched(hipError_t e, const char* what) {
  return e == hipSuccess ? CE_OK : ofail(CE_EHIP, "%s: %s", what, hipGetErrorString(e));
}

int elem_bytes(int32_t dtype) { return dtype == CE_BF16 ? 2 : 4; }
bool known(int32_t dtype) { return dtype == CE_F32 || dtype == CE_BF16; }
bool off(const void* p, int32_t dtype) { return (uintptr_t)p % (uintptr_t)elem_bytes(dtype) != 0; }

constexpr int64_t kMax31 = 0x7fffffffLL;
constexpr int64_t kMaxCols32 = 0xffffffffLL / 4;  // FP32 columns of a row below 4 GiB: kernels use 32-bit byte offsets

// a matrix of `rows` rows of D contiguous elements, ld apart
ce_status check_rows(const char* name, const void* p, int32_t dtype, int64_t rows, int64_t D, int64_t ld) {
  if (rows > 0 && !p) return ofail(CE_EINVAL, "%s is NULL", name);
  if (off(p, dtype)) return ofail(CE_ELAYOUT, "%s is not aligned to its dtype", name);
  if (ld < D) return ofail(CE_ELAYOUT, "the row stride of %s must be >= %lld (got %lld)", name, (long long)D, (long long)ld);
  return CE_OK;
}

// n0 x n1 rows of `width` bytes, s0 and s1 bytes apart, none of which meets another
struct RowSet {
  typedef __int128 wide;  // (strides are the caller's numbers)
  wide p, n0, n1, s0, s1, width;
};
RowSet row_set(const void* p, int64_t n0, int64_t n1, int64_t s0, int64_t s1, int64_t columns, int bytes) {
  typedef RowSet::wide wide;
  return {(wide)(uintptr_t)p, n0, n1, n0 > 1 ? (wide)s0 * bytes : 0, n1 > 1 ? (wide)s1 * bytes : 0, (wide)columns * bytes};
}

// Whether two sets of equally many rows meet anywhere, other than by being the same rows where that is allowed.
// Exact where their strides are equal (columns side by side, rows in turn); sets of other strides may not share a
// range of addresses.
bool rows_meet(const RowSet& a, const RowSet& b, bool in_place) {
  typedef RowSet::wide wide;
  if (a.n0 == 0 || a.n1 == 0) return false;
  const bool alike = a.s0 == b.s0 && a.s1 == b.s1;
  if (a.p == b.p && alike && a.width == b.width) return !in_place;
  const auto end = [](const RowSet& r) { return r.p + (r.n0 - 1) * r.s0 + (r.n1 - 1) * r.s1 + r.width; };
  if (end(a) <= b.p || end(b) <= a.p) return false;
  if (!alike) return true;
  // b's row lies i outer and j inner steps from a's: only the steps next to where the two are nearest can meet
  const bool outer0 = a.s0 >= a.s1;
  const wide so = outer0 ? a.s0 : a.s1, no = outer0 ? a.n0 : a.n1, si = outer0 ? a.s1 : a.s0, ni = outer0 ? a.n1 : a.n0;
  const wide off = b.p - a.p, io = so ? -off / so : 0;
  for (wide i = io - 1; i <= io + 1; ++i) {
    if (i <= -no || i >= no) continue;
    const wide rest = off + i * so, ji = si ? -rest / si : 0;
    for (wide j = ji - 1; j <= ji + 1; ++j) {
      if (j <= -ni || j >= ni) continue;
      const wide d = rest + j * si;
      if (d < a.width && -d < b.width) return true;
    }
  }
  return false;
}

ce_status overlap(const char* out, const char* other) {
  return ofail(CE_ELAYOUT, "%s overlaps %s (in place: the same address and strides, where that is allowed)", out, other);
}

// ---- logit processing
ce_status check_process(const ce_logits* x, const ce_logits* out, const ce_process* p, bool backward) {
  ce_status st;
  if ((st = vce::check_logits_desc(x)) || (st = vce::check_logits_desc(out))) return st;
  if (!p) return ofail(CE_EINVAL, "process descriptor is NULL");
  if (x->dtype != out->dtype) return ofail(CE_EDTYPE, "input and output differ in dtype");
  if (x->d0 != out->d0 || x->d1 != out->d1 || x->v_local != out->v_local || x->vocab_start != out->vocab_start ||
      x->vocab_total != out->vocab_total)
    return ofail(CE_ELAYOUT, "input and output differ in shape");
  const int eb = elem_bytes(x->dtype);
  if (rows_meet(row_set(x->data, x->d0, x->d1, x->s0, x->s1, x->v_local, eb),
                row_set(out->data, out->d0, out->d1, out->s0, out->s1, out->v_local, eb), true))
    return overlap("the output", "the input");
  if (p->history) {
    if ((uintptr_t)p->history % 8u || p->history_s0 < 0 || p->history_s1 < 0)
      return ofail(CE_ELAYOUT, "history misaligned or negative stride");
    if (p->history_max < 0 || p->history_max > kMax31)
      return ofail(CE_EINVAL, "history_max %lld outside [0, 2^31)", (long long)p->history_max);
  } else if (p->history_len || p->prompt_len || p->history_max) {
    return ofail(CE_EINVAL, "history_len, prompt_len and history_max need a history");
  }
  for (const void* q : {(const void*)p->history_len, (const void*)p->prompt_len, (const void*)p->repetition,
                        (const void*)p->frequency, (const void*)p->presence, (const void*)p->temperature,
                        (const void*)p->bias, (const void*)p->mask})
    if ((uintptr_t)q % 4u) return ofail(CE_ELAYOUT, "a per-row parameter, bias or mask is not 4-byte aligned");
  if (!p->history && (p->repetition || p->frequency || p->presence))
    return ofail(CE_EINVAL, "penalties need a history");
  if (p->bias && x->v_local > kMaxCols32)
    return ofail(CE_ELAYOUT, "bias rows of %lld columns exceed 4 GiB", (long long)x->v_local);
  if (p->bias && (p->bias_s0 < 0 || p->bias_s1 < 0)) return ofail(CE_ELAYOUT, "negative bias strides are not supported");
  if (p->mask && (p->mask_s0 < 0 || p->mask_s1 < 0)) return ofail(CE_ELAYOUT, "negative mask strides are not supported");
  if (p->signs && p->signs_ld < (x->v_local + 7) / 8)
    return ofail(CE_ELAYOUT, "signs_ld %lld is below %lld bytes", (long long)p->signs_ld,
                 (long long)((x->v_local + 7) / 8));
  if (backward && p->repetition && !p->signs)
    return ofail(CE_EINVAL, "the gradient of a repetition penalty needs the forward's signs");
  return CE_OK;
}

ce_status process(const ce_logits* x, const ce_logits* out, const ce_process* p, bool backward, hipStream_t stream) {
  ce_status st = check_process(x, out, p, backward);
  if (st) return st;
  vce::ProcessArgs a{};
  a.x = static_cast<const char*>(x->data);
  a.z = static_cast<char*>(out->data);
  a.dtype = x->dtype;
  a.N = x->d0 * x->d1;
  a.d1 = x->d1;
  a.V = x->v_local;
  a.s0 = x->s0;
  a.s1 = x->s1;
  a.zs0 = out->s0;
  a.zs1 = out->s1;
  a.vocab_start = x->vocab_start;
  // the gradient looks at the history for the repetition penalty alone
  if (!backward || p->repetition) {
    a.hist = p->history;
    a.hs0 = p->history_s0;
    a.hs1 = p->history_s1;
    a.hist_max = p->history_max;
    a.hist_len = p->history_len;
    a.prompt_len = p->prompt_len;
  }
  if (!p->repetition && !p->frequency && !p->presence) a.hist = nullptr;
  a.repetition = p->repetition;
  a.frequency = p->frequency;
  a.presence = p->presence;
  a.temperature = p->temperature;
  a.bias = p->bias;
  a.bs0 = p->bias_s0;
  a.bs1 = p->bias_s1;
  a.mask = p->mask;
  a.ms0 = p->mask_s0;
  a.ms1 = p->mask_s1;
  a.signs = p->signs;
  a.signs_ld = p->signs_ld;
  if (a.N == 0) return CE_OK;
  vce::process_plan(&a);
  if (a.chunks > 0xffffffffLL / a.N) return ofail(CE_EINVAL, "more than 2^32-1 chunks of columns");
  hipEvent_t e0, e1;
  vce::profile_next(a.N, &e0, &e1);
  return launched(vce::launch_process(a, backward, stream, e0, e1), backward ? "process backward" : "process");
}

// ---- token log-probabilities and distillation: whole rows
ce_status check_whole_rows(const ce_logits* x, int64_t most) {
  const ce_status st = vce::check_logits_desc(x);
  if (st) return st;
  if (x->vocab_start != 0 || x->v_local != x->vocab_total)
    return ofail(CE_ELAYOUT, "this call needs unsharded logits (vocab_start 0, v_local == vocab_total)");
  if (x->v_local > most)
    return ofail(CE_ELAYOUT, "rows of %lld columns exceed %lld", (long long)x->v_local, (long long)most);
  return CE_OK;
}

// `out` takes x's rows in place or lies elsewhere
ce_status check_gradient_rows(const ce_logits* x, const ce_logits* out) {
  const ce_status st = vce::check_logits_desc(out);
  if (st) return st;
  if (x->dtype != out->dtype) return ofail(CE_EDTYPE, "logits and gradient differ in dtype");
  if (x->d0 != out->d0 || x->d1 != out->d1 || x->v_local != out->v_local || x->vocab_start != out->vocab_start ||
      x->vocab_total != out->vocab_total)
    return ofail(CE_ELAYOUT, "logits and gradient differ in shape");
  const int eb = elem_bytes(x->dtype);
  if (rows_meet(row_set(x->data, x->d0, x->d1, x->s0, x->s1, x->v_local, eb),
                row_set(out->data, out->d0, out->d1, out->s0, out->s1, out->v_local, eb), true))
    return overlap("the gradient", "the logits");
  return CE_OK;
}

ce_status check_prepared(const void* ws, size_t ws_bytes, size_t need) {
  if (!ws || ws_bytes < need)
    return ofail(CE_EWORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? ws_bytes : (size_t)0);
  if ((uintptr_t)ws % 256u) return ofail(CE_EWORKSPACE, "workspace must be 256-byte aligned");
  return CE_OK;
}

ce_status check_aligned(std::initializer_list<const void*> ps, unsigned bytes, const char* what) {
  for (const void* p : ps)
    if ((uintptr_t)p % bytes) return ofail(CE_ELAYOUT, "%s is not %u-byte aligned", what, bytes);
  return CE_OK;
}

ce_status check_logprobs(const ce_logits* x, const ce_logprobs* q) {
  if (!q) return ofail(CE_EINVAL, "logprobs descriptor is NULL");
  if (q->M < 0 || q->M > vce::kLogprobMaxList || q->K < 0 || q->K > vce::kLogprobMaxList)
    return ofail(CE_EINVAL, "M = %d or K = %d outside [0, %d]", q->M, q->K, vce::kLogprobMaxList);
  if (q->K > x->v_local)
    return ofail(CE_EINVAL, "%d alternatives of %lld columns", q->K, (long long)x->v_local);
  if (q->M > 0 && x->d0 > 0 && !q->ids) return ofail(CE_EINVAL, "ids is NULL");
  if ((uintptr_t)q->ids % 8u || q->ids_s0 < 0 || q->ids_s1 < 0)
    return ofail(CE_ELAYOUT, "ids misaligned or negative stride");
  return CE_OK;
}

ce_status check_distill(const ce_logits* x, const ce_distill* d) {
  if (!d) return ofail(CE_EINVAL, "distillation descriptor is NULL");
  if (d->K < 1 || d->K > vce::kDistillMaxTop)
    return ofail(CE_EINVAL, "%d entries a row outside [1, %d]", d->K, vce::kDistillMaxTop);
  if (!known(d->values_dtype)) return ofail(CE_EDTYPE, "unsupported dtype %d of the teacher's values", d->values_dtype);
  if (d->kind != CE_TEACHER_LOGITS && d->kind != CE_TEACHER_LOGPROBS)
    return ofail(CE_EINVAL, "unknown kind of teacher values %d", d->kind);
  if (!(d->temperature >= 0x1p-32f && d->temperature <= 0x1p32f))
    return ofail(CE_EINVAL, "temperature %g outside [2^-32, 2^32]", (double)d->temperature);
  if (x->d0 > 0 && (!d->ids || !d->values)) return ofail(CE_EINVAL, "the teacher's ids or values are NULL");
  if ((uintptr_t)d->ids % 8u || d->ids_s0 < 0 || d->ids_s1 < 0)
    return ofail(CE_ELAYOUT, "ids misaligned or negative stride");
  if (off(d->values, d->values_dtype) || d->values_s0 < 0 || d->values_s1 < 0)
    return ofail(CE_ELAYOUT, "the teacher's values are misaligned or have a negative stride");
  return check_aligned({d->len}, 4, "len");
}

// ---- embedding
ce_status check_embedding(const ce_embedding_desc* m, bool table) {
  if (!m) return ofail(CE_EINVAL, "embedding descriptor is NULL");
  if (!known(m->dtype)) return ofail(CE_EDTYPE, "unsupported dtype %d", m->dtype);
  if (m->reserved != 0) return ofail(CE_EINVAL, "embedding.reserved must be 0");
  if (m->N < 0 || m->N > vce::kEmbedMaxTokens)
    return ofail(CE_EINVAL, "%lld tokens outside [0, 2^26]", (long long)m->N);
  if (m->D < 1 || m->D > kMax31 || m->v_local < 1 || m->v_local > kMax31)
    return ofail(CE_EINVAL, "need 1 <= D, v_local < 2^31 (got %lld, %lld)", (long long)m->D, (long long)m->v_local);
  if (m->D > kMaxCols32) return ofail(CE_ELAYOUT, "rows of %lld FP32 columns exceed 4 GiB", (long long)m->D);
  if (m->vocab_start < 0 || m->vocab_total < 1 || m->vocab_start > m->vocab_total - m->v_local)
    return ofail(CE_ELAYOUT, "shard [%lld, %lld) does not fit a vocabulary of %lld", (long long)m->vocab_start,
                 (long long)(m->vocab_start + m->v_local), (long long)m->vocab_total);
  if (m->N > 0 && !m->ids) return ofail(CE_EINVAL, "ids is NULL");
  if ((uintptr_t)m->ids % 8u || m->id_stride < 0) return ofail(CE_ELAYOUT, "ids misaligned or negative stride");
  if (table) return check_rows("weight", m->weight, m->dtype, m->v_local, m->D, m->w_ld);
  return CE_OK;
}

// ---- RMS norm
ce_status check_norm(const ce_norm* n) {
  if (!n) return ofail(CE_EINVAL, "norm descriptor is NULL");
  if (!known(n->dtype)) return ofail(CE_EDTYPE, "unsupported dtype %d", n->dtype);
  if (!known(n->weight_dtype)) return ofail(CE_EDTYPE, "unsupported weight dtype %d", n->weight_dtype);
  if (n->N < 0 || n->N > kMax31) return ofail(CE_EINVAL, "%lld rows outside [0, 2^31)", (long long)n->N);
  if (n->D < 1) return ofail(CE_EINVAL, "D must be >= 1");
  if (n->D > vce::kNormMaxCols)
    return ofail(CE_ELAYOUT, "rows of %lld columns exceed %lld", (long long)n->D, (long long)vce::kNormMaxCols);
  if (!(n->eps >= 0.f) || !isfinite(n->eps)) return ofail(CE_EINVAL, "eps %g is not a finite value >= 0", (double)n->eps);
  if (!n->weight) return ofail(CE_EINVAL, "weight is NULL");
  if (off(n->weight, n->weight_dtype)) return ofail(CE_ELAYOUT, "weight is not aligned to its dtype");
  return check_rows("x", n->x, n->dtype, n->N, n->D, n->x_ld);
}

ce_status norm(const ce_norm* n, void* y, int64_t y_ld, void* q, int64_t q_ld, int32_t group, float* scales, void* sum,
               int64_t sum_ld, hipStream_t stream) {
  ce_status st;
  if (n->residual && (st = check_rows("residual", n->residual, n->dtype, n->N, n->D, n->residual_ld))) return st;
  if (sum && (st = check_rows("sum", sum, n->dtype, n->N, n->D, sum_ld))) return st;
  const int eb = elem_bytes(n->dtype);
  const auto rows = [n](const void* p, int64_t ld, int bytes) { return row_set(p, n->N, 1, ld, 0, n->D, bytes); };
  const RowSet xs = rows(n->x, n->x_ld, eb), rs = rows(n->residual, n->residual_ld, eb), ss = rows(sum, sum_ld, eb);
  const RowSet ys = q ? rows(q, q_ld, 1) : rows(y, y_ld, eb);
  const char* const name = q ? "q" : "y";
  if (rows_meet(ys, xs, !q)) return overlap(name, "x");
  if (n->residual && rows_meet(ys, rs, !q)) return overlap(name, "residual");
  if (sum) {
    if (rows_meet(ys, ss, false)) return overlap(name, "sum");
    if (rows_meet(ss, xs, true)) return overlap("sum", "x");
    if (n->residual && rows_meet(ss, rs, true)) return overlap("sum", "residual");
  }
  vce::NormArgs a{};
  a.x = static_cast<const char*>(n->x);
  a.residual = static_cast<const char*>(n->residual);
  a.weight = static_cast<const char*>(n->weight);
  a.dtype = n->dtype;
  a.wdtype = n->weight_dtype;
  a.N = n->N;
  a.D = n->D;
  a.x_ld = n->x_ld;
  a.r_ld = n->residual_ld;
  a.eps = n->eps;
  a.y = static_cast<char*>(y);
  a.y_ld = y_ld;
  a.q = static_cast<uint8_t*>(q);
  a.q_ld = q_ld;
  a.scales = scales;
  a.group = group;
  a.group_shift = group == 32 ? 5 : group == 64 ? 6 : 7;
  a.groups = group ? (n->D + group - 1) / group : 1;
  a.sum = static_cast<char*>(sum);
  a.sum_ld = sum_ld;
  return launched(vce::launch_norm(a, stream), "norm launch");
}

}  // namespace

extern "C" {

ce_status ce_logits_process(const ce_logits* x, const ce_logits* out, const ce_process* p, hipStream_t stream) {
  return process(x, out, p, false, stream);
}

ce_status ce_logits_process_backward(const ce_logits* dz, const ce_logits* out, const ce_process* p,
                                     hipStream_t stream) {
  return process(dz, out, p, true, stream);
}

size_t ce_token_logprobs_workspace_bytes(const ce_logits* x, int32_t K) {
  const ce_logprobs q{nullptr, 0, 0, 0, K, 0};
  if (vce::check_logits_desc(x) || check_whole_rows(x, vce::logprob_max_cols(x->dtype)) || check_logprobs(x, &q))
    return 0;
  const size_t need = vce::logprob_workspace(x->d0 * x->d1, x->v_local, x->dtype, K);
  return need < 256 ? 256 : (need + 255) / 256 * 256;
}

ce_status ce_token_logprobs(const ce_logits* x, const ce_logprobs* q, float* logp, float* entropy, float* lse,
                            int64_t* top_ids, float* top_logp, float* stats, void* ws, size_t ws_bytes,
                            hipStream_t stream) {
  ce_status st;
  if ((st = vce::check_logits_desc(x)) || (st = check_whole_rows(x, vce::logprob_max_cols(x->dtype))) ||
      (st = check_logprobs(x, q)))
    return st;
  const int64_t N = x->d0 * x->d1;
  if (N > 0 && q->M > 0 && !logp) return ofail(CE_EINVAL, "logp is NULL");
  if (N > 0 && q->K > 0 && (!top_ids || !top_logp)) return ofail(CE_EINVAL, "top_ids or top_logp is NULL");
  if ((st = check_aligned({logp, entropy, lse, top_logp}, 4, "an output")) ||
      (st = check_aligned({top_ids}, 8, "top_ids")) || (st = check_aligned({stats}, 16, "stats")))
    return st;
  const size_t need = vce::logprob_workspace(N, x->v_local, x->dtype, q->K);
  if (need && (st = check_prepared(ws, ws_bytes, need))) return st;
  if (N == 0 || (q->M == 0 && q->K == 0 && !entropy && !lse && !stats)) return CE_OK;
  vce::LogprobArgs a{};
  a.x = static_cast<const char*>(x->data);
  a.dtype = x->dtype;
  a.N = N;
  a.d1 = x->d1;
  a.V = x->v_local;
  a.s0 = x->s0;
  a.s1 = x->s1;
  a.ids = q->M ? q->ids : nullptr;
  a.is0 = q->ids_s0;
  a.is1 = q->ids_s1;
  a.M = q->M;
  a.K = q->K;
  a.ignore_idx = q->ignore_idx;
  a.logp = logp;
  a.entropy = entropy;
  a.lse = lse;
  a.top_ids = top_ids;
  a.top_logp = top_logp;
  a.stats = stats;
  vce::logprob_plan(N, a.V, a.dtype, &a.shape, &a.chunks, &a.chunk_cols);
  hipEvent_t e0, e1;
  vce::profile_next(N, &e0, &e1);
  return launched(vce::launch_logprobs(a, ws, stream, e0, e1), "log-probabilities launch");
}

ce_status ce_token_logprobs_backward(const ce_logits* x, const ce_logits* out, const ce_logprobs* q,
                                     const float* stats, const float* dlogp, const float* dentropy,
                                     const int64_t* top_ids, const float* dtop, hipStream_t stream) {
  ce_status st;
  if ((st = vce::check_logits_desc(x)) || (st = check_whole_rows(x, vce::logprob_max_cols(x->dtype))) ||
      (st = check_gradient_rows(x, out)) || (st = check_logprobs(x, q)))
    return st;
  const int64_t N = x->d0 * x->d1;
  if (N > 0 && !stats) return ofail(CE_EINVAL, "stats is NULL");
  if (N > 0 && q->M > 0 && !dlogp) return ofail(CE_EINVAL, "dlogp is NULL");
  if (N > 0 && q->K > 0 && (!top_ids || !dtop)) return ofail(CE_EINVAL, "top_ids or dtop is NULL");
  if ((st = check_aligned({dlogp, dentropy, dtop}, 4, "a gradient")) ||
      (st = check_aligned({top_ids}, 8, "top_ids")) || (st = check_aligned({stats}, 16, "stats")))
    return st;
  if (N == 0) return CE_OK;
  vce::LogprobGradArgs a{};
  a.x = static_cast<const char*>(x->data);
  a.out = static_cast<char*>(out->data);
  a.dtype = x->dtype;
  a.N = N;
  a.d1 = x->d1;
  a.V = x->v_local;
  a.s0 = x->s0;
  a.s1 = x->s1;
  a.os0 = out->s0;
  a.os1 = out->s1;
  a.ids = q->ids;
  a.is0 = q->ids_s0;
  a.is1 = q->ids_s1;
  a.M = q->M;
  a.K = q->K;
  a.ignore_idx = q->ignore_idx;
  a.stats = stats;
  a.dlogp = dlogp;
  a.dentropy = dentropy;
  a.top_ids = top_ids;
  a.dtop = dtop;
  hipEvent_t e0, e1;
  vce::profile_next(N, &e0, &e1);
  return launched(vce::launch_logprobs_bwd(a, stream, e0, e1), "log-probabilities gradient launch");
}

size_t ce_distill_workspace_bytes(const ce_logits* x) {
  if (vce::check_logits_desc(x) || check_whole_rows(x, vce::distill_max_cols(x->dtype))) return 0;
  return (vce::distill_workspace(x->d0 * x->d1, x->v_local, x->dtype) + 255) / 256 * 256;
}

ce_status ce_distill_fwd_bwd(const ce_logits* x, const ce_logits* out, const ce_distill* d, int32_t reduce_loss,
                             const float* grad_out, float* loss, int32_t* n_valid, void* ws, size_t ws_bytes,
                             hipStream_t stream) {
  ce_status st;
  if ((st = vce::check_logits_desc(x)) || (st = check_whole_rows(x, vce::distill_max_cols(x->dtype))) ||
      (out && (st = check_gradient_rows(x, out))) || (st = check_distill(x, d)))
    return st;
  if (reduce_loss != CE_REDUCE_NONE && reduce_loss != CE_REDUCE_MEAN && reduce_loss != CE_REDUCE_SUM)
    return ofail(CE_EINVAL, "unknown reduction %d", reduce_loss);
  const int64_t N = x->d0 * x->d1;
  if (!loss && (N > 0 || reduce_loss != CE_REDUCE_NONE)) return ofail(CE_EINVAL, "loss is NULL");
  if ((st = check_aligned({grad_out, loss, n_valid}, 4, "grad_out, loss or n_valid")) ||
      (st = check_prepared(ws, ws_bytes, vce::distill_workspace(N, x->v_local, x->dtype))))
    return st;
  vce::DistillArgs a{};
  a.x = static_cast<const char*>(x->data);
  a.out = out ? static_cast<char*>(out->data) : nullptr;
  a.dtype = x->dtype;
  a.N = N;
  a.d1 = x->d1;
  a.V = x->v_local;
  a.s0 = x->s0;
  a.s1 = x->s1;
  if (out) {
    a.os0 = out->s0;
    a.os1 = out->s1;
  }
  a.ids = d->ids;
  a.is0 = d->ids_s0;
  a.is1 = d->ids_s1;
  a.teacher = static_cast<const char*>(d->values);
  a.ts0 = d->values_s0;
  a.ts1 = d->values_s1;
  a.tdtype = d->values_dtype;
  a.kind = d->kind;
  a.K = d->K;
  a.len = d->len;
  a.t = (double)d->temperature;
  a.inv_t = 1.0 / a.t;
  a.kb64 = 1.4426950408889634074 / a.t;
  a.kb = (float)a.kb64;
  a.reduce = reduce_loss;
  a.g = grad_out;
  a.loss = loss;
  vce::distill_plan(a.V, a.dtype, &a.chunks, &a.chunk_cols);
  hipEvent_t e0, e1;
  vce::profile_next(N, &e0, &e1);
  return launched(vce::launch_distill(a, ws, n_valid, stream, e0, e1), "distillation launch");
}

ce_status ce_embedding(const ce_embedding_desc* m, void* out, int64_t out_ld, hipStream_t stream) {
  ce_status st;
  if ((st = check_embedding(m, true)) || (st = check_rows("out", out, m->dtype, m->N, m->D, out_ld))) return st;
  vce::EmbedArgs a{};
  a.ids = m->ids;
  a.id_stride = m->id_stride;
  a.N = m->N;
  a.D = m->D;
  a.w = static_cast<const char*>(m->weight);
  a.w_ld = m->w_ld;
  a.V = m->v_local;
  a.vocab_start = m->vocab_start;
  a.vocab_total = m->vocab_total;
  a.out = static_cast<char*>(out);
  a.out_ld = out_ld;
  a.dtype = m->dtype;
  a.scale = m->scale;
  return launched(vce::launch_embed(a, stream), "embedding launch");
}

size_t ce_embedding_workspace_bytes(int64_t N, int64_t D, int64_t v_local) {
  if (N < 0 || N > vce::kEmbedMaxTokens || D < 1 || D > kMax31 || v_local < 1 || v_local > kMax31) {
    ofail(CE_EINVAL, "need 0 <= N <= 2^26 and 1 <= D, v_local < 2^31 (got %lld, %lld, %lld)", (long long)N,
          (long long)D, (long long)v_local);
    return 0;
  }
  return vce::embed_grad_workspace(N, D, v_local);
}

ce_status ce_embedding_backward(const ce_embedding_desc* m, const void* dout, int64_t dout_ld, int64_t padding_idx,
                                float* dw, int64_t dw_ld, int32_t accumulate, void* ws, size_t ws_bytes,
                                hipStream_t stream) {
  ce_status st;
  if ((st = check_embedding(m, false)) || (st = check_rows("dout", dout, m->dtype, m->N, m->D, dout_ld)) ||
      (st = check_rows("dw", dw, CE_F32, m->v_local, m->D, dw_ld)))
    return st;
  if (accumulate != 0 && accumulate != 1) return ofail(CE_EINVAL, "accumulate must be 0 or 1");
  const size_t need = vce::embed_grad_workspace(m->N, m->D, m->v_local);
  if (!ws || ws_bytes < need)
    return ofail(CE_EWORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? ws_bytes : (size_t)0);
  if ((uintptr_t)ws % 256u) return ofail(CE_EWORKSPACE, "workspace must be 256-byte aligned");
  vce::EmbedGradArgs a{};
  a.ids = m->ids;
  a.id_stride = m->id_stride;
  a.N = m->N;
  a.D = m->D;
  a.dout = static_cast<const char*>(dout);
  a.dout_ld = dout_ld;
  a.dtype = m->dtype;
  a.V = m->v_local;
  a.vocab_start = m->vocab_start;
  a.padding_idx = padding_idx;
  a.dw = dw;
  a.dw_ld = dw_ld;
  a.scale = m->scale;
  a.accumulate = accumulate;
  a.ws = static_cast<char*>(ws);
  return launched(vce::launch_embed_grad(a, stream), "embedding gradient launch");
}

ce_status ce_rms_norm(const ce_norm* n, void* y, int64_t y_ld, void* sum, int64_t sum_ld, hipStream_t stream) {
  ce_status st;
  if ((st = check_norm(n)) || (st = check_rows("y", y, n->dtype, n->N, n->D, y_ld))) return st;
  return norm(n, y, y_ld, nullptr, 0, 0, nullptr, sum, sum_ld, stream);
}

ce_status ce_rms_norm_quant(const ce_norm* n, void* q, int64_t q_ld, int32_t group, float* scales, void* sum,
                            int64_t sum_ld, hipStream_t stream) {
  ce_status st;
  if ((st = check_norm(n))) return st;
  if (group != 0 && group != 32 && group != 64 && group != 128)
    return ofail(CE_EINVAL, "group %d is not 0 (a row), 32, 64 or 128", group);
  if (n->N > 0 && (!q || !scales)) return ofail(CE_EINVAL, "q or scales is NULL");
  if (q_ld < n->D) return ofail(CE_ELAYOUT, "the row stride of q must be >= %lld (got %lld)", (long long)n->D, (long long)q_ld);
  if ((uintptr_t)scales % 4u) return ofail(CE_ELAYOUT, "scales is not 4-byte aligned");
  return norm(n, nullptr, 0, q, q_ld, group, scales, sum, sum_ld, stream);
}

size_t ce_rms_norm_workspace_bytes(int64_t N, int64_t D) {
  if (N < 0 || N > kMax31 || D < 1 || D > vce::kNormMaxCols) {
    ofail(CE_EINVAL, "need 0 <= N < 2^31 and 1 <= D <= %lld (got %lld, %lld)", (long long)vce::kNormMaxCols,
          (long long)N, (long long)D);
    return 0;
  }
  const size_t b = vce::norm_grad_workspace(N, D);
  return b < 256 ? 256 : b;
}

ce_status ce_rms_norm_backward(const ce_norm* n, const void* dy, int64_t dy_ld, const void* dsum, int64_t dsum_ld,
                               void* dx, int64_t dx_ld, float* dweight, int32_t accumulate, void* ws, size_t ws_bytes,
                               hipStream_t stream) {
  ce_status st;
  if ((st = check_norm(n)) || (st = check_rows("dy", dy, n->dtype, n->N, n->D, dy_ld))) return st;
  if (n->residual) return ofail(CE_EINVAL, "the gradient takes the forward's sum as x and no residual");
  if (dsum && (st = check_rows("dsum", dsum, n->dtype, n->N, n->D, dsum_ld))) return st;
  if (dx && (st = check_rows("dx", dx, n->dtype, n->N, n->D, dx_ld))) return st;
  if ((uintptr_t)dweight % 4u) return ofail(CE_ELAYOUT, "dweight is not 4-byte aligned");
  if (accumulate != 0 && accumulate != 1) return ofail(CE_EINVAL, "accumulate must be 0 or 1");
  if (dweight) {
    const size_t need = vce::norm_grad_workspace(n->N, n->D);
    if (need > 0 && (!ws || ws_bytes < need))
      return ofail(CE_EWORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? ws_bytes : (size_t)0);
    if ((uintptr_t)ws % 256u) return ofail(CE_EWORKSPACE, "workspace must be 256-byte aligned");
  }
  if (dx) {
    const int eb = elem_bytes(n->dtype);
    const auto rows = [n, eb](const void* p, int64_t ld) { return row_set(p, n->N, 1, ld, 0, n->D, eb); };
    const RowSet ds = rows(dx, dx_ld);
    if (rows_meet(ds, rows(n->x, n->x_ld), true)) return overlap("dx", "x");
    if (rows_meet(ds, rows(dy, dy_ld), true)) return overlap("dx", "dy");
    if (dsum && rows_meet(ds, rows(dsum, dsum_ld), true)) return overlap("dx", "dsum");
  }
  vce::NormGradArgs a{};
  a.s = static_cast<const char*>(n->x);
  a.dy = static_cast<const char*>(dy);
  a.dsum = static_cast<const char*>(dsum);
  a.weight = static_cast<const char*>(n->weight);
  a.dtype = n->dtype;
  a.wdtype = n->weight_dtype;
  a.N = n->N;
  a.D = n->D;
  a.s_ld = n->x_ld;
  a.dy_ld = dy_ld;
  a.dsum_ld = dsum_ld;
  a.eps = n->eps;
  a.dx = static_cast<char*>(dx);
  a.dx_ld = dx_ld;
  a.dweight = dweight;
  a.accumulate = accumulate;
  a.parts = static_cast<float*>(ws);
  return launched(vce::launch_norm_grad(a, stream), "norm gradient launch");
}

}  // extern "C"
