// kv_api.hip -- extern "C" entry points of the operators on a paged cache
// (declared, with their argument contracts, in include/splitzip.h): the
// checks that need no device access, and the rotation's frequencies.
#include "splitzip.h"
#include "kv_internal.h"

#include <cmath>

namespace {

constexpr uint64_t kMaxHeads = 65535;
constexpr uint64_t kMaxStride = uint64_t{1} << 32;
constexpr uint64_t kMaxTokens = (uint64_t{1} << 31) - 1;
constexpr uint64_t kMaxSeqs = 65535;
// A block of 16 cached tokens is addressed by 31-bit byte offsets.
constexpr uint64_t kMaxPageStride = uint64_t{1} << 26;
constexpr uint64_t kMaxLen = uint64_t{1} << 30;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

sz_status hip_status(hipError_t e) { return e == hipSuccess ? SZ_OK : SZ_ERR_HIP; }

// A launch goes to the current device; a stream of another one is refused.
sz_status check_stream(hipStream_t stream) {
    int current = 0;
    hipDevice_t of = 0;
    if (hipGetDevice(&current) != hipSuccess) return SZ_ERR_HIP;
    if (stream == nullptr || stream == hipStreamPerThread) return SZ_OK;
    if (hipStreamGetDevice(stream, &of) != hipSuccess) return SZ_ERR_HIP;
    return (int)of == current ? SZ_OK : SZ_ERR_INVALID_ARGUMENT;
}

bool head_dim_ok(uint64_t d) { return d >= 8 && d <= 256 && d % 8 == 0; }

bool strides_ok(uint64_t token_stride, uint64_t head_stride) {
    return token_stride % 8 == 0 && head_stride % 8 == 0 && token_stride < kMaxStride &&
           head_stride < kMaxStride;
}

// Rows of `dim` elements that do not overlap: tokens of heads, or heads of
// tokens.
bool rows_apart(uint64_t tokens, uint64_t heads, uint64_t token_stride, uint64_t head_stride,
                uint64_t dim) {
    if (tokens > 1 && token_stride < dim) return false;
    if (heads > 1 && head_stride < dim) return false;
    if (tokens <= 1 || heads <= 1) return true;
    return token_stride >= (heads - 1) * head_stride + dim ||
           head_stride >= (tokens - 1) * token_stride + dim;
}

uint64_t size_of(uint32_t type) { return type == SZ_TYPE_F32 ? 4 : 2; }

bool heads_ok(const sz_heads* t, uint64_t tokens, uint64_t dim, bool written) {
    if (t == nullptr || (t->type != SZ_TYPE_BF16 && t->type != SZ_TYPE_F32)) return false;
    if (t->heads == 0 || t->heads > kMaxHeads || !strides_ok(t->token_stride, t->head_stride))
        return false;
    if (tokens > 0 && (t->data == nullptr || !aligned(t->data, 16))) return false;
    return !written || rows_apart(tokens, t->heads, t->token_stride, t->head_stride, dim);
}

// The bytes that a tensor spans
struct Span {
    uintptr_t begin, end;
};
Span span(const sz_heads& t, uint64_t tokens, uint64_t dim) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(t.data);
    if (tokens == 0) return {at, at};
    return {at, at + ((tokens - 1) * t.token_stride + (t.heads - 1) * t.head_stride + dim) *
                         size_of(t.type)};
}

// Whether a call that writes b may have a beside it: apart, in place (the
// caller says whether that is allowed), or slices of the same tokens or heads.
bool apart(const sz_heads& a, const sz_heads& b, uint64_t tokens, uint64_t dim, bool in_place) {
    const Span x = span(a, tokens, dim), y = span(b, tokens, dim);
    if (x.end <= y.begin || y.end <= x.begin) return true;
    if (in_place && a.data == b.data && a.type == b.type && a.heads == b.heads &&
        a.token_stride == b.token_stride && a.head_stride == b.head_stride)
        return true;
    // the same step from token to token in bytes, and within a step the one
    // before the other
    const uint64_t step = a.token_stride * size_of(a.type);
    if (step == 0 || step != b.token_stride * size_of(b.type)) return false;
    const uint64_t a_bytes = ((a.heads - 1) * a.head_stride + dim) * size_of(a.type);
    const uint64_t b_bytes = ((b.heads - 1) * b.head_stride + dim) * size_of(b.type);
    const uint64_t ahead = x.begin <= y.begin ? (y.begin - x.begin) % step
                                              : (step - (x.begin - y.begin) % step) % step;
    if (ahead >= a_bytes && ahead + b_bytes <= step) return true;
    // or the same step from head to head too, within which the one is before
    // the other (slices of every head of a fused tensor), where a token's
    // heads line up with the next one's or do not reach it
    const uint64_t head = a.head_stride * size_of(a.type);
    if (head == 0 || head != b.head_stride * size_of(b.type)) return false;
    const uint64_t in_head = ahead % head;
    return in_head >= dim * size_of(a.type) && in_head + dim * size_of(b.type) <= head &&
           (step % head == 0 || (a_bytes <= step && ahead + b_bytes <= step));
}

bool overlap(const void* p, uint64_t bytes, Span s) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    return bytes > 0 && at < s.end && s.begin < at + bytes;
}

sz::Rows rows_of(const sz_heads* t) {
    if (t == nullptr) return sz::Rows{};
    return sz::Rows{t->data, t->token_stride, t->head_stride, (uint32_t)t->heads,
                    t->type == SZ_TYPE_F32};
}

bool cache_ok(const sz_kv_cache* c) {
    if (c == nullptr || c->d_k_pages == nullptr || c->d_v_pages == nullptr ||
        !aligned(c->d_k_pages, 8) || !aligned(c->d_v_pages, 8))
        return false;
    if (!head_dim_ok(c->head_dim) || c->kv_heads == 0 || c->kv_heads > kMaxHeads) return false;
    if (c->page_tokens < 16 || c->page_tokens > 65536 ||
        (c->page_tokens & (c->page_tokens - 1)) != 0)
        return false;
    if (c->pages_per_seq == 0 || c->pages_per_seq > kMaxTokens ||
        c->table_pitch < c->pages_per_seq || c->table_pitch > (uint64_t{1} << 40))
        return false;
    return strides_ok(c->token_stride, c->head_stride) && c->token_stride < kMaxPageStride &&
           rows_apart(c->page_tokens, c->kv_heads, c->token_stride, c->head_stride, c->head_dim);
}

sz::Cache cache_of(const sz_kv_cache& c) {
    uint32_t lg = 0;
    while ((1u << lg) < c.page_tokens) lg++;
    return sz::Cache{reinterpret_cast<const uint64_t*>(c.d_k_pages),
                     reinterpret_cast<const uint64_t*>(c.d_v_pages),
                     c.pages_per_seq, c.table_pitch, c.token_stride, c.head_stride,
                     c.kv_heads, c.head_dim, lg};
}

bool batch_ok(const sz_batch* b) {
    if (b == nullptr || b->n_seqs > kMaxSeqs || b->n_tokens > kMaxTokens) return false;
    return b->n_seqs == 0 || (b->d_starts != nullptr && b->d_lens != nullptr &&
                              aligned(b->d_starts, 4) && aligned(b->d_lens, 4));
}

sz::Batch batch_of(const sz_batch& b) {
    return sz::Batch{b.d_starts, b.d_lens, (uint32_t)b.n_seqs, (uint32_t)b.n_tokens};
}

bool rope_ok(const sz_rope* r, uint64_t dim) {
    if (r == nullptr || r->rotary_dim == 0) return true;
    return r->rotary_dim % 8 == 0 && r->rotary_dim <= dim && r->interleaved <= 1 &&
           r->d_phases != nullptr && aligned(r->d_phases, 8) && std::isfinite(r->magnitude);
}

sz::Turn turn_of(const sz_rope* r) {
    if (r == nullptr || r->rotary_dim == 0) return sz::Turn{nullptr, 0, 0, 1.0f};
    return sz::Turn{r->d_phases, r->rotary_dim, r->interleaved, r->magnitude};
}

// Source and destination of one of the turned tensors
bool turned_ok(const sz_heads* src, const sz_heads* dst, const float* weight, uint64_t tokens,
               uint64_t dim) {
    return heads_ok(src, tokens, dim, false) && heads_ok(dst, tokens, dim, true) &&
           dst->type == SZ_TYPE_BF16 && dst->heads == src->heads && aligned(weight, 16) &&
           apart(*src, *dst, tokens, dim, true);
}

uint64_t most_len(const sz_kv_cache& c) {
    const uint64_t n = c.pages_per_seq * c.page_tokens;
    return n > kMaxLen ? kMaxLen : n;
}

// Attention counts a call's rows in 31 bits, and a launch has fewer than 2^32
// threads: 256 for a tile of a KV head, rows / 16 + n_seqs of them where rows
// <= 16 n_seqs, rows / 128 + n_seqs otherwise.
bool attend_fits(uint64_t n_seqs, uint64_t n_tokens, uint64_t q_heads, uint64_t kv_heads) {
    return n_tokens * q_heads <= kMaxTokens &&
           n_tokens * q_heads / 128 + 2 * n_seqs * kv_heads < uint64_t{1} << 24;
}

}  // namespace

extern "C" {

sz_status sz_rope_frequencies(uint32_t rotary_dim, double base, int stretch, double factor,
                              double original_len, double slow, double fast, double* inv_freq,
                              float* magnitude) {
    if (rotary_dim == 0 || rotary_dim % 2 != 0 || inv_freq == nullptr || magnitude == nullptr ||
        !std::isfinite(base) || base <= 1 || stretch < SZ_ROPE_PLAIN || stretch > SZ_ROPE_BANDS)
        return SZ_ERR_INVALID_ARGUMENT;
    const double dims = rotary_dim, pi = 3.14159265358979323846;
    const bool blends = stretch == SZ_ROPE_RAMP || stretch == SZ_ROPE_BANDS;
    if (stretch != SZ_ROPE_PLAIN && !(std::isfinite(factor) && factor >= 1))
        return SZ_ERR_INVALID_ARGUMENT;
    if (blends && !(std::isfinite(original_len) && original_len >= 1 && slow > 0 && fast > slow &&
                    std::isfinite(fast)))
        return SZ_ERR_INVALID_ARGUMENT;
    if (stretch == SZ_ROPE_BASE) {
        if (rotary_dim <= 2) return SZ_ERR_INVALID_ARGUMENT;
        base *= std::pow(factor, dims / (dims - 2));
    }
    // RAMP: the pairs between which the frequencies blend
    double first = 0, last = 0;
    if (stretch == SZ_ROPE_RAMP) {
        const auto pair_of = [&](double turns) {
            return dims * std::log(original_len / (2 * pi * turns)) / (2 * std::log(base));
        };
        first = std::fmax(std::floor(pair_of(fast)), 0.0);
        last = std::fmin(std::ceil(pair_of(slow)), dims - 1);
        if (last <= first) last = first + 1e-3;
    }
    for (uint32_t i = 0; i < rotary_dim / 2; i++) {
        double f = std::pow(base, -2.0 * i / dims);
        double kept = 1;  // the share of f that is not stretched
        if (stretch == SZ_ROPE_LINEAR) kept = 0;
        if (stretch == SZ_ROPE_RAMP) kept = 1 - (i - first) / (last - first);
        if (stretch == SZ_ROPE_BANDS)
            kept = (original_len * f / (2 * pi) - slow) / (fast - slow);
        kept = std::fmin(std::fmax(kept, 0.0), 1.0);
        if (stretch == SZ_ROPE_LINEAR || blends) f = kept * f + (1 - kept) * f / factor;
        inv_freq[i] = f;
    }
    *magnitude = stretch == SZ_ROPE_RAMP ? (float)(0.1 * std::log(factor) + 1) : 1.0f;
    return SZ_OK;
}

sz_status sz_rope_phases(const double* inv_freq, uint64_t n, uint64_t* phases) {
    if (n > 0 && (inv_freq == nullptr || phases == nullptr)) return SZ_ERR_INVALID_ARGUMENT;
    for (uint64_t i = 0; i < n; i++)
        if (!std::isfinite(inv_freq[i])) return SZ_ERR_INVALID_ARGUMENT;
    for (uint64_t i = 0; i < n; i++) {
        // long double has the 64 bits of the fraction
        long double t = (long double)inv_freq[i] / 6.283185307179586476925286766559005768L;
        t -= floorl(t);
        const long double units = rintl(t * 18446744073709551616.0L);
        phases[i] = units >= 18446744073709551616.0L ? 0 : (uint64_t)units;
    }
    return SZ_OK;
}

sz_status sz_qk_norm_rope(const sz_heads* q, const sz_heads* q_out, const float* d_q_weight,
                          const sz_heads* k, const sz_heads* k_out, const float* d_k_weight,
                          uint32_t head_dim, uint64_t n_tokens, const int32_t* d_positions,
                          float eps, const sz_rope* rope, hipStream_t stream) {
    if (!head_dim_ok(head_dim) || n_tokens > kMaxTokens || !rope_ok(rope, head_dim))
        return SZ_ERR_INVALID_ARGUMENT;
    if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr) ||
        (q == nullptr && k == nullptr))
        return SZ_ERR_INVALID_ARGUMENT;
    if (q != nullptr && !turned_ok(q, q_out, d_q_weight, n_tokens, head_dim))
        return SZ_ERR_INVALID_ARGUMENT;
    if (k != nullptr && !turned_ok(k, k_out, d_k_weight, n_tokens, head_dim))
        return SZ_ERR_INVALID_ARGUMENT;
    if (q != nullptr && k != nullptr &&
        !(apart(*q, *k_out, n_tokens, head_dim, false) &&
          apart(*k, *q_out, n_tokens, head_dim, false) &&
          apart(*q_out, *k_out, n_tokens, head_dim, false)))
        return SZ_ERR_INVALID_ARGUMENT;
    if (!(eps >= 0) || !std::isfinite(eps)) return SZ_ERR_INVALID_ARGUMENT;
    const sz::Turn turn = turn_of(rope);
    if (n_tokens > 0 && turn.dims > 0 && (d_positions == nullptr || !aligned(d_positions, 4)))
        return SZ_ERR_INVALID_ARGUMENT;
    if (n_tokens == 0) return SZ_OK;
    if (sz_status s = check_stream(stream)) return s;
    const sz::TurnRows a{rows_of(q), rows_of(q_out), rows_of(k), rows_of(k_out), sz::Rows{},
                         d_q_weight, d_k_weight, d_positions, turn, eps, head_dim,
                         (uint32_t)n_tokens};
    return hip_status(sz::launch_turn(a, stream));
}

sz_status sz_kv_append(const sz_heads* k, const sz_heads* v, const float* d_k_weight,
                       const sz_heads* q, const sz_heads* q_out, const float* d_q_weight,
                       float eps, const sz_rope* rope, const int32_t* d_positions,
                       const sz_kv_cache* cache, const sz_batch* batch, int32_t* d_status,
                       hipStream_t stream) {
    if (!cache_ok(cache) || !batch_ok(batch) || !rope_ok(rope, cache->head_dim))
        return SZ_ERR_INVALID_ARGUMENT;
    const uint64_t n = batch->n_tokens;
    const uint32_t dim = cache->head_dim;
    if (!heads_ok(k, n, dim, false) || !heads_ok(v, n, dim, false) ||
        k->heads != cache->kv_heads || v->heads != cache->kv_heads || !aligned(d_k_weight, 16))
        return SZ_ERR_INVALID_ARGUMENT;
    if ((q == nullptr) != (q_out == nullptr)) return SZ_ERR_INVALID_ARGUMENT;
    if (q != nullptr &&
        !(turned_ok(q, q_out, d_q_weight, n, dim) && apart(*k, *q_out, n, dim, false) &&
          apart(*v, *q_out, n, dim, false)))
        return SZ_ERR_INVALID_ARGUMENT;
    if (!(eps >= 0) || !std::isfinite(eps) || !aligned(d_positions, 4) || !aligned(d_status, 4))
        return SZ_ERR_INVALID_ARGUMENT;
    if (batch->n_seqs == 0 || (n == 0 && d_status == nullptr)) return SZ_OK;
    if (sz_status s = check_stream(stream)) return s;
    const sz::Cache c = cache_of(*cache);
    const sz::Batch b = batch_of(*batch);
    const sz::TurnRows a{rows_of(q), rows_of(q_out), rows_of(k), sz::Rows{}, rows_of(v),
                         d_q_weight, d_k_weight, d_positions, turn_of(rope), eps, dim,
                         (uint32_t)n};
    sz_status st = hip_status(sz::launch_append(a, c, b, stream));
    if (st == SZ_OK && d_status != nullptr)
        st = hip_status(sz::launch_check_seqs(
            sz::SeqCheck{c, b, (int64_t)most_len(*cache), 1, 1, 0, d_status}, stream));
    return st;
}

uint64_t sz_attend_workspace_size(uint64_t q_heads, const sz_kv_cache* cache,
                                  const sz_batch* batch, uint64_t max_len) {
    if (cache == nullptr || batch == nullptr || !head_dim_ok(cache->head_dim) ||
        cache->kv_heads == 0 || cache->kv_heads > kMaxHeads || q_heads == 0 ||
        q_heads > kMaxHeads || q_heads % cache->kv_heads != 0 || batch->n_seqs > kMaxSeqs ||
        batch->n_tokens > kMaxTokens || cache->pages_per_seq == 0 ||
        cache->pages_per_seq > kMaxTokens || cache->page_tokens > 65536)
        return 0;
    const uint64_t most = most_len(*cache);
    if (!attend_fits(batch->n_seqs, batch->n_tokens, q_heads, cache->kv_heads)) return 0;
    if (batch->n_seqs == 0 || batch->n_tokens == 0) return 0;
    return sz::attend_workspace((uint32_t)q_heads, cache_of(*cache), batch->n_seqs,
                                batch->n_tokens,
                                max_len == 0 || max_len > most ? most : max_len);
}

sz_status sz_attend_pages(const sz_heads* q, const sz_heads* out, float* d_lse,
                          const sz_kv_cache* cache, const sz_batch* batch, uint64_t max_len,
                          float scale, float softcap, int causal, uint64_t window,
                          void* d_workspace, uint64_t workspace_bytes, int32_t* d_status,
                          hipStream_t stream) {
    if (!cache_ok(cache) || !batch_ok(batch)) return SZ_ERR_INVALID_ARGUMENT;
    const uint64_t n = batch->n_tokens;
    const uint32_t dim = cache->head_dim;
    if (!heads_ok(q, n, dim, false) || !heads_ok(out, n, dim, true) || q->type != SZ_TYPE_BF16 ||
        q->heads != out->heads || q->heads % cache->kv_heads != 0 ||
        !attend_fits(batch->n_seqs, n, q->heads, cache->kv_heads) ||
        !apart(*q, *out, n, dim, false))
        return SZ_ERR_INVALID_ARGUMENT;
    // (the kernels multiply by scale log2 e, or 2 scale log2 e / softcap)
    if (!(scale > 0 && scale < 1e38f) || !(softcap >= 0 && softcap < 1e38f) ||
        (softcap > 0 && !(scale / softcap < 0.99e38f)) ||
        (window != 0 && !causal) || !aligned(d_lse, 4) || !aligned(d_status, 4))
        return SZ_ERR_INVALID_ARGUMENT;
    const uint64_t most = most_len(*cache);
    if (max_len == 0 || max_len > most) max_len = most;
    if (window > kMaxLen) window = 0;  // (it hides nothing; the kernels count in 32 bits)
    if (overlap(d_lse, d_lse == nullptr ? 0 : 4 * n * q->heads, span(*q, n, dim)) ||
        overlap(d_lse, d_lse == nullptr ? 0 : 4 * n * q->heads, span(*out, n, dim)))
        return SZ_ERR_INVALID_ARGUMENT;
    const uint64_t need = sz_attend_workspace_size(q->heads, cache, batch, max_len);
    if (need > 0 && (d_workspace == nullptr || !aligned(d_workspace, 256) ||
                     workspace_bytes < need || overlap(d_workspace, need, span(*q, n, dim)) ||
                     overlap(d_workspace, need, span(*out, n, dim))))
        return SZ_ERR_INVALID_ARGUMENT;
    if (batch->n_seqs == 0 || (n == 0 && d_status == nullptr)) return SZ_OK;
    if (sz_status s = check_stream(stream)) return s;
    const sz::Attend a{rows_of(q), rows_of(out), d_lse, cache_of(*cache), batch_of(*batch),
                       (int64_t)max_len, scale, softcap, causal != 0, window};
    sz_status st = hip_status(sz::launch_attend(a, static_cast<uint8_t*>(d_workspace), stream));
    if (st == SZ_OK && d_status != nullptr)
        st = hip_status(sz::launch_check_seqs(
            sz::SeqCheck{a.cache, a.batch, a.max_len, 0, a.causal, window, d_status}, stream));
    return st;
}

}  // extern "C"
