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
bool apart(const sz_heads& a, uint64_t a_dim, const sz_heads& b, uint64_t b_dim, uint64_t tokens,
           bool in_place) {
    const Span x = span(a, tokens, a_dim), y = span(b, tokens, b_dim);
    if (x.end <= y.begin || y.end <= x.begin) return true;
    if (in_place && a.data == b.data && a.type == b.type && a.heads == b.heads &&
        a.token_stride == b.token_stride && a.head_stride == b.head_stride)
        return true;
    // the same step from token to token in bytes, and within a step the one
    // before the other
    const uint64_t step = a.token_stride * size_of(a.type);
    if (step == 0 || step != b.token_stride * size_of(b.type)) return false;
    const uint64_t a_bytes = ((a.heads - 1) * a.head_stride + a_dim) * size_of(a.type);
    const uint64_t b_bytes = ((b.heads - 1) * b.head_stride + b_dim) * size_of(b.type);
    const uint64_t ahead = x.begin <= y.begin ? (y.begin - x.begin) % step
                                              : (step - (x.begin - y.begin) % step) % step;
    if (ahead >= a_bytes && ahead + b_bytes <= step) return true;
    // or the same step from head to head too, within which the one is before
    // the other (slices of every head of a fused tensor), where a token's
    // heads line up with the next one's or do not reach it
    const uint64_t head = a.head_stride * size_of(a.type);
    if (head == 0 || head != b.head_stride * size_of(b.type)) return false;
    const uint64_t in_head = ahead % head;
    return in_head >= a_dim * size_of(a.type) && in_head + b_dim * size_of(b.type) <= head &&
           (step % head == 0 || (a_bytes <= step && ahead + b_bytes <= step));
}
bool apart(const sz_heads& a, const sz_heads& b, uint64_t tokens, uint64_t dim, bool in_place) {
    return apart(a, dim, b, dim, tokens, in_place);
}

bool overlap(const void* p, uint64_t bytes, Span s) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    return bytes > 0 && at < s.end && s.begin < at + bytes;
}

Span span_of(const void* p, uint64_t bytes) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    return {at, at + bytes};
}

sz::Rows rows_of(const sz_heads* t) {
    if (t == nullptr) return sz::Rows{};
    return sz::Rows{t->data, t->token_stride, t->head_stride, (uint32_t)t->heads,
                    t->type == SZ_TYPE_F32};
}

bool table_ok(uint64_t pages_per_seq, uint64_t table_pitch, uint32_t page_tokens) {
    if (page_tokens < 16 || page_tokens > 65536 || (page_tokens & (page_tokens - 1)) != 0)
        return false;
    return pages_per_seq > 0 && pages_per_seq <= kMaxTokens && table_pitch >= pages_per_seq &&
           table_pitch <= (uint64_t{1} << 40);
}

bool cache_ok(const sz_kv_cache* c) {
    if (c == nullptr || c->d_k_pages == nullptr || c->d_v_pages == nullptr ||
        !aligned(c->d_k_pages, 8) || !aligned(c->d_v_pages, 8))
        return false;
    if (!head_dim_ok(c->head_dim) || c->kv_heads == 0 || c->kv_heads > kMaxHeads ||
        !table_ok(c->pages_per_seq, c->table_pitch, c->page_tokens))
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

bool latent_dims_ok(uint64_t latent, uint64_t rotary) {
    return latent >= 8 && latent <= 512 && latent % 8 == 0 && rotary <= 64 && rotary % 8 == 0;
}

bool latent_ok(const sz_latent_cache* c) {
    if (c == nullptr || c->d_pages == nullptr || !aligned(c->d_pages, 8) ||
        !latent_dims_ok(c->latent_dim, c->rotary_dim) ||
        !table_ok(c->pages_per_seq, c->table_pitch, c->page_tokens))
        return false;
    return c->token_stride % 8 == 0 && c->token_stride < kMaxPageStride &&
           c->token_stride >= c->latent_dim + c->rotary_dim;
}

// A cache of one head, whose keys and values are the same rows
sz_kv_cache rows_of(const sz_latent_cache& c) {
    return sz_kv_cache{c.d_pages, c.d_pages, c.pages_per_seq, c.table_pitch, c.token_stride, 0, 1,
                       c.latent_dim + c.rotary_dim, c.page_tokens};
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

// (a tile of 128 rows of latent attention is two workgroups', in groups of eight)
bool latent_fits(uint64_t n_seqs, uint64_t n_tokens, uint64_t heads) {
    return 2 * n_tokens * heads <= kMaxTokens &&
           n_tokens * heads / 64 + 2 * n_seqs < (uint64_t{1} << 24) - 16;
}

bool expanded_dim_ok(uint64_t d) { return d >= 8 && d <= 128 && d % 8 == 0; }

bool spans_meet(Span a, Span b) {
    return a.begin < a.end && b.begin < b.end && a.begin < b.end && b.begin < a.end;
}

// (the kernels multiply by scale log2 e, or 2 scale log2 e / softcap)
bool score_ok(float scale, float softcap, int causal, uint64_t window) {
    return scale > 0 && scale < 1e38f && softcap >= 0 && softcap < 1e38f &&
           !(softcap > 0 && !(scale / softcap < 0.99e38f)) && !(window != 0 && !causal);
}

bool weigh_sizes_ok(uint64_t q_heads, const sz_kv_cache* c, const sz_batch* b) {
    return c != nullptr && b != nullptr && head_dim_ok(c->head_dim) && c->kv_heads > 0 &&
           c->kv_heads <= kMaxHeads && q_heads > 0 && q_heads <= kMaxHeads &&
           q_heads % c->kv_heads == 0 && b->n_seqs <= kMaxSeqs && b->n_tokens <= kMaxTokens &&
           table_ok(c->pages_per_seq, c->table_pitch, c->page_tokens) &&
           attend_fits(b->n_seqs, b->n_tokens, q_heads, c->kv_heads);
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
    if (!score_ok(scale, softcap, causal, window) || !aligned(d_lse, 4) || !aligned(d_status, 4))
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
                       (int64_t)max_len, scale, softcap, causal != 0, window, dim};
    sz_status st = hip_status(sz::launch_attend(a, static_cast<uint8_t*>(d_workspace), stream));
    if (st == SZ_OK && d_status != nullptr)
        st = hip_status(sz::launch_check_seqs(
            sz::SeqCheck{a.cache, a.batch, a.max_len, 0, a.causal, window, d_status}, stream));
    return st;
}

sz_status sz_latent_append(const sz_heads* latent, const float* d_weight, float eps,
                           const sz_heads* k_rotary, const sz_heads* q, const sz_heads* q_out,
                           const sz_rope* rope, const int32_t* d_positions,
                           const sz_latent_cache* cache, const sz_batch* batch,
                           int32_t* d_status, hipStream_t stream) {
    if (!latent_ok(cache) || !batch_ok(batch)) return SZ_ERR_INVALID_ARGUMENT;
    const uint64_t n = batch->n_tokens;
    const uint32_t dim = cache->latent_dim, rotary = cache->rotary_dim;
    if (!rope_ok(rope, rotary) ||
        (rope != nullptr && rope->rotary_dim != 0 && rope->rotary_dim != rotary) ||
        !heads_ok(latent, n, dim, false) || latent->heads != 1 || !aligned(d_weight, 16))
        return SZ_ERR_INVALID_ARGUMENT;
    if ((k_rotary == nullptr) != (rotary == 0) || (q == nullptr) != (q_out == nullptr) ||
        (q != nullptr && rotary == 0))
        return SZ_ERR_INVALID_ARGUMENT;
    if (k_rotary != nullptr && (!heads_ok(k_rotary, n, rotary, false) || k_rotary->heads != 1))
        return SZ_ERR_INVALID_ARGUMENT;
    if (q != nullptr && !(turned_ok(q, q_out, nullptr, n, rotary) &&
                          apart(*latent, dim, *q_out, rotary, n, false) &&
                          apart(*k_rotary, *q_out, n, rotary, false)))
        return SZ_ERR_INVALID_ARGUMENT;
    if (!(eps >= 0) || !std::isfinite(eps) || !aligned(d_positions, 4) || !aligned(d_status, 4))
        return SZ_ERR_INVALID_ARGUMENT;
    if (batch->n_seqs == 0 || (n == 0 && d_status == nullptr)) return SZ_OK;
    if (sz_status s = check_stream(stream)) return s;
    const sz_kv_cache rows = rows_of(*cache);
    const sz::Cache c = cache_of(rows);
    const sz::Batch b = batch_of(*batch);
    const sz::LatentRows a{rows_of(latent), rows_of(k_rotary), rows_of(q), rows_of(q_out),
                           d_weight, d_positions, turn_of(rope), eps, dim, rotary, (uint32_t)n};
    sz_status st = hip_status(sz::launch_latent_append(a, c, b, stream));
    if (st == SZ_OK && d_status != nullptr)
        st = hip_status(sz::launch_check_seqs(
            sz::SeqCheck{c, b, (int64_t)most_len(rows), 1, 1, 0, d_status}, stream));
    return st;
}

uint64_t sz_attend_latent_workspace_size(uint64_t heads, const sz_latent_cache* cache,
                                         const sz_batch* batch, uint64_t max_len) {
    if (cache == nullptr || batch == nullptr ||
        !latent_dims_ok(cache->latent_dim, cache->rotary_dim) || heads == 0 || heads > kMaxHeads ||
        !table_ok(cache->pages_per_seq, cache->table_pitch, cache->page_tokens) ||
        batch->n_seqs > kMaxSeqs || batch->n_tokens > kMaxTokens ||
        !latent_fits(batch->n_seqs, batch->n_tokens, heads) || batch->n_seqs == 0 ||
        batch->n_tokens == 0)
        return 0;
    const sz_kv_cache rows = rows_of(*cache);
    const uint64_t most = most_len(rows);
    return sz::attend_latent_workspace((uint32_t)heads, cache_of(rows), cache->latent_dim,
                                       batch->n_seqs, batch->n_tokens,
                                       max_len == 0 || max_len > most ? most : max_len);
}

sz_status sz_attend_latent(const sz_heads* q, const sz_heads* out, float* d_lse,
                           const sz_latent_cache* cache, const sz_batch* batch, uint64_t max_len,
                           float scale, int causal, void* d_workspace, uint64_t workspace_bytes,
                           int32_t* d_status, hipStream_t stream) {
    if (!latent_ok(cache) || !batch_ok(batch)) return SZ_ERR_INVALID_ARGUMENT;
    const sz_kv_cache rows = rows_of(*cache);
    const uint64_t n = batch->n_tokens;
    const uint32_t dim = rows.head_dim, value = cache->latent_dim;
    if (!heads_ok(q, n, dim, false) || !heads_ok(out, n, value, true) ||
        q->type != SZ_TYPE_BF16 || q->heads != out->heads ||
        !latent_fits(batch->n_seqs, n, q->heads) || !apart(*q, dim, *out, value, n, false))
        return SZ_ERR_INVALID_ARGUMENT;
    if (!(scale > 0 && scale < 1e38f) || !aligned(d_lse, 4) || !aligned(d_status, 4))
        return SZ_ERR_INVALID_ARGUMENT;
    const uint64_t most = most_len(rows);
    if (max_len == 0 || max_len > most) max_len = most;
    const uint64_t lse_bytes = d_lse == nullptr ? 0 : 4 * n * q->heads;
    if (overlap(d_lse, lse_bytes, span(*q, n, dim)) ||
        overlap(d_lse, lse_bytes, span(*out, n, value)))
        return SZ_ERR_INVALID_ARGUMENT;
    const uint64_t need = sz_attend_latent_workspace_size(q->heads, cache, batch, max_len);
    if (need > 0 && (d_workspace == nullptr || !aligned(d_workspace, 256) ||
                     workspace_bytes < need || overlap(d_workspace, need, span(*q, n, dim)) ||
                     overlap(d_workspace, need, span(*out, n, value)) ||
                     spans_meet(span_of(d_workspace, need), span_of(d_lse, lse_bytes))))
        return SZ_ERR_INVALID_ARGUMENT;
    if (batch->n_seqs == 0 || (n == 0 && d_status == nullptr)) return SZ_OK;
    if (sz_status s = check_stream(stream)) return s;
    const sz::Attend a{rows_of(q), rows_of(out), d_lse, cache_of(rows), batch_of(*batch),
                       (int64_t)max_len, scale, 0, causal != 0, 0, value};
    sz_status st =
        hip_status(sz::launch_attend_latent(a, static_cast<uint8_t*>(d_workspace), stream));
    if (st == SZ_OK && d_status != nullptr)
        st = hip_status(sz::launch_check_seqs(
            sz::SeqCheck{a.cache, a.batch, a.max_len, 0, a.causal, 0, d_status}, stream));
    return st;
}

uint64_t sz_attend_expanded_workspace_size(uint64_t heads, uint32_t value_dim,
                                           const sz_batch* batch, uint64_t max_len) {
    if (batch == nullptr || heads == 0 || heads > kMaxHeads || !expanded_dim_ok(value_dim) ||
        batch->n_seqs > kMaxSeqs || batch->n_tokens > kMaxTokens ||
        !attend_fits(batch->n_seqs, batch->n_tokens, heads, heads) || batch->n_seqs == 0 ||
        batch->n_tokens == 0)
        return 0;
    return sz::attend_expanded_workspace((uint32_t)heads, value_dim, batch->n_seqs,
                                         batch->n_tokens, max_len > kMaxLen ? kMaxLen : max_len);
}

sz_status sz_attend_expanded(const sz_heads* q, const sz_heads* out, float* d_lse,
                             const sz_heads* k, const sz_heads* k_rotary, const sz_heads* v,
                             uint32_t key_dim, uint32_t rotary_dim, uint32_t value_dim,
                             const int32_t* d_key_starts, uint64_t n_keys,
                             const sz_batch* batch, uint64_t max_len, float scale, int causal,
                             void* d_workspace, uint64_t workspace_bytes, int32_t* d_status,
                             hipStream_t stream) {
    if (!batch_ok(batch) || !expanded_dim_ok(key_dim) || !expanded_dim_ok(value_dim) ||
        rotary_dim > 64 || rotary_dim % 8 != 0 || n_keys > kMaxTokens)
        return SZ_ERR_INVALID_ARGUMENT;
    const uint64_t n = batch->n_tokens;
    const uint32_t dim = key_dim + rotary_dim;
    if (!heads_ok(q, n, dim, false) || !heads_ok(out, n, value_dim, true) ||
        q->type != SZ_TYPE_BF16 || q->heads != out->heads ||
        !attend_fits(batch->n_seqs, n, q->heads, q->heads) ||
        !apart(*q, dim, *out, value_dim, n, false))
        return SZ_ERR_INVALID_ARGUMENT;
    const auto keys_ok = [&](const sz_heads* x, uint32_t d) {
        return heads_ok(x, n_keys, d, false) && x->type == SZ_TYPE_BF16 &&
               x->token_stride < kMaxPageStride &&
               !spans_meet(span(*x, n_keys, d), span(*out, n, value_dim));
    };
    if (!keys_ok(k, key_dim) || !keys_ok(v, value_dim) || k->heads != q->heads ||
        v->heads != q->heads || (k_rotary == nullptr) != (rotary_dim == 0))
        return SZ_ERR_INVALID_ARGUMENT;
    if (k_rotary != nullptr && (!keys_ok(k_rotary, rotary_dim) ||
                                (k_rotary->heads != 1 && k_rotary->heads != q->heads)))
        return SZ_ERR_INVALID_ARGUMENT;
    if (!(scale > 0 && scale < 1e38f) || !aligned(d_lse, 4) || !aligned(d_status, 4) ||
        !aligned(d_key_starts, 4) || (batch->n_seqs > 0 && d_key_starts == nullptr))
        return SZ_ERR_INVALID_ARGUMENT;
    if (max_len == 0 || max_len > n_keys) max_len = n_keys;
    if (max_len > kMaxLen) max_len = kMaxLen;
    const uint64_t need =
        max_len == 0 ? 0 : sz_attend_expanded_workspace_size(q->heads, value_dim, batch, max_len);
    const Span lse = span_of(d_lse, d_lse == nullptr ? 0 : 4 * n * q->heads);
    const Span work = span_of(d_workspace, need);
    if (need > 0 && (d_workspace == nullptr || !aligned(d_workspace, 256) ||
                     workspace_bytes < need || spans_meet(work, lse)))
        return SZ_ERR_INVALID_ARGUMENT;
    const Span others[5] = {span(*q, n, dim), span(*out, n, value_dim), span(*k, n_keys, key_dim),
                            span(*v, n_keys, value_dim),
                            k_rotary == nullptr ? Span{0, 0} : span(*k_rotary, n_keys, rotary_dim)};
    for (const Span& x : others)
        if (spans_meet(lse, x) || spans_meet(work, x)) return SZ_ERR_INVALID_ARGUMENT;
    if (batch->n_seqs == 0 || (n == 0 && d_status == nullptr)) return SZ_OK;
    if (sz_status s = check_stream(stream)) return s;
    sz::Cache heads{};
    heads.kv_heads = (uint32_t)q->heads;
    heads.head_dim = value_dim;
    const sz::Attend a{rows_of(q), rows_of(out), d_lse, heads, batch_of(*batch), (int64_t)max_len,
                       scale, 0, causal != 0, 0, value_dim};
    const sz::Expanded e{rows_of(k), rows_of(k_rotary), rows_of(v), key_dim, rotary_dim, value_dim,
                         d_key_starts, (int64_t)n_keys};
    sz_status st =
        hip_status(sz::launch_attend_expanded(a, e, static_cast<uint8_t*>(d_workspace), stream));
    if (st == SZ_OK && d_status != nullptr)
        st = hip_status(sz::launch_check_seqs(
            sz::SeqCheck{heads, a.batch, a.max_len, 0, a.causal, 0, d_status, d_key_starts,
                         (int64_t)n_keys}, stream));
    return st;
}

uint64_t sz_weigh_workspace_size(uint64_t q_heads, const sz_kv_cache* cache,
                                 const sz_batch* batch, uint64_t max_len) {
    if (!weigh_sizes_ok(q_heads, cache, batch) || batch->n_seqs == 0) return 0;
    const uint64_t most = most_len(*cache);
    return sz::weigh_workspace((uint32_t)q_heads, cache_of(*cache), batch->n_seqs,
                               batch->n_tokens, max_len == 0 || max_len > most ? most : max_len);
}

sz_status sz_weigh_pages(const sz_heads* q, const float* d_lse, const float* d_before,
                         float* d_weights, uint64_t weights_pitch, float keep,
                         const sz_kv_cache* cache, const sz_batch* batch, uint64_t max_len,
                         float scale, float softcap, int causal, uint64_t window,
                         void* d_workspace, uint64_t workspace_bytes, int32_t* d_status,
                         hipStream_t stream) {
    if (!cache_ok(cache) || !batch_ok(batch)) return SZ_ERR_INVALID_ARGUMENT;
    const uint64_t n = batch->n_tokens;
    const uint32_t dim = cache->head_dim;
    if (!heads_ok(q, n, dim, false) || q->type != SZ_TYPE_BF16 ||
        !weigh_sizes_ok(q->heads, cache, batch))
        return SZ_ERR_INVALID_ARGUMENT;
    if (!score_ok(scale, softcap, causal, window) || !std::isfinite(keep) || !aligned(d_lse, 4) ||
        !aligned(d_before, 4) || !aligned(d_weights, 4) || !aligned(d_status, 4))
        return SZ_ERR_INVALID_ARGUMENT;
    const uint64_t most = most_len(*cache);
    if (max_len == 0 || max_len > most) max_len = most;
    if (window > kMaxLen) window = 0;
    if (weights_pitch < max_len || weights_pitch > kMaxTokens) return SZ_ERR_INVALID_ARGUMENT;
    if (keep == 0) d_before = nullptr;
    const uint64_t bytes = 4 * batch->n_seqs * cache->kv_heads * weights_pitch;
    const uint64_t need = sz_weigh_workspace_size(q->heads, cache, batch, max_len);
    if (batch->n_seqs > 0) {
        if ((n > 0 && d_lse == nullptr) || d_weights == nullptr) return SZ_ERR_INVALID_ARGUMENT;
        if (overlap(d_weights, bytes, span(*q, n, dim)) ||
            overlap(d_weights, bytes, span_of(d_lse, 4 * n * q->heads)) ||
            (d_before != d_weights && overlap(d_weights, bytes, span_of(d_before, bytes))))
            return SZ_ERR_INVALID_ARGUMENT;
        if (need > 0 && (d_workspace == nullptr || !aligned(d_workspace, 256) ||
                         workspace_bytes < need || overlap(d_workspace, need, span(*q, n, dim)) ||
                         overlap(d_workspace, need, span_of(d_lse, 4 * n * q->heads)) ||
                         overlap(d_workspace, need, span_of(d_before, bytes)) ||
                         overlap(d_workspace, need, span_of(d_weights, bytes))))
            return SZ_ERR_INVALID_ARGUMENT;
        // (a launch holds fewer than 2^32 threads, 256 a workgroup)
        if (sz::weigh_groups((uint32_t)q->heads, cache_of(*cache), batch->n_seqs, n, max_len) >=
            uint64_t{1} << 24)
            return SZ_ERR_INVALID_ARGUMENT;
    }
    if (batch->n_seqs == 0) return SZ_OK;
    if (sz_status s = check_stream(stream)) return s;
    sz::Cache c = cache_of(*cache);
    c.v_pages = c.k_pages;
    const sz::Weigh a{rows_of(q), d_lse, d_before, d_weights, weights_pitch, keep, c,
                      batch_of(*batch), (int64_t)max_len, scale, softcap, causal != 0, window};
    sz_status st = hip_status(sz::launch_weigh(a, static_cast<float*>(d_workspace), stream));
    if (st == SZ_OK && d_status != nullptr)
        st = hip_status(sz::launch_check_seqs(
            sz::SeqCheck{c, a.batch, a.max_len, 0, a.causal, window, d_status}, stream));
    return st;
}

sz_status sz_evict_pages(const float* d_weights, uint64_t weight_heads, uint64_t weights_pitch,
                         const sz_kv_cache* from, const int32_t* d_lens, uint64_t n_seqs,
                         uint64_t max_len, uint64_t budget, uint64_t first, uint64_t recent,
                         const sz_kv_cache* to, float* d_weights_to, int32_t* d_kept,
                         int32_t* d_lens_to, int32_t* d_status, hipStream_t stream) {
    return sz_evict_pages_pitched(d_weights, weight_heads, weights_pitch, from, d_lens, n_seqs,
                                  max_len, budget, first, recent, to, d_weights_to, budget,
                                  d_kept, d_lens_to, d_status, stream);
}

sz_status sz_evict_pages_pitched(const float* d_weights, uint64_t weight_heads,
                                 uint64_t weights_pitch, const sz_kv_cache* from,
                                 const int32_t* d_lens, uint64_t n_seqs, uint64_t max_len,
                                 uint64_t budget, uint64_t first, uint64_t recent,
                                 const sz_kv_cache* to, float* d_weights_to,
                                 uint64_t weights_to_pitch, int32_t* d_kept, int32_t* d_lens_to,
                                 int32_t* d_status, hipStream_t stream) {
    if (!cache_ok(from) || !cache_ok(to) || from->kv_heads != to->kv_heads ||
        from->head_dim != to->head_dim || n_seqs > kMaxSeqs)
        return SZ_ERR_INVALID_ARGUMENT;
    if ((weight_heads != 1 && weight_heads != from->kv_heads) || budget == 0 || budget > kMaxLen ||
        first > budget || recent > budget - first || weights_pitch > kMaxTokens ||
        weights_to_pitch < budget || weights_to_pitch > kMaxTokens)
        return SZ_ERR_INVALID_ARGUMENT;
    const uint64_t most = most_len(*from);
    if (max_len == 0 || max_len > most) max_len = most;
    const uint64_t room = budget < max_len ? budget : max_len;
    if (weights_pitch < max_len || most_len(*to) < room ||
        n_seqs * weight_heads >= uint64_t{1} << 22 ||
        (room + 15) / 16 * n_seqs >= uint64_t{1} << 24)
        return SZ_ERR_INVALID_ARGUMENT;
    if (!aligned(d_weights, 4) || !aligned(d_weights_to, 4) || !aligned(d_kept, 4) ||
        !aligned(d_lens, 4) || !aligned(d_lens_to, 4) || !aligned(d_status, 4))
        return SZ_ERR_INVALID_ARGUMENT;
    if (n_seqs == 0) return SZ_OK;
    if (d_weights == nullptr || d_weights_to == nullptr || d_kept == nullptr ||
        d_lens == nullptr || d_lens_to == nullptr)
        return SZ_ERR_INVALID_ARGUMENT;
    // what is read and what is written, apart
    const uint64_t lines = 4 * n_seqs * weight_heads, lens = 4 * n_seqs;
    const Span read[2] = {span_of(d_weights, lines * weights_pitch), span_of(d_lens, lens)};
    const uint64_t to_bytes = (lines - 4) * weights_to_pitch + 4 * budget;
    const Span written[4] = {span_of(d_weights_to, to_bytes), span_of(d_kept, lines * budget),
                             span_of(d_lens_to, lens),
                             span_of(d_status, d_status == nullptr ? 0 : lens)};
    for (int i = 0; i < 4; i++) {
        for (const Span& r : read)
            if (spans_meet(written[i], r)) return SZ_ERR_INVALID_ARGUMENT;
        for (int j = 0; j < i; j++)
            if (spans_meet(written[i], written[j])) return SZ_ERR_INVALID_ARGUMENT;
    }
    if (sz_status s = check_stream(stream)) return s;
    const sz::Evict a{d_weights, weights_pitch, (uint32_t)weight_heads, (uint32_t)budget,
                      (uint32_t)first, (uint32_t)recent, cache_of(*from), cache_of(*to), d_lens,
                      (int64_t)max_len, d_weights_to, weights_to_pitch, d_kept, d_lens_to};
    sz_status st = hip_status(sz::launch_evict(a, (uint32_t)n_seqs, stream));
    if (st == SZ_OK && d_status != nullptr)
        st = hip_status(sz::launch_evict_check(a, (uint32_t)n_seqs, d_status, stream));
    return st;
}

}  // extern "C"
