// kv_internal.h -- shared by the operators on a paged cache (append.hip,
// attend.hip) and their entry points (kv_api.hip); not installed.
#pragma once

#include "sz_internal.h"

namespace sz {

// sz_heads as the kernels take it
struct Rows {
    void* data;
    uint64_t token_stride, head_stride;
    uint32_t heads;
    uint32_t f32;  // 1: float, 0: BF16
};

// sz_kv_cache
struct Cache {
    const uint64_t* k_pages;
    const uint64_t* v_pages;
    uint64_t pages_per_seq, table_pitch;
    uint64_t token_stride, head_stride;
    uint32_t kv_heads, head_dim;
    uint32_t page_log2;
};

// sz_batch
struct Batch {
    const int32_t* starts;
    const int32_t* lens;
    uint32_t n_seqs, n_tokens;
};

struct Turn {
    const uint64_t* phases;
    uint32_t dims;         // rotary_dim
    uint32_t interleaved;
    float magnitude;
};

constexpr uint32_t kWave = 64;

// A page address that may be read or written: the tables hold what the
// caller put there, and a NULL, misaligned or impossible entry (addresses
// have 48 bits, as has the base of a buffer) is never followed.
__device__ __forceinline__ bool good_page(uint64_t address) {
    return address != 0 && (address & 15) == 0 && address >> 48 == 0;
}

// The last s in [0, n_seqs) with first(s) <= x, for ascending `first` with
// first(0) <= x: 64 candidates are probed at a time, one per lane (one
// round of loads up to 64 sequences, two up to 4096).  Ends, in range, for
// any values; the caller checks the answer.
template <class First>
__device__ __forceinline__ uint32_t find_seq(uint32_t n_seqs, int64_t x, First first) {
    const uint32_t lane = threadIdx.x % kWave;
    uint32_t lo = 0, count = n_seqs;
    while (count > 1) {
        const uint32_t step = (count + kWave - 1) / kWave;
        const uint32_t off = lane * step;
        const bool below = off < count && first(lo + off) <= x;
        const uint32_t hits = __popcll(__ballot(below));
        const uint32_t at = (hits > 0 ? hits - 1 : 0) * step;
        const uint32_t left = count - at;
        lo += at;
        count = step < left ? step : left;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// A sequence's row range and length as the device arrays give them, and
// whether they make sense together.
struct Seq {
    int32_t begin, end, len;
    bool good;
};
__device__ __forceinline__ Seq load_seq(const Batch& b, uint32_t s, int64_t max_len) {
    Seq q;
    q.begin = __builtin_amdgcn_readfirstlane(b.starts[s]);
    q.end = __builtin_amdgcn_readfirstlane(b.starts[s + 1]);
    q.len = __builtin_amdgcn_readfirstlane(b.lens[s]);
    q.good = q.begin >= 0 && q.begin <= q.end && q.end <= (int64_t)b.n_tokens && q.len >= 0 &&
             q.len <= max_len;
    return q;
}

constexpr int32_t kSeqGood = 0;  // SZ_OK (kBlockInvalid: SZ_ERR_INVALID_ARGUMENT)

struct TurnRows {
    Rows q, q_out, k, k_out, v;  // heads 0 where absent
    const float* q_weight;
    const float* k_weight;
    const int32_t* positions;
    Turn turn;
    float eps;
    uint32_t head_dim, n_tokens;
};
hipError_t launch_turn(const TurnRows& a, hipStream_t stream);
hipError_t launch_append(const TurnRows& a, const Cache& cache, const Batch& batch,
                         hipStream_t stream);

struct Attend {
    Rows q, out;
    float* lse;
    Cache cache;
    Batch batch;
    int64_t max_len;
    float scale, softcap;
    uint32_t causal;
    uint64_t window;
};
// Bytes of workspace that launch_attend may use, whatever the window.
uint64_t attend_workspace(uint32_t q_heads, const Cache& cache, uint64_t n_seqs,
                          uint64_t n_tokens, uint64_t max_len);
hipError_t launch_attend(const Attend& a, uint8_t* ws, hipStream_t stream);

// Every sequence's status: one wave per sequence checks its range, its
// length and the pages that the call touches (append: those of the new
// tokens; attention: those of the visible ones).
struct SeqCheck {
    Cache cache;
    Batch batch;
    int64_t max_len;
    uint32_t append;
    uint32_t causal;
    uint64_t window;
    int32_t* status;
};
hipError_t launch_check_seqs(const SeqCheck& c, hipStream_t stream);

}  // namespace sz
