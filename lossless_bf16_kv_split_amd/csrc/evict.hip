// evict.hip -- the attention weight that each cached token has received, and
// the eviction of those that have received the least.
//
// Weights: for every cached token j of a KV head
//   w_j = keep * before_j + sum over the rows i that see j of exp(s_ij - lse_i)
// with the scores s and log-sums lse of attention: a second pass over the keys
// alone.  A workgroup owns keys and walks the rows, so that every sum is made
// in one place and in one order.  The product runs on the matrix cores as
// S^T = K Q^T: a lane's results belong to one row, whose log-sum it holds, and
// the sums over rows are kept lane by lane until the end.
#include "attend_parts.h"

namespace sz {
namespace {

constexpr uint64_t kCus = 256;

// Two forms.  Few rows a sequence (a token's heads, drafts): k_weigh_few, a
// wave streams blocks of 32 keys against the rows that it holds.  Many:
// k_weigh_tile, a wave holds 64 keys and the rows pass by, staged in LDS for
// the four waves of a workgroup; up to `splits` workgroups share a tile's rows,
// as many as the sequence has kSplitRows of them (the sums then meet in the
// workspace).
//
// A call goes by its sequences' average, but a sequence with more than kFewRows
// rows among few (a chunk of a prompt beside single tokens, or idle sequences)
// goes through the tile's loop in the first kernel as well, unsplit: streaming
// reads and places every row again for each 32 keys.  Streamed and so, 128
// elements, us: 16 single tokens and 500 new ones, group 1, 149 and 70; 255 and
// 1700, group 4, 1738 and 597; 32 and 128 136 and 75; 32 and 64 (256 rows) 78 and
// 53; 63 idle sequences and 256 new tokens 345 and 130; 24 and 500, 256 elements,
// 57 and 34.  With 64 or 256 for kFewRows they take the same, but for the 256
// rows, streamed with 256.  (Workgroups of 256 keys where that can be took a
// third off some, but cost uniform drafts, 64 of 5 tokens, 70.9 for 68.3.)
constexpr uint64_t kFewRows = 128;
constexpr uint64_t kSplitRows = 256;
constexpr uint64_t kSplitBytes = uint64_t{1} << 28;  // of workspace, no more
struct WeighPlan {
    uint32_t group;   // G
    bool few;
    uint32_t keys;    // of a workgroup
    uint32_t chunks;  // of so many keys up to max_len
    uint32_t splits;
    __device__ uint32_t splits_of(uint64_t rows) const {
        const uint64_t most = (rows + kSplitRows - 1) / kSplitRows;
        return most < 1 ? 1 : most < splits ? (uint32_t)most : splits;
    }
};
// Blocks of 16 keys that a wave has of a tile, and a tile's keys.  Within
// k_weigh_few half of them, for which its registers are enough: four take 20%
// off such chunks, but cost all batches of few rows a wave or two a SIMD with 64
// elements (64 drafts of 5 tokens 44 us, not 36.5) and spills with 128 and 256.
constexpr int kBlocks = 4, kBlocksFew = 2;
constexpr uint32_t tile_keys(int blocks) { return kWaves * 16 * blocks; }

// What a workgroup works on
struct Work {
    uint32_t kv, s, split;
    int32_t tile;  // its first key
    __device__ __forceinline__ Work(const Weigh& a, const WeighPlan& p) {
        uint32_t rest = blockIdx.x;
        kv = rest % a.cache.kv_heads;
        rest /= a.cache.kv_heads;
        s = rest % a.batch.n_seqs;
        rest /= a.batch.n_seqs;
        split = rest % p.splits;
        tile = (int32_t)(rest / p.splits * p.keys);
    }
};

// The new tokens of a sequence, of which `count` stand from c0 on, that see any
// of the keys key0 .. key0 + keys - 1
struct Tokens {
    int64_t lo, hi;
    __device__ __forceinline__ Tokens(const Weigh& a, int32_t count, int32_t c0, int32_t key0,
                                      int32_t keys)
        : lo(0), hi(count) {
        if (a.causal) {
            if (key0 > c0) lo = (int64_t)key0 - c0;
            const int64_t past = (int64_t)key0 + keys - 1 + (int64_t)a.window - c0;
            if (a.window != 0 && past < hi) hi = past;
        }
        if (lo > hi) hi = lo;
    }
};

// Keys that the row of a token at position c sees: low .. high - 1
__device__ __forceinline__ void seen_keys(const Weigh& a, int32_t len, int32_t c, int32_t& low,
                                          int32_t& high) {
    low = 0;
    high = len;
    if (a.causal) {
        high = c + 1;
        if (a.window != 0 && (int64_t)c + 1 > (int64_t)a.window) low = c + 1 - (int32_t)a.window;
    }
}

// 16 keys' rows as the first operand: key n, elements 32 c + 8 h .. + 7
template <int SLICES>
__device__ __forceinline__ void load_keys(const Weigh& a, uint32_t s, uint32_t kv, int32_t j,
                                          int32_t len, uint32_t lane, bf16x8 (&k)[SLICES]) {
    const uint32_t n = lane % 16, h = lane / 16;
    uint64_t page = 0;
    if (j < len)
        page = page_address(a.cache.k_pages, (uint64_t)s * a.cache.table_pitch +
                                                 ((uint32_t)j >> a.cache.page_log2));
    const auto rows = block_rows(a.cache, page, (uint32_t)j & ((1u << a.cache.page_log2) - 1), kv,
                                 len - j);
#pragma unroll
    for (int c = 0; c < SLICES; c++) {
        const uint32_t off = 32 * c + 8 * h < a.cache.head_dim
                                 ? n * 2 * (uint32_t)a.cache.token_stride + 64 * c + 16 * h
                                 : 0x80000000u;
        k[c] = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(rows, off, 0, 0));
    }
}

// The sum over a row of 16 lanes of each of N values: lane n gets value n %
// N's.
template <int N>
__device__ __forceinline__ float sum_lanes(float (&x)[N], uint32_t n) {
#pragma unroll
    for (int half = N / 2; half >= 1; half /= 2) {
        const bool upper = n & half;
#pragma unroll
        for (int i = 0; i < half; i++) {
            float low = x[i], high = x[i + half];
            // (two values to choose from; unseen, the compiler makes all the
            // steps' choices one index into x, a chain of a thousand selects)
            asm("" : "+v"(low), "+v"(high));
            x[i] = (upper ? high : low) + __shfl_xor(upper ? low : high, half);
        }
    }
#pragma unroll
    for (int d = N; d < 16; d *= 2) x[0] += __shfl_xor(x[0], d);
    return x[0];
}

template <bool CAPPED>
__device__ __forceinline__ float weight_of(const Score& score, float z, float minus) {
    const float x = CAPPED ? capped(score, z) + minus : fmaf(z, score.by, minus);
    return __builtin_amdgcn_exp2f(x);
}

// ---- many rows ---------------------------------------------------------------
//
// Rows pass in steps of 32 through LDS: each wave fetches eight of them while
// the step before is worked on, one barrier a step.  LDS rows are cut into
// 16-byte pieces, piece c of row r at c ^ (r & 15) (r >> 1 & 7 with 64
// elements), so that 16 rows' same piece lies in 16 places.  Bound by the vector
// instructions, an exponential and two more for every score (62% of the cycles,
// the products 33%): a prompt of 4096 tokens, 32/8 heads of 128, 81 to 98 us by
// card with the join's 4.7.
constexpr uint32_t kStepRows = 32;
template <int DP>
struct TileLds {
    uint8_t rows[2][kStepRows * 2 * DP];
    float minus[2][kStepRows];
    int32_t place[2][kStepRows];  // positions; none: INT32_MIN
};

// The sums of this lane's key over the rows of split w.split of `splits`, keys
// from w.tile on and before `past`.  All waves of the workgroup.
template <int DP, bool CAPPED, int BLOCKS>
__device__ __forceinline__ float tile_sums(const Weigh& a, const WeighPlan& p, const Score& score,
                                           const Work& w, const Seq& seq, int32_t past,
                                           uint32_t splits, TileLds<DP>& lds) {
    constexpr int kSlices = DP / 32;
    constexpr uint32_t kRowBytes = 2 * DP;
    constexpr int kLoads = DP / 64;  // 16-byte pieces of a lane, eight lanes a row
    constexpr uint32_t kMixMask = DP == 64 ? 7 : 15;
    auto& staged = lds.rows;
    auto& minus_of = lds.minus;
    auto& place_of = lds.place;
    const uint32_t lane = threadIdx.x % kWave, n = lane % 16, h = lane / 16;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    constexpr int kWaveKeys = 16 * BLOCKS;
    const int32_t key0 = w.tile + kWaveKeys * (int32_t)wave;
    const int32_t count = seq.end - seq.begin, c0 = seq.len - count;
    const uint32_t dim = a.cache.head_dim;

    // the rows of the tokens that see any of the workgroup's keys, in steps
    const Tokens t(a, count, c0, w.tile, (int32_t)tile_keys(BLOCKS));
    const uint32_t row_lo = (uint32_t)t.lo * p.group, row_hi = (uint32_t)t.hi * p.group;
    const uint64_t all = (row_hi - row_lo + kStepRows - 1) / kStepRows;
    const uint32_t step0 = (uint32_t)(all * w.split / splits);
    const uint32_t steps = (uint32_t)(all * (w.split + 1) / splits) - step0;

    float acc[4 * BLOCKS];  // keys 16 b + 4 h + i of key0
#pragma unroll
    for (int i = 0; i < 4 * BLOCKS; i++) acc[i] = 0;
    if (steps > 0) {
        // the row that this lane fetches a part of: its address and its
        // log-sum's move on by a step's tokens and heads, with or without a
        // token more
        const uint32_t mine = 8 * wave + lane / 8;
        const uint32_t d_token = kStepRows / p.group, d_head = kStepRows % p.group;
        const int64_t q_step = 2 * ((int64_t)d_token * (int64_t)a.q.token_stride +
                                    (int64_t)d_head * (int64_t)a.q.head_stride);
        const int64_t q_wrap = 2 * ((int64_t)a.q.token_stride -
                                    (int64_t)p.group * (int64_t)a.q.head_stride);
        const int64_t l_step = 4 * ((int64_t)d_token * a.q.heads + d_head);
        const int64_t l_wrap = 4 * ((int64_t)a.q.heads - p.group);
        uint32_t row = row_lo + step0 * kStepRows + mine;
        uint32_t head = row % p.group;
        int32_t place = c0 + (int32_t)(row / p.group);
        uint64_t from, lse_at;
        {
            const uint64_t token = (uint32_t)seq.begin + row / p.group;
            const uint32_t at = w.kv * p.group + head;
            from = reinterpret_cast<uint64_t>(a.q.data) +
                   2 * (token * a.q.token_stride + at * a.q.head_stride + 8 * (lane % 8));
            lse_at = reinterpret_cast<uint64_t>(a.lse) + 4 * (token * a.q.heads + at);
        }
        struct Fetch {
            u32x4 v[kLoads];
            float lse;
            int32_t place;
        };
        const auto fetch = [&](Fetch& f) {
            const bool on = row < row_hi;
#pragma unroll
            for (int i = 0; i < kLoads; i++) f.v[i] = u32x4{0, 0, 0, 0};
            f.lse = -INFINITY;
            if (on) {
                f.lse = *(const SZ_GLOBAL float*)lse_at;
#pragma unroll
                for (int i = 0; i < kLoads; i++)
                    if (64 * i + 8 * (lane % 8) < dim)
                        f.v[i] = *(const SZ_GLOBAL u32x4*)(from + 128 * i);
            }
            f.place = place;
            row += kStepRows;
            head += d_head;
            const bool wraps = head >= p.group;
            head -= wraps ? p.group : 0;
            place += (int32_t)d_token + wraps;
            from += q_step + (wraps ? q_wrap : 0);
            lse_at += l_step + (wraps ? l_wrap : 0);
        };
        const uint32_t put_mix = (DP == 64 ? mine >> 1 : mine) & kMixMask;
        const auto put = [&](const Fetch& f, uint32_t buffer) {
#pragma unroll
            for (int i = 0; i < kLoads; i++)
                *reinterpret_cast<u32x4*>(&staged[buffer][mine * kRowBytes +
                                                          ((8 * i + lane % 8) ^ put_mix) * 16]) =
                    f.v[i];
            if (lane % 8 == 0) {
                // (a row whose log-sum is -infinity has seen nothing)
                minus_of[buffer][mine] = -f.lse * kLog2e;
                place_of[buffer][mine] = f.lse == -INFINITY ? INT32_MIN : f.place;
            }
        };
        // Steps [none, ..) have a row that sees one of this wave's keys, steps
        // [full0, full1) only rows that see all of them.
        const auto step_of = [&](int64_t rows_before, bool up) {
            int64_t x = rows_before - row_lo + (up ? (int64_t)kStepRows - 1 : 0);
            x = (x < 0 ? 0 : x) / kStepRows - step0;
            return (uint32_t)(x < 0 ? 0 : x > steps ? steps : x);
        };
        const int64_t group = p.group;
        uint32_t none = key0 < past ? 0 : steps, full0 = 0, full1 = step_of(row_hi, false);
        if (a.causal) {
            const int64_t first = key0 - (int64_t)c0;  // the token that stands at key0
            if (key0 < past && first > 0)
                none = first * group >= row_hi ? steps : step_of(first * group, false);
            full0 = step_of((first + kWaveKeys - 1) * group, true);
            if (a.window != 0) {
                const uint32_t end = step_of((first + (int64_t)a.window) * group, false);
                full1 = end < full1 ? end : full1;
            }
        }
        Fetch next;
        fetch(next);
        bf16x8 k[BLOCKS][kSlices];
#pragma unroll
        for (int b = 0; b < BLOCKS; b++)
            load_keys<kSlices>(a, w.s, w.kv, key0 + 16 * b, past, lane, k[b]);
        put(next, 0);
        // (here, or every step waits for them again, and for the rows behind)
#pragma unroll
        for (int b = 0; b < BLOCKS; b++)
#pragma unroll
            for (int u = 0; u < kSlices; u++) asm volatile("" : "+v"(k[b][u]));
        fetch(next);
        const uint32_t q_mix = (DP == 64 ? n >> 1 : n) & kMixMask;
        uint32_t step = 0;
        // 16 of a step's rows: the lane's, its products with the keys
        struct Products {
            f32x4 z[BLOCKS];
            float minus;
            int32_t place;
        };
        const auto products = [&](Products& x, int r) {
            const uint32_t buffer = step & 1;
            x.minus = minus_of[buffer][16 * r + n];
            x.place = place_of[buffer][16 * r + n];
            bf16x8 q[kSlices];
#pragma unroll
            for (int u = 0; u < kSlices; u++)
                q[u] = *reinterpret_cast<const bf16x8*>(
                    &staged[buffer][(16 * r + n) * kRowBytes + ((4 * u + h) ^ q_mix) * 16]);
#pragma unroll
            for (int b = 0; b < BLOCKS; b++) {
                x.z[b] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int u = 0; u < kSlices; u++)
                    x.z[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k[b][u], q[u], x.z[b], 0, 0,
                                                                     0);
            }
        };
        const auto end_step = [&] {
            put(next, (step & 1) ^ 1);
            fetch(next);
            step++;
        };
        const auto edges = [&](uint32_t stop) {
#pragma unroll 1
            while (step < stop) {
                lds_barrier();
#pragma unroll 1
                for (int r = 0; r < 2; r++) {
                    Products x;
                    products(x, r);
                    int32_t low, high;
                    seen_keys(a, seq.len, x.place, low, high);
                    if (x.place == INT32_MIN) high = low;
                    const Sees sees(low, high, key0 + 4 * (int32_t)h);
#pragma unroll
                    for (int i = 0; i < 4 * BLOCKS; i++) {
                        const float e = weight_of<CAPPED>(score, x.z[i / 4][i % 4], x.minus);
                        acc[i] += sees(16 * (i / 4) + i % 4) ? e : 0.0f;
                    }
                }
                end_step();
            }
        };
#pragma unroll 1
        while (step < none) {
            lds_barrier();
            end_step();
        }
        edges(full0 < steps ? full0 : steps);
#pragma unroll 1
        while (step < full1) {
            lds_barrier();
#pragma unroll
            for (int r = 0; r < 2; r++) {
                Products x;
                products(x, r);
                const bool nothing = x.place == INT32_MIN;
                if (__ballot(nothing) != 0) {
#pragma unroll
                    for (int b = 0; b < BLOCKS; b++)
#pragma unroll
                        for (int i = 0; i < 4; i++) x.z[b][i] = nothing ? 0 : x.z[b][i];
                    x.minus = nothing ? -INFINITY : x.minus;
                }
#pragma unroll
                for (int i = 0; i < 4 * BLOCKS; i++)
                    acc[i] += weight_of<CAPPED>(score, x.z[i / 4][i % 4], x.minus);
            }
            end_step();
        }
        edges(steps);
    }

    return sum_lanes<4 * BLOCKS>(acc, n);
}

// The key whose sum a lane gets, of a tile's from `tile` on (past every key where
// another lane has it too)
template <int BLOCKS>
__device__ __forceinline__ int32_t tile_key(int32_t tile) {
    const uint32_t lane = threadIdx.x % kWave, n = lane % 16, h = lane / 16;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (n >= 4 * BLOCKS) return INT32_MAX;
    return tile + 16 * BLOCKS * (int32_t)wave + 16 * (int32_t)(n / 4) + 4 * (int32_t)h +
           (int32_t)(n % 4);
}

template <int DP, bool CAPPED>
__global__ __launch_bounds__(kThreads, DP > 128 ? 2 : 3) void k_weigh_tile(Weigh a, WeighPlan p,
                                                                           Score score,
                                                                           float* ws) {
    __shared__ __attribute__((aligned(256))) TileLds<DP> lds;
    const Work w(a, p);
    const Seq seq = load_seq(a.batch, w.s, a.max_len);
    if (!seq.good || w.tile >= seq.len) return;
    const int32_t count = seq.end - seq.begin, c0 = seq.len - count;
    const uint32_t splits = p.splits_of((uint64_t)count * p.group);
    if (w.split >= splits) return;
    const float sum = tile_sums<DP, CAPPED, kBlocks>(a, p, score, w, seq, seq.len, splits, lds);
    const int32_t j = tile_key<kBlocks>(w.tile);
    if (j >= seq.len) return;
    const uint64_t line = (uint64_t)w.s * a.cache.kv_heads + w.kv;
    if (splits > 1) {
        ws[((uint64_t)w.split * a.batch.n_seqs * a.cache.kv_heads + line) * (uint64_t)a.max_len +
           (uint32_t)j] = sum;
    } else {
        const uint64_t at = line * a.pitch + (uint32_t)j;
        a.weights[at] = a.before != nullptr && j < c0 ? fmaf(a.keep, a.before[at], sum) : sum;
    }
}

// ---- few rows ----------------------------------------------------------------
//
// Bound by the reads of keys: 48 tokens of 32/8 heads on 130 to 8192 keys, 432 MB,
// 86 to 95 us by card, 4.5 to 5.0 TB/s.
template <int DP, bool CAPPED>
__global__ __launch_bounds__(kThreads, DP > 128 ? 2 : 3) void k_weigh_few(Weigh a, WeighPlan p,
                                                                          Score score) {
    constexpr int kSlices = DP / 32;
    constexpr uint32_t kRowBytes = 2 * DP;
    __shared__ __attribute__((aligned(256))) union {
        uint8_t turned[kWaves][32 * kRowBytes];
        TileLds<DP> tile;
    } lds;
    const uint32_t lane = threadIdx.x % kWave, n = lane % 16, h = lane / 16;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    Work w(a, p);
    const Seq seq = load_seq(a.batch, w.s, a.max_len);
    if (!seq.good || w.tile >= seq.len) return;
    const int32_t count = seq.end - seq.begin, c0 = seq.len - count;
    const int32_t past = seq.len - w.tile < (int32_t)p.keys ? seq.len : w.tile + (int32_t)p.keys;
    const uint32_t dim = a.cache.head_dim;
    const uint64_t line = ((uint64_t)w.s * a.cache.kv_heads + w.kv) * a.pitch;
    if ((uint64_t)count * p.group > kFewRows) {
        w.split = 0;
        for (; w.tile < past; w.tile += (int32_t)tile_keys(kBlocksFew)) {
            const float sum =
                tile_sums<DP, CAPPED, kBlocksFew>(a, p, score, w, seq, past, 1, lds.tile);
            const int32_t j = tile_key<kBlocksFew>(w.tile);
            if (j < past)
                a.weights[line + (uint32_t)j] =
                    a.before != nullptr && j < c0
                        ? fmaf(a.keep, a.before[line + (uint32_t)j], sum) : sum;
            lds_barrier();  // (every wave is done with the rows)
        }
        return;
    }

    // 16 rows from r0 on: the lane's own, its log-sum and what it sees
    struct RowBlock {
        bf16x8 q[kSlices];
        float minus;
        int32_t low, high, least;  // least: of its tokens' positions
    };
    const uint32_t rows = (uint32_t)count * p.group;
    const auto load_rows = [&](uint32_t r0, RowBlock& b) {
        const uint32_t row = r0 + n;
        const bool on = row < rows;
        const uint32_t token = on ? row / p.group : 0, head = on ? row % p.group : 0;
        const uint64_t t = (uint32_t)seq.begin + token;
        const uint32_t at = w.kv * p.group + head;
        float lse = -INFINITY;
        if (on) lse = *(const SZ_GLOBAL float*)(a.lse + t * a.q.heads + at);
        const uint16_t* x = static_cast<const uint16_t*>(a.q.data) + t * a.q.token_stride +
                            at * a.q.head_stride;
#pragma unroll
        for (int u = 0; u < kSlices; u++) {
            u32x4 v = {0, 0, 0, 0};
            if (on && 32 * u + 8 * h < dim) v = *(const SZ_GLOBAL u32x4*)(x + 32 * u + 8 * h);
            b.q[u] = __builtin_bit_cast(bf16x8, v);
        }
        seen_keys(a, seq.len, c0 + (int32_t)token, b.low, b.high);
        // (a row whose log-sum is -infinity has seen nothing)
        if (lse == -INFINITY) b.high = b.low;
        b.minus = -lse * kLog2e;
    };
    RowBlock row;
    const uint32_t blocks = (rows + 15) / 16;
    // 32 keys as they are loaded, DP / 8 lanes a row, which LDS turns into
    // operands (asked for in the operands' order, 16 rows at a time, they keep
    // the address units busy four times as long: 48 tokens 103 us, now 94.5).
    constexpr int kLanes = DP / 8, kLoads = 32 * kLanes / (int)kWave;
    constexpr uint32_t kMixMask = DP == 64 ? 7 : 15;
    const auto mix = [](uint32_t r) { return (DP == 64 ? r >> 1 : r) & kMixMask; };
    struct Keys {
        u32x4 k[kLoads];
        float before;
    };
    const uint32_t piece = lane % kLanes;
    const uint32_t row_bytes = 2 * (uint32_t)a.cache.token_stride;
    const uint32_t off0 =
        8 * piece < dim ? lane / kLanes * row_bytes + 16 * piece : 0x80000000u;
    // Keys of a block of 32, and what the lane's key had before.  Lane (n, h)
    // ends with the sum of key 16 (n / 4 % 2) + 4 h + n % 4.
    const int32_t mine = 16 * (int32_t)(n / 4 % 2) + 4 * (int32_t)h + (int32_t)(n % 4);
    const auto load = [&](Keys& x, int32_t j) {
        // (keys that no row sees are not read)
        const Tokens t(a, count, c0, j, 32);
        const int32_t upto = t.lo < t.hi ? past : j;
#pragma unroll
        for (int b = 0; b < 2; b++) {
            const int32_t jb = j + 16 * b;
            uint64_t page = 0;
            if (jb < upto)
                page = page_address(a.cache.k_pages, (uint64_t)w.s * a.cache.table_pitch +
                                                         ((uint32_t)jb >> a.cache.page_log2));
            const auto rows =
                block_rows(a.cache, page, (uint32_t)jb & ((1u << a.cache.page_log2) - 1), w.kv,
                           upto - jb);
#pragma unroll
            for (int i = 0; i < kLoads / 2; i++)
                x.k[kLoads / 2 * b + i] = __builtin_amdgcn_raw_buffer_load_b128(
                    rows, off0 + i * ((int)kWave / kLanes) * row_bytes, 0, 0);
        }
        x.before = 0;
        if (a.before != nullptr && j + mine < past && j + mine < c0)
            x.before = *(const SZ_GLOBAL float*)(a.before + line + (uint32_t)(j + mine));
    };
    const auto compute = [&](const Keys& x, int32_t j) {
        bf16x8 k[2][kSlices];
        {
            uint8_t* const to = lds.turned[wave];
#pragma unroll
            for (int i = 0; i < kLoads; i++) {
                const uint32_t r = i * (kWave / kLanes) + lane / kLanes;
                *reinterpret_cast<u32x4*>(to + r * kRowBytes + (piece ^ mix(r)) * 16) = x.k[i];
            }
            __builtin_amdgcn_wave_barrier();  // (the wave's own: in order)
#pragma unroll
            for (int i = 0; i < 2; i++)
#pragma unroll
                for (int u = 0; u < kSlices; u++)
                    k[i][u] = *reinterpret_cast<const bf16x8*>(
                        to + (16 * i + n) * kRowBytes + ((4 * u + h) ^ mix(n)) * 16);
        }
        float acc[8];
#pragma unroll
        for (int i = 0; i < 8; i++) acc[i] = 0;
        for (uint32_t b = 0; b < blocks; b++) {
            if (blocks > 1) load_rows(16 * b, row);
            f32x4 z[2];
#pragma unroll
            for (int i = 0; i < 2; i++) {
                z[i] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int u = 0; u < kSlices; u++)
                    z[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k[i][u], row.q[u], z[i], 0, 0,
                                                                   0);
            }
            const Sees sees(row.low, row.high, j + 4 * (int32_t)h);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float e = weight_of<CAPPED>(score, z[i / 4][i % 4], row.minus);
                acc[i] += sees(16 * (i / 4) + i % 4) ? e : 0.0f;
            }
        }
        const float sum = sum_lanes<8>(acc, n);
        if (n < 8 && j + mine < past)
            a.weights[line + (uint32_t)(j + mine)] = fmaf(a.keep, x.before, sum);
    };
    constexpr int32_t kStride = 32 * kWaves;
    int32_t j = w.tile + 32 * (int32_t)wave;
    Keys even, odd;
    load(even, j);
    if (blocks == 1) load_rows(0, row);
    for (; j < past; j += 2 * kStride) {
        load(odd, j + kStride);
        compute(even, j);
        load(even, j + 2 * kStride);
        if (j + kStride < past) compute(odd, j + kStride);
    }
}

// Joins what the workgroups that shared a tile's rows have summed, in order.
__global__ __launch_bounds__(kThreads) void k_weigh_join(Weigh a, WeighPlan p, const float* ws) {
    const uint32_t chunks = ((uint32_t)a.max_len + kThreads - 1) / kThreads;
    const uint32_t j = blockIdx.x % chunks * kThreads + threadIdx.x;
    const uint32_t line = blockIdx.x / chunks;
    const uint32_t s = line / a.cache.kv_heads;
    const Seq seq = load_seq(a.batch, s, a.max_len);
    if (!seq.good || j >= (uint32_t)seq.len) return;
    const int32_t c0 = seq.len - (seq.end - seq.begin);
    const uint32_t splits = p.splits_of((uint64_t)(seq.end - seq.begin) * p.group);
    if (splits == 1) return;  // (written already)
    const uint64_t lines = (uint64_t)a.batch.n_seqs * a.cache.kv_heads;
    float total = 0;
#pragma unroll 8
    for (uint32_t i = 0; i < splits; i++) total += ws[(i * lines + line) * (uint64_t)a.max_len + j];
    const uint64_t at = line * a.pitch + j;
    if (a.before != nullptr && (int32_t)j < c0) total = fmaf(a.keep, a.before[at], total);
    a.weights[at] = total;
}

WeighPlan plan_weigh(uint32_t q_heads, const Cache& c, uint64_t n_seqs, uint64_t n_tokens,
                     uint64_t max_len) {
    WeighPlan p;
    p.group = q_heads / c.kv_heads;
    const uint64_t rows = n_tokens * p.group, lines = n_seqs * c.kv_heads;
    p.few = rows <= 32 * n_seqs;
    p.splits = 1;
    if (p.few) {
        // as many keys a workgroup as leave four of them to a CU, 128 (a block a
        // wave) to 512
        uint64_t keys = 512;
        while (keys > 128 && (max_len + keys - 1) / keys * lines < 4 * kCus) keys /= 2;
        p.keys = (uint32_t)keys;
    } else {
        p.keys = tile_keys(kBlocks);
    }
    p.chunks = (uint32_t)((max_len + p.keys - 1) / p.keys);
    if (!p.few) {
        // Rows among so many workgroups that the causal ones' uneven shares even
        // out, or one long sequence among short ones fills the chip: by the
        // tiles of those sequences that can have 2048 rows (a prompt of 4096
        // tokens, 128 tiles: 93 us in 12 parts each, 92 in 16, 98 in 24; 500
        // tokens beside 24 single ones, 256 elements, capped: 193 us whole).
        const uint64_t long_seqs = rows / 2048 < 1 ? 1 : rows / 2048 < n_seqs ? rows / 2048 : n_seqs;
        uint64_t splits = 8 * kCus / (uint64_t{p.chunks} * c.kv_heads * long_seqs);
        const uint64_t most = (rows + kSplitRows - 1) / kSplitRows;
        splits = splits < most ? splits : most;
        const uint64_t fits = kSplitBytes / (4 * lines * max_len);
        splits = splits < fits ? splits : fits;
        p.splits = (uint32_t)(splits < 1 ? 1 : splits);
    }
    return p;
}

template <int DP, bool CAPPED>
void go(const Weigh& a, const WeighPlan& p, float* ws, hipStream_t stream) {
    const dim3 grid(p.chunks * p.splits * a.batch.n_seqs * a.cache.kv_heads), block(kThreads);
    Score score{};
    score.by = a.scale * kLog2e;
    if (CAPPED) {
        Attend x{};
        x.scale = a.scale;
        x.softcap = a.softcap;
        score = score_of(x);
    }
    if (p.few) k_weigh_few<DP, CAPPED><<<grid, block, 0, stream>>>(a, p, score);
    else k_weigh_tile<DP, CAPPED><<<grid, block, 0, stream>>>(a, p, score, ws);
}

// ---- eviction --------------------------------------------------------------
//
// One workgroup for every row of weights finds which tokens stay; then the
// rows of those are copied into other pages.  Tokens get order-preserving keys:
// FP32 weights as unsigned numbers, tokens that stay in any case above them
// all.  The key of the last one that stays is found by counting digits, eleven
// bits at a time, from the top; of equal keys the first stay.  Up to 32,768
// weights and keys stay in registers over the passes, every load under way at
// once; more are read again in pieces of so many for each.  A wave has
// consecutive weights, 64 at a time, so that ballots give each token its place.
// Bound by the vector instructions and LDS of one CU: 32768 weights 26 us, 24 x 8
// rows of up to 8192 17.6; four copies of the counts, by lane, keep equal digits
// apart (one row 41.8 us with the copying, with two 42.7, with one 43.6).
constexpr uint32_t kPickThreads = 1024;
constexpr uint32_t kPickWaves = kPickThreads / kWave;
constexpr uint32_t kDigit = 11, kBins = 1u << kDigit, kCopies = 4;
constexpr uint32_t kHold = 32;  // weights of a thread
constexpr uint32_t kPiece = kHold * kPickThreads;

// Keys: 0 no token, kNan, numbers from 0x007FFFFF (-infinity) to 0xFF800000,
// kSafe.  Both zeros have the same.
constexpr uint32_t kNan = 1, kSafe = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t key_of(float w) {
    const uint32_t u = __float_as_uint(w + 0.0f);  // (-0 + 0 is 0)
    const uint32_t key = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    return w != w ? kNan : key;
}

// Running sums over the lanes of a wave
__device__ __forceinline__ uint32_t wave_scan(uint32_t x) {
    const uint32_t lane = threadIdx.x % kWave;
#pragma unroll
    for (uint32_t d = 1; d < kWave; d *= 2) {
        const uint32_t y = __shfl_up(x, d);
        if (lane >= d) x += y;
    }
    return x;
}

// What the waves before this one have, and all of them, of a number for each
struct Before {
    uint32_t before = 0, all = 0;
    __device__ __forceinline__ Before(const uint32_t* of, uint32_t wave) {
        u32x4 v[kPickWaves / 4];
#pragma unroll
        for (uint32_t i = 0; i < kPickWaves / 4; i++) v[i] = reinterpret_cast<const u32x4*>(of)[i];
#pragma unroll
        for (uint32_t i = 0; i < kPickWaves; i++) {
            const uint32_t x = __builtin_amdgcn_readfirstlane(v[i / 4][i % 4]);
            before += i < wave ? x : 0;
            all += x;
        }
    }
};

__global__ __launch_bounds__(kPickThreads) void k_evict_pick(Evict a) {
    __shared__ uint32_t bins[kCopies][kBins];
    __shared__ __attribute__((aligned(16))) uint32_t sums[2][kPickWaves];
    __shared__ uint32_t chosen[3];
    const uint32_t s = blockIdx.x / a.weight_heads, t = threadIdx.x, lane = t % kWave;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(t / kWave);
    const int32_t len = a.lens[s];
    const bool good = len >= 0 && len <= a.max_len;
    const uint32_t n = good ? (uint32_t)len : 0;
    const uint32_t stay = n < a.budget ? n : a.budget;
    const float* w = a.weights + blockIdx.x * a.pitch;
    int32_t* kept = a.kept + blockIdx.x * (uint64_t)a.budget;
    float* out = a.weights_to + blockIdx.x * a.to_pitch;
    if (blockIdx.x % a.weight_heads == 0 && t == 0) a.lens_to[s] = (int32_t)stay;
    for (uint32_t i = stay + t; i < a.budget; i += kPickThreads) kept[i] = -1;
    if (n <= a.budget) {
        for (uint32_t i = t; i < n; i += kPickThreads) {
            kept[i] = (int32_t)i;
            out[i] = w[i];
        }
        return;
    }
    // A wave's weights of a piece: rounds of 64 consecutive ones.
    const uint32_t rounds = n < kPiece ? (n + kPickThreads - 1) / kPickThreads : kHold;
    const uint32_t mine = (wave * rounds) * kWave + lane;
    const uint32_t lo = a.first, hi = n - a.recent;  // the tokens that may go
    float x[kHold];
    uint32_t key[kHold];
    const auto each = [&](auto f) {
#pragma unroll
        for (uint32_t k = 0; k < kHold; k++)
            if (k < rounds) f(k);
    };
    const auto load = [&](uint32_t base) {
        each([&](uint32_t k) {
            const uint32_t i = base + mine + k * kWave;
            x[k] = 0;
            if (i < n) x[k] = *(const SZ_GLOBAL float*)(w + i);
        });
        each([&](uint32_t k) {
            const uint32_t i = base + mine + k * kWave;
            key[k] = i - lo < hi - lo ? key_of(x[k]) : i < n ? kSafe : 0;
        });
    };
    const bool whole = n <= kPiece;
    if (whole) load(0);

    uint32_t prefix = 0, take = stay;  // of the keys that begin with prefix, the top `take`
    for (int32_t shift = 32 - (int32_t)kDigit; shift > -(int32_t)kDigit; shift -= kDigit) {
        const uint32_t low = shift > 0 ? (uint32_t)shift : 0;
        const uint32_t width = shift > 0 ? kDigit : kDigit + (uint32_t)shift;
        const uint32_t above_digit = low + width;  // bits from here on are settled
        for (uint32_t i = t; i < kCopies * kBins; i += kPickThreads) (&bins[0][0])[i] = 0;
        lds_barrier();
        for (uint32_t base = 0; base < n; base += kPiece) {
            if (!whole) load(base);
            uint32_t* const copy = bins[lane % kCopies];
            if (above_digit >= 32) {  // the first digit: every key counts
                each([&](uint32_t k) { atomicAdd(copy + (key[k] >> low), 1u); });
            } else {
                const uint32_t settled = prefix >> above_digit;
                const uint32_t digit = (1u << width) - 1;
                each([&](uint32_t k) {
                    if (key[k] >> above_digit == settled)
                        atomicAdd(copy + (key[k] >> low & digit), 1u);
                });
            }
        }
        lds_barrier();
        // thread t has bins kBins - 2 t - 2 and the one above it
        uint32_t own[2];
#pragma unroll
        for (uint32_t i = 0; i < 2; i++) {
            own[i] = 0;
#pragma unroll
            for (uint32_t c = 0; c < kCopies; c++) own[i] += bins[c][kBins - 1 - 2 * t - i];
        }
        const uint32_t upto = wave_scan(own[0] + own[1]);
        if (lane == kWave - 1) sums[0][wave] = upto;
        lds_barrier();
        const uint32_t above = upto - own[0] - own[1] + Before(sums[0], wave).before;
        if (above < take && above + own[0] + own[1] >= take) {
            const bool first = above + own[0] >= take;
            chosen[0] = kBins - 1 - 2 * t - (first ? 0 : 1);
            chosen[1] = take - above - (first ? 0 : own[0]);
            chosen[2] = own[first ? 0 : 1];
        }
        lds_barrier();
        prefix = above_digit >= 32 ? chosen[0] << low
                                   : (prefix >> above_digit << above_digit) | chosen[0] << low;
        take = chosen[1];
        // (all that begin like this stay, as distinct weights do after two digits)
        if (take == chosen[2] && prefix != 0) {
            prefix--;
            take = 0;
            break;
        }
    }
    // every key above `prefix` stays, and of those equal to it the first `take`
    uint32_t base_sure = 0, base_ties = 0;
    for (uint32_t base = 0; base < n; base += kPiece) {
        if (!whole) load(base);
        uint32_t sures = 0, ties = 0;
        each([&](uint32_t k) {
            sures += __popcll(__ballot(key[k] > prefix));
            ties += __popcll(__ballot(key[k] == prefix));
        });
        lds_barrier();  // (sums have been read)
        if (lane == 0) {
            sums[0][wave] = sures;
            sums[1][wave] = ties;
        }
        lds_barrier();
        const Before more_before(sums[0], wave), same_before(sums[1], wave);
        uint32_t at = base_sure + more_before.before, rank = base_ties + same_before.before;
        base_sure += more_before.all;
        base_ties += same_before.all;
        each([&](uint32_t k) {
            // (ties that stay counted in, as far as they go)
            const uint64_t more = __ballot(key[k] > prefix), same = __ballot(key[k] == prefix);
            uint64_t stays = more;
            uint32_t place = at + (rank < take ? rank : take);
            if (same != 0 && rank < take) {
                const uint32_t before = __builtin_amdgcn_mbcnt_hi(
                    (uint32_t)(same >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0));
                stays |= __ballot(key[k] == prefix && rank + before < take);
            }
            if (stays >> lane & 1) {
                place += __builtin_amdgcn_mbcnt_hi(
                    (uint32_t)(stays >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)stays, 0));
                kept[place] = (int32_t)(base + mine + k * kWave);
                out[place] = x[k];
            }
            at += __popcll(more);
            rank += __popcll(same);
        });
    }
}

// Copies kept rows, 16 destination tokens and all heads a workgroup: LANES
// lanes a row, 16 bytes each.  At the rate of memory: 206 MB in 37.8 us, 5.4 TB/s.
template <int LANES>
__global__ __launch_bounds__(kThreads) void k_evict_copy(Evict a, uint32_t blocks) {
    constexpr uint32_t kRows = kThreads / LANES;  // of a round
    const uint32_t s = blockIdx.x / blocks, d0 = blockIdx.x % blocks * 16;
    const int32_t len = a.lens[s];
    if (len < 0 || len > a.max_len) return;
    const uint32_t stay = (uint32_t)len < a.budget ? (uint32_t)len : a.budget;
    if (d0 >= stay) return;
    const uint32_t tokens = stay - d0 < 16 ? stay - d0 : 16;
    const uint32_t e = threadIdx.x % LANES * 8;
    const uint64_t entry = (uint64_t)s * a.to.table_pitch + (d0 >> a.to.page_log2);
    const uint64_t to_page[2] = {page_address(a.to.k_pages, entry),
                                 page_address(a.to.v_pages, entry)};
    const uint32_t heads = a.from.kv_heads;
    for (uint32_t r = threadIdx.x / LANES; r < tokens * heads; r += kRows) {
        const uint32_t d = d0 + r / heads, h = r % heads;
        const uint32_t line = s * a.weight_heads + (a.weight_heads == 1 ? 0 : h);
        const uint32_t j = (uint32_t)a.kept[(uint64_t)line * a.budget + d];
        const uint64_t at = (uint64_t)s * a.from.table_pitch + (j >> a.from.page_log2);
        const uint64_t from_off = (j & ((1u << a.from.page_log2) - 1)) * a.from.token_stride +
                                  h * a.from.head_stride + e;
        const uint64_t to_off = (d & ((1u << a.to.page_log2) - 1)) * a.to.token_stride +
                                h * a.to.head_stride + e;
        if (e >= a.from.head_dim) continue;
        const uint64_t from_page[2] = {a.from.k_pages[at], a.from.v_pages[at]};
#pragma unroll
        for (int i = 0; i < 2; i++)
            if (good_page(from_page[i]) && good_page(to_page[i]))
                store_global(reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(to_page[i]) +
                                                      to_off),
                             load_global(reinterpret_cast<const uint4*>(
                                 reinterpret_cast<const uint16_t*>(from_page[i]) + from_off)));
    }
}

// Every sequence's status: a wave each.
__global__ __launch_bounds__(kWave) void k_evict_check(Evict a, int32_t* status) {
    const uint32_t s = blockIdx.x, lane = threadIdx.x;
    const int32_t len = a.lens[s];
    bool good = len >= 0 && len <= a.max_len;
    if (good) {
        const uint32_t stay = (uint32_t)len < a.budget ? (uint32_t)len : a.budget;
        const auto check = [&](const Cache& c, uint32_t tokens) {
            const uint64_t pages = ((uint64_t)tokens + (1u << c.page_log2) - 1) >> c.page_log2;
            const uint64_t row = (uint64_t)s * c.table_pitch;
            for (uint64_t i = lane; i < pages; i += kWave)
                good = good && good_page(c.k_pages[row + i]) && good_page(c.v_pages[row + i]);
        };
        check(a.from, (uint32_t)len);
        check(a.to, stay);
    }
    const bool all = __ballot(!good) == 0;
    if (lane == 0) status[s] = all ? kSeqGood : kBlockInvalid;
}

}  // namespace

uint64_t weigh_groups(uint32_t q_heads, const Cache& cache, uint64_t n_seqs, uint64_t n_tokens,
                      uint64_t max_len) {
    const WeighPlan p = plan_weigh(q_heads, cache, n_seqs, n_tokens, max_len);
    const uint64_t lines = n_seqs * cache.kv_heads;
    const uint64_t join = (max_len + kThreads - 1) / kThreads * lines;
    const uint64_t groups = (uint64_t)p.chunks * p.splits * lines;
    return groups > join ? groups : join;
}

uint64_t weigh_workspace(uint32_t q_heads, const Cache& cache, uint64_t n_seqs, uint64_t n_tokens,
                         uint64_t max_len) {
    const WeighPlan p = plan_weigh(q_heads, cache, n_seqs, n_tokens, max_len);
    if (p.splits == 1) return 0;
    return (4 * p.splits * n_seqs * cache.kv_heads * max_len + 255) / 256 * 256;
}

hipError_t launch_weigh(const Weigh& a, float* ws, hipStream_t stream) {
    const WeighPlan p = plan_weigh(a.q.heads, a.cache, a.batch.n_seqs, a.batch.n_tokens,
                                   (uint64_t)a.max_len);
    const uint32_t dim = a.cache.head_dim;
    if (a.softcap > 0) {
        if (dim <= 64) go<64, true>(a, p, ws, stream);
        else if (dim <= 128) go<128, true>(a, p, ws, stream);
        else go<256, true>(a, p, ws, stream);
    } else {
        if (dim <= 64) go<64, false>(a, p, ws, stream);
        else if (dim <= 128) go<128, false>(a, p, ws, stream);
        else go<256, false>(a, p, ws, stream);
    }
    if (hipError_t e = hipGetLastError()) return e;
    if (p.splits == 1) return hipSuccess;
    const uint32_t chunks = ((uint32_t)a.max_len + kThreads - 1) / kThreads;
    k_weigh_join<<<dim3(chunks * a.batch.n_seqs * a.cache.kv_heads), dim3(kThreads), 0, stream>>>(
        a, p, ws);
    return hipGetLastError();
}

hipError_t launch_evict(const Evict& a, uint32_t n_seqs, hipStream_t stream) {
    k_evict_pick<<<dim3(n_seqs * a.weight_heads), dim3(kPickThreads), 0, stream>>>(a);
    if (hipError_t e = hipGetLastError()) return e;
    const uint32_t most = a.budget < (uint64_t)a.max_len ? a.budget : (uint32_t)a.max_len;
    const uint32_t blocks = (most + 15) / 16, dim = a.from.head_dim;
    if (blocks == 0) return hipSuccess;
    const dim3 grid(blocks * n_seqs), block(kThreads);
    if (dim <= 64) k_evict_copy<8><<<grid, block, 0, stream>>>(a, blocks);
    else if (dim <= 128) k_evict_copy<16><<<grid, block, 0, stream>>>(a, blocks);
    else k_evict_copy<32><<<grid, block, 0, stream>>>(a, blocks);
    return hipGetLastError();
}

hipError_t launch_evict_check(const Evict& a, uint32_t n_seqs, int32_t* status,
                              hipStream_t stream) {
    k_evict_check<<<dim3(n_seqs), dim3(kWave), 0, stream>>>(a, status);
    return hipGetLastError();
}

}  // namespace sz
