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
constexpr int kBlocks = 4;           // of 16 keys, a wave's
constexpr int kWaveKeys = 16 * kBlocks;

// ROWS: the four waves have the same keys and share the rows; otherwise each
// has keys of its own and all rows.  `splits` workgroups share a tile's rows.
struct WeighPlan {
    uint32_t group;   // G
    uint32_t splits;
    uint32_t chunks;  // tiles of keys up to max_len
    bool rows;
    __host__ __device__ uint32_t tile() const { return rows ? kWaveKeys : kWaves * kWaveKeys; }
};

// The sum over a row of 16 lanes of each of 16 values: lane n gets value n's.
__device__ __forceinline__ float sum_lanes(float (&x)[16], uint32_t n) {
#pragma unroll
    for (int half = 8; half >= 1; half /= 2) {
        const bool upper = n & half;
#pragma unroll
        for (int i = 0; i < half; i++) {
            const float mine = upper ? x[i + half] : x[i];
            const float other = upper ? x[i] : x[i + half];
            x[i] = mine + __shfl_xor(other, half);
        }
    }
    return x[0];
}

template <int DP, bool CAPPED, bool ROWS>
__global__ __launch_bounds__(kThreads, 2) void k_weigh(Weigh a, WeighPlan p, Score score,
                                                       float* ws) {
    constexpr int kSlices = DP / 32;
    constexpr int kRowBlocks = DP > 128 ? 1 : 2;  // of 16 rows, worked on at a time
    constexpr uint32_t kStepRows = 16 * kRowBlocks;
    const uint32_t lane = threadIdx.x % kWave, n = lane % 16, h = lane / 16;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    uint32_t rest = blockIdx.x;
    const uint32_t kv = rest % a.cache.kv_heads;
    rest /= a.cache.kv_heads;
    const uint32_t s = rest % a.batch.n_seqs;
    rest /= a.batch.n_seqs;
    const uint32_t split = rest % p.splits;
    const int32_t tile = (int32_t)(rest / p.splits * p.tile());
    const Seq seq = load_seq(a.batch, s, a.max_len);
    if (!seq.good || tile >= seq.len) return;
    const int32_t key0 = tile + (ROWS ? 0 : kWaveKeys * (int32_t)wave);
    const int32_t count = seq.end - seq.begin, c0 = seq.len - count;
    const uint32_t dim = a.cache.head_dim;

    // the rows (tokens of the sequence) that see any of this wave's keys
    int64_t i_lo = 0, i_hi = count;
    if (a.causal) {
        if (key0 > c0) i_lo = (int64_t)key0 - c0;
        const int64_t past = (int64_t)key0 + kWaveKeys - 1 + (int64_t)a.window - c0;
        if (a.window != 0 && past < i_hi) i_hi = past;
    }
    if (key0 >= seq.len || i_lo > i_hi) i_hi = i_lo;
    const uint32_t row_lo = (uint32_t)i_lo * p.group, row_hi = (uint32_t)i_hi * p.group;
    const uint64_t all = (row_hi - row_lo + kStepRows - 1) / kStepRows;
    const uint32_t step0 = (uint32_t)(all * split / p.splits);
    const uint32_t steps = (uint32_t)(all * (split + 1) / p.splits) - step0;

    float acc[16];  // keys 16 b + 4 h + i of key0
#pragma unroll
    for (int i = 0; i < 16; i++) acc[i] = 0;
    if (steps > 0) {
        bf16x8 k[kBlocks][kSlices];
#pragma unroll
        for (int b = 0; b < kBlocks; b++) {
            const int32_t j = key0 + 16 * b;
            uint64_t page = 0;
            if (j < seq.len)
                page = page_address(a.cache.k_pages, (uint64_t)s * a.cache.table_pitch +
                                                         ((uint32_t)j >> a.cache.page_log2));
            const auto rows = block_rows(a.cache, page,
                                         (uint32_t)j & ((1u << a.cache.page_log2) - 1), kv,
                                         seq.len - j);
#pragma unroll
            for (int c = 0; c < kSlices; c++) {
                const uint32_t off = 32 * c + 8 * h < dim
                                         ? n * 2 * (uint32_t)a.cache.token_stride + 64 * c + 16 * h
                                         : 0x80000000u;
                k[b][c] = __builtin_bit_cast(
                    bf16x8, __builtin_amdgcn_raw_buffer_load_b128(rows, off, 0, 0));
            }
        }
        // this lane's row of each block: token and head advance by a step's rows
        constexpr uint32_t kWalk = ROWS ? kWaves : 1;
        const uint32_t stride = kWalk * kStepRows;
        const uint32_t d_token = stride / p.group, d_head = stride % p.group;
        uint32_t row = row_lo + (step0 + (ROWS ? wave : 0)) * kStepRows + n;
        uint32_t token[kRowBlocks], head[kRowBlocks];
#pragma unroll
        for (int r = 0; r < kRowBlocks; r++) {
            token[r] = (row + 16 * r) / p.group;
            head[r] = (row + 16 * r) % p.group;
        }
        bf16x8 q[kRowBlocks][kSlices];
        float lse[kRowBlocks];
        int32_t c[kRowBlocks];
        const auto load = [&] {
#pragma unroll
            for (int r = 0; r < kRowBlocks; r++) {
                const bool on = row + 16 * r < row_hi;
                c[r] = c0 + (int32_t)token[r];
                lse[r] = INFINITY;
                const uint64_t t = (uint32_t)seq.begin + token[r];
                const uint32_t at = kv * p.group + head[r];
                if (on) lse[r] = *(const SZ_GLOBAL float*)(a.lse + t * a.q.heads + at);
                const uint16_t* x = static_cast<const uint16_t*>(a.q.data) +
                                    t * a.q.token_stride + at * a.q.head_stride;
#pragma unroll
                for (int u = 0; u < kSlices; u++) {
                    u32x4 v = {0, 0, 0, 0};
                    if (on && 32 * u + 8 * h < dim)
                        v = *(const SZ_GLOBAL u32x4*)(x + 32 * u + 8 * h);
                    q[r][u] = __builtin_bit_cast(bf16x8, v);
                }
                token[r] += d_token;
                head[r] += d_head;
                if (head[r] >= p.group) {
                    head[r] -= p.group;
                    token[r]++;
                }
            }
            row += stride;
        };
        load();
        for (uint32_t step = ROWS ? wave : 0; step < steps; step += kWalk) {
            // rows of this step, and whether each of them sees each key
            const uint32_t r0 = row_lo + (step0 + step) * kStepRows;
            const int32_t first = c0 + (int32_t)(r0 / p.group);
            const int32_t last = c0 + (int32_t)((r0 + kStepRows - 1) / p.group);
            bool full = r0 + kStepRows <= row_hi &&
                              (!a.causal || (first >= key0 + kWaveKeys - 1 &&
                                             (a.window == 0 || (int64_t)last - (int64_t)a.window <
                                                                   key0)));
            f32x4 z[kRowBlocks][kBlocks];
            float minus[kRowBlocks];
            int32_t low[kRowBlocks], high[kRowBlocks];  // keys that a row sees
#pragma unroll
            for (int r = 0; r < kRowBlocks; r++) {
                minus[r] = -lse[r] * kLog2e;
                low[r] = 0;
                high[r] = seq.len;
                if (a.causal) {
                    high[r] = c[r] + 1;
                    if (a.window != 0 && (int64_t)c[r] + 1 > (int64_t)a.window)
                        low[r] = c[r] + 1 - (int32_t)a.window;
                }
                // (a row whose log-sum is -infinity has seen nothing)
                const bool none = lse[r] == -INFINITY;
                if (none || row - stride + 16 * r >= row_hi) high[r] = low[r];
                full = full && __ballot(none) == 0;
#pragma unroll
                for (int b = 0; b < kBlocks; b++) {
                    z[r][b] = f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int u = 0; u < kSlices; u++)
                        z[r][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k[b][u], q[r][u], z[r][b],
                                                                          0, 0, 0);
                }
            }
            load();
#pragma unroll
            for (int b = 0; b < kBlocks; b++)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    float sum = 0;
#pragma unroll
                    for (int r = 0; r < kRowBlocks; r++) {
                        const float x = CAPPED ? capped(score, z[r][b][i]) + minus[r]
                                               : fmaf(z[r][b][i], score.by, minus[r]);
                        float w = __builtin_amdgcn_exp2f(x);
                        if (!full && !Sees(low[r], high[r], key0 + 4 * (int32_t)h)(16 * b + i))
                            w = 0;
                        sum += w;
                    }
                    acc[4 * b + i] += sum;
                }
        }
    }

    // lane (n, h) gets the sum of key 16 (n / 4) + 4 h + n % 4
    const float sum = sum_lanes(acc, n);
    const int32_t mine = 16 * (int32_t)(n / 4) + 4 * (int32_t)h + (int32_t)(n % 4);
    float total = sum;
    if constexpr (ROWS) {
        __shared__ float parts[kWaves][kWaveKeys];
        parts[wave][mine] = sum;
        __syncthreads();
        if (wave != 0) return;
        total = 0;
#pragma unroll
        for (uint32_t w = 0; w < kWaves; w++) total += parts[w][mine];
    }
    const int32_t j = key0 + mine;
    if (j >= seq.len) return;
    const uint64_t line = (uint64_t)s * a.cache.kv_heads + kv;
    if (p.splits > 1) {
        ws[((uint64_t)split * a.batch.n_seqs * a.cache.kv_heads + line) * (uint64_t)a.max_len +
           (uint32_t)j] = total;
    } else {
        const uint64_t at = line * a.pitch + (uint32_t)j;
        if (a.before != nullptr && j < c0) total = fmaf(a.keep, a.before[at], total);
        a.weights[at] = total;
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
    const uint64_t lines = (uint64_t)a.batch.n_seqs * a.cache.kv_heads;
    float total = 0;
    for (uint32_t i = 0; i < p.splits; i++) total += ws[(i * lines + line) * (uint64_t)a.max_len + j];
    const uint64_t at = line * a.pitch + j;
    if (a.before != nullptr && (int32_t)j < c0) total = fmaf(a.keep, a.before[at], total);
    a.weights[at] = total;
}

WeighPlan plan_weigh(uint32_t q_heads, const Cache& c, uint64_t n_seqs, uint64_t n_tokens,
                     uint64_t max_len) {
    WeighPlan p;
    p.group = q_heads / c.kv_heads;
    const uint64_t rows = n_tokens * p.group;
    const uint64_t lines = n_seqs * c.kv_heads;
    // rows among the waves where a sequence has many, unless whole waves' keys
    // fill the chip
    const uint64_t wide = (max_len + kWaves * kWaveKeys - 1) / (kWaves * kWaveKeys);
    p.rows = rows >= 128 * n_seqs && wide * lines < 4 * kCus;
    p.chunks = (uint32_t)((max_len + p.tile() - 1) / p.tile());
    const uint64_t groups = p.chunks * lines;
    uint64_t splits = 2 * kCus / groups;
    const uint64_t most = rows / n_seqs / 512;  // 512 rows each at least
    splits = splits < most ? splits : most;
    p.splits = (uint32_t)(splits < 1 ? 1 : splits);
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
    if (p.rows) k_weigh<DP, CAPPED, true><<<grid, block, 0, stream>>>(a, p, score, ws);
    else k_weigh<DP, CAPPED, false><<<grid, block, 0, stream>>>(a, p, score, ws);
}

// ---- eviction --------------------------------------------------------------
//
// One workgroup for every row of weights finds which tokens stay; then the
// rows of those are copied into other pages.  Order-preserving: FP32 weights
// as unsigned numbers (NaN lowest, both zeros the same) and the key of the last
// one that stays by counting digits, eleven bits at a time, from the top;
// among equals the first ones stay.  Bound by latency: five passes over the
// weights by one workgroup.
constexpr uint32_t kPickThreads = 1024;
constexpr uint32_t kPickWaves = kPickThreads / kWave;
constexpr uint32_t kDigit = 11, kBins = 1u << kDigit, kCopies = 4;
constexpr uint32_t kRun = 8;  // consecutive weights of a thread in the last pass

__device__ __forceinline__ uint32_t rank_of(float w) {
    if (w != w) return 0;
    const uint32_t u = __float_as_uint(w + 0.0f);  // (-0 + 0 is 0)
    return u >> 31 ? ~u : u | 0x80000000u;
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

// The sum of x over the threads before this one, and over all of them
struct Scan {
    uint32_t before, all;
};
__device__ __forceinline__ Scan group_scan(uint32_t x, uint32_t* lds) {
    const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const uint32_t upto = wave_scan(x);
    __syncthreads();  // (lds has been read)
    if (lane == kWave - 1) lds[wave] = upto;
    __syncthreads();
    Scan r{upto - x, 0};
#pragma unroll
    for (uint32_t i = 0; i < kPickWaves; i++) {
        const uint32_t y = lds[i];
        if (i < wave) r.before += y;
        r.all += y;
    }
    return r;
}

__global__ __launch_bounds__(kPickThreads) void k_evict_pick(Evict a) {
    __shared__ uint32_t bins[kCopies][kBins];
    __shared__ uint32_t sums[kPickWaves];
    __shared__ uint32_t chosen[2];
    const uint32_t s = blockIdx.x / a.weight_heads, t = threadIdx.x;
    const int32_t len = a.lens[s];
    const bool good = len >= 0 && len <= a.max_len;
    const uint32_t n = good ? (uint32_t)len : 0;
    const uint32_t stay = n < a.budget ? n : a.budget;
    const float* w = a.weights + blockIdx.x * a.pitch;
    int32_t* kept = a.kept + blockIdx.x * (uint64_t)a.budget;
    float* out = a.weights_to + blockIdx.x * (uint64_t)a.budget;
    if (blockIdx.x % a.weight_heads == 0 && t == 0) a.lens_to[s] = (int32_t)stay;
    for (uint32_t i = stay + t; i < a.budget; i += kPickThreads) kept[i] = -1;
    if (n <= a.budget) {
        for (uint32_t i = t; i < n; i += kPickThreads) {
            kept[i] = (int32_t)i;
            out[i] = w[i];
        }
        return;
    }
    // the tokens between the first and the recent ones; `left` of them stay
    const uint32_t lo = a.first, hi = n - a.recent;
    const uint32_t left = a.budget - a.first - a.recent;
    uint32_t prefix = 0, mask = 0, take = left;  // of keys that match in `mask`, the top `take`
    if (left > 0) {
        for (int32_t shift = 32 - (int32_t)kDigit; shift > -(int32_t)kDigit; shift -= kDigit) {
            const uint32_t low = shift > 0 ? (uint32_t)shift : 0;
            const uint32_t width = shift > 0 ? kDigit : kDigit + (uint32_t)shift;
            for (uint32_t i = t; i < kCopies * kBins; i += kPickThreads) (&bins[0][0])[i] = 0;
            __syncthreads();
            for (uint32_t i = lo + t; i < hi; i += kPickThreads) {
                const uint32_t key = rank_of(w[i]);
                if ((key & mask) == prefix)
                    atomicAdd(&bins[t % kCopies][key >> low & ((1u << width) - 1)], 1u);
            }
            __syncthreads();
            // thread t has bins kBins - 2 t - 2 and the one above it
            uint32_t own[2];
#pragma unroll
            for (uint32_t i = 0; i < 2; i++) {
                own[i] = 0;
#pragma unroll
                for (uint32_t c = 0; c < kCopies; c++) own[i] += bins[c][kBins - 1 - 2 * t - i];
            }
            const uint32_t above = group_scan(own[0] + own[1], sums).before;
            if (above < take && above + own[0] + own[1] >= take) {
                const bool first = above + own[0] >= take;
                chosen[0] = kBins - 1 - 2 * t - (first ? 0 : 1);
                chosen[1] = take - above - (first ? 0 : own[0]);
            }
            __syncthreads();
            prefix |= chosen[0] << low;
            mask |= ((1u << width) - 1) << low;
            take = chosen[1];
            __syncthreads();
        }
    }
    // every key above `prefix` stays, and of those equal to it the first `take`
    uint32_t base = 0, ties = 0;
    for (uint32_t i0 = 0; i0 < n; i0 += kRun * kPickThreads) {
        const uint32_t first = i0 + kRun * t;
        float x[kRun];
        uint32_t sure = 0, equal = 0;
#pragma unroll
        for (uint32_t e = 0; e < kRun; e++) {
            const uint32_t i = first + e;
            x[e] = 0;
            if (i >= n) continue;
            x[e] = w[i];
            if (i < lo || i >= hi) {
                sure |= 1u << e;
            } else if (left > 0) {
                const uint32_t key = rank_of(x[e]);
                if (key > prefix) sure |= 1u << e;
                if (key == prefix) equal |= 1u << e;
            }
        }
        const Scan r = group_scan(__popc(sure) | __popc(equal) << 16, sums);
        uint32_t at = base + (r.before & 0xFFFFu);
        uint32_t rank = ties + (r.before >> 16);
        at += rank < take ? rank : take;
#pragma unroll
        for (uint32_t e = 0; e < kRun; e++) {
            bool stays = sure >> e & 1;
            if (equal >> e & 1) {
                stays = rank < take;
                rank++;
            }
            if (stays) {
                kept[at] = (int32_t)(first + e);
                out[at] = x[e];
                at++;
            }
        }
        base += r.all & 0xFFFFu;
        ties += r.all >> 16;
    }
}

// Copies kept rows, 16 destination tokens and all heads a workgroup: LANES
// lanes a row, 16 bytes each.
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
