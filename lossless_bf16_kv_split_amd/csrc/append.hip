// append.hip -- norms and rotation of queries and keys, and the append of
// new tokens' keys and values to a paged cache.
//
// For a head row x of D elements and a token at position p:
//   y = x / sqrt(mean(x^2) + eps) * weight           (with a weight)
//   (a, b) -> m (a cos t - b sin t), m (b cos t + a sin t)
// for each pair (a, b) = (y_i, y_{i+R/2}) or (y_2i, y_{2i+1}), i < R/2, with
// the angle t = p * phase_i / 2^64 turns.  FP32 throughout, one rounding to
// BF16 at the store.
//
// The angle is exact: p * phase_i modulo 2^64 is the fraction of a turn in
// fixed point, whatever p, and its top 32 bits carry an error below 2^-32
// turns.  No table is read.
//
// Bound by the bytes of the rows, and for few tokens by latency.  A row
// lies across 8 to 64 lanes of a wave, each with 8 (or 4) consecutive
// elements; a wave works on one token, computes that token's angles once
// and walks rows of it.
#include "kv_internal.h"

#include <cstdint>

namespace sz {
namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kWavesPerGroup = kThreads / kWave;
// A token's rows are shared among several waves until there are this many
// of them, twice what 256 CUs hold at once: fewer leave rows in a queue
// behind their wave's loads, more work out the token's angles too often
// (8192 tokens' 72 rows from 32 bits, normed: 94 us with 4096, 87 with
// 16384, 84 with 32768, 89 with 65536; their 48 rows of BF16 into the cache:
// 42, 42, 44, 58).  Stores stay cached: attention reads the rows next
// (non-temporal ones save 3 to 5% of this kernel).
constexpr uint64_t kFillWaves = 16384;
// Tokens of a launch, a wave each where there are so many
constexpr uint64_t kMostTokens = uint64_t{1} << 25;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// cos and sin of a / 2^32 turns: the hardware's own, which take turns (off
// by at most 1.3e-7 over the whole circle, measured against 64 bits)
__device__ __forceinline__ void turn_of(uint32_t a, float& c, float& s) {
    const float turns = (float)(int32_t)a * 0x1p-32f;
    c = __builtin_amdgcn_cosf(turns);
    s = __builtin_amdgcn_sinf(turns);
}

// VEC elements of a row from element e of it, as floats
template <int VEC>
__device__ __forceinline__ void load_row(const Rows& r, uint64_t at, float (&x)[VEC]) {
    if (r.f32) {
        const float* p = static_cast<const float*>(r.data) + at;
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            const uint4 w = load_global(reinterpret_cast<const uint4*>(p + i));
            x[i] = __uint_as_float(w.x);
            x[i + 1] = __uint_as_float(w.y);
            x[i + 2] = __uint_as_float(w.z);
            x[i + 3] = __uint_as_float(w.w);
        }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(r.data) + at;
        uint32_t w[VEC / 2];
        if constexpr (VEC == 8) {
            const uint4 v = load_global(reinterpret_cast<const uint4*>(p));
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
            const u32x2 v = *(const SZ_GLOBAL u32x2*)p;
            w[0] = v.x, w[1] = v.y;
        }
#pragma unroll
        for (int i = 0; i < VEC / 2; i++) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

template <int VEC>
__device__ __forceinline__ void store_words(uint16_t* p, const uint32_t (&w)[VEC / 2]) {
    if constexpr (VEC == 8) {
        store_global(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
    } else {
        const u32x2 v = {w[0], w[1]};
        *(SZ_GLOBAL u32x2*)p = v;
    }
}

template <int VEC>
__device__ __forceinline__ void store_row(uint16_t* p, const float (&x)[VEC]) {
    uint32_t w[VEC / 2];
#pragma unroll
    for (int i = 0; i < VEC / 2; i++) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
    store_words<VEC>(p, w);
}

enum { kNoTurn = 0, kHalves = 1, kInterleaved = 2 };

// LANES lanes hold a row, VEC elements each; slices waves share a token.
template <int LANES, int VEC, int MODE, bool APPEND>
__global__ __launch_bounds__(kThreads) void k_turn(TurnRows a, Cache cache, Batch batch,
                                                   uint32_t slices, uint32_t first) {
    constexpr uint32_t kRows = kWave / LANES;  // rows a wave holds at once
    const uint32_t lane = threadIdx.x % kWave;
    const uint64_t wave =
        (uint64_t)blockIdx.x * kWavesPerGroup + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint64_t token = first + wave / slices;
    const uint32_t slice = (uint32_t)(wave % slices);
    if (token >= a.n_tokens) return;

    // where the token goes in the cache
    uint64_t k_page = 0, v_page = 0, slot = 0;
    int32_t position = 0;
    if constexpr (APPEND) {
        const uint32_t s = find_seq(batch.n_seqs, (int64_t)token,
                                    [&](uint32_t i) { return (int64_t)batch.starts[i]; });
        const Seq q = load_seq(batch, s, (int64_t)(cache.pages_per_seq << cache.page_log2));
        if (!q.good || (int64_t)token < q.begin || (int64_t)token >= q.end) return;
        const int64_t c = (int64_t)q.len - q.end + (int64_t)token;
        if (c < 0) return;
        const uint64_t entry = (uint64_t)s * cache.table_pitch + ((uint64_t)c >> cache.page_log2);
        k_page = cache.k_pages[entry];
        v_page = cache.v_pages[entry];
        slot = ((uint64_t)c & ((1u << cache.page_log2) - 1)) * cache.token_stride;
        position = (int32_t)c;
    }
    if (MODE != kNoTurn && a.positions != nullptr) position = a.positions[token];

    const uint32_t l = lane % LANES;
    const uint32_t e = l * VEC;  // this lane's first element
    const bool live = e < a.head_dim;
    // the lane's angles
    constexpr int kAngles = MODE == kInterleaved ? VEC / 2 : VEC;
    float c[kAngles], sn[kAngles];
    const uint32_t half = a.turn.dims / 2;
    const bool turns = MODE != kNoTurn && e < a.turn.dims;
    const bool lower = e < half;
    uint32_t partner = lane;
    if (MODE == kHalves && turns) partner = lower ? lane + half / VEC : lane - half / VEC;
    if (turns) {
        const uint32_t first = MODE == kInterleaved ? e / 2 : lower ? e : e - half;
        const uint32_t far = position < 0 ? 0u - (uint32_t)position : (uint32_t)position;
#pragma unroll
        for (int i = 0; i < kAngles; i++) {
            const uint64_t turn = (uint64_t)far * a.turn.phases[first + i];
            turn_of((uint32_t)(turn >> 32), c[i], sn[i]);
            c[i] *= a.turn.magnitude;
            sn[i] *= position < 0 ? -a.turn.magnitude : a.turn.magnitude;
            if (MODE == kHalves && lower) sn[i] = -sn[i];
        }
    }

    // the rows of queries and keys, the next one's load under way
    const uint32_t turned = a.q.heads + a.k.heads;
    const uint32_t stride = slices * kRows;
    const auto load = [&](uint32_t r, float (&x)[VEC]) {
        const bool is_k = r >= a.q.heads;
        const Rows& src = is_k ? a.k : a.q;
        const uint32_t h = is_k ? r - a.q.heads : r;
        if (live && r < turned)
            load_row<VEC>(src, token * src.token_stride + h * src.head_stride + e, x);
    };
    float next[VEC] = {};
    load(slice * kRows + lane / LANES, next);
    for (uint32_t r0 = slice * kRows; r0 < turned; r0 += stride) {
        const uint32_t r = r0 + lane / LANES;
        const bool is_k = r >= a.q.heads;
        const uint32_t h = is_k ? r - a.q.heads : r;
        const bool on = live && r < turned;
        float x[VEC];
#pragma unroll
        for (int i = 0; i < VEC; i++) x[i] = next[i];
        load(r + stride, next);
        const float* weight = is_k ? a.k_weight : a.q_weight;
        float sum = 0;
#pragma unroll
        for (int i = 0; i < VEC; i++) sum = fmaf(x[i], x[i], sum);
#pragma unroll
        for (int d = 1; d < LANES; d *= 2) sum += __shfl_xor(sum, d);
        if (weight != nullptr && on) {
            const float inv = 1.0f / sqrtf(sum / (float)a.head_dim + a.eps);
#pragma unroll
            for (int i = 0; i < VEC; i++) x[i] = x[i] * inv * weight[e + i];
        }
        if constexpr (MODE == kHalves) {
#pragma unroll
            for (int i = 0; i < VEC; i++) {
                const float other = __shfl(x[i], partner);
                if (turns) x[i] = fmaf(x[i], c[i], other * sn[i]);
            }
        } else if constexpr (MODE == kInterleaved) {
            if (turns) {
#pragma unroll
                for (int i = 0; i < VEC / 2; i++) {
                    const float u = x[2 * i], v = x[2 * i + 1];
                    x[2 * i] = fmaf(u, c[i], -v * sn[i]);
                    x[2 * i + 1] = fmaf(v, c[i], u * sn[i]);
                }
            }
        }
        if (on) {
            if (APPEND && is_k) {
                if (good_page(k_page))
                    store_row<VEC>(reinterpret_cast<uint16_t*>(k_page) + slot +
                                       h * cache.head_stride + e, x);
            } else {
                const Rows& dst = is_k ? a.k_out : a.q_out;
                store_row<VEC>(static_cast<uint16_t*>(dst.data) + token * dst.token_stride +
                                   h * dst.head_stride + e, x);
            }
        }
    }
    if constexpr (APPEND) {
        for (uint32_t h0 = slice * kRows; h0 < a.v.heads; h0 += slices * kRows) {
            const uint32_t h = h0 + lane / LANES;
            if (!live || h >= a.v.heads || !good_page(v_page)) continue;
            const uint64_t at = token * a.v.token_stride + h * a.v.head_stride + e;
            uint16_t* to = reinterpret_cast<uint16_t*>(v_page) + slot + h * cache.head_stride + e;
            if (a.v.f32) {
                float x[VEC];
                load_row<VEC>(a.v, at, x);
                store_row<VEC>(to, x);
            } else {  // the words as they are
                const uint16_t* p = static_cast<const uint16_t*>(a.v.data) + at;
                if constexpr (VEC == 8) {
                    store_global(reinterpret_cast<uint4*>(to),
                                 load_global(reinterpret_cast<const uint4*>(p)));
                } else {
                    *(SZ_GLOBAL u32x2*)to = *(const SZ_GLOBAL u32x2*)p;
                }
            }
        }
    }
}

template <int LANES, int VEC, int MODE, bool APPEND>
hipError_t go(const TurnRows& a, const Cache& cache, const Batch& batch, hipStream_t stream) {
    const uint64_t rows = a.q.heads + a.k.heads + (uint64_t)a.v.heads;
    const uint64_t most = (rows + kWave / LANES - 1) / (kWave / LANES);
    uint64_t slices = (kFillWaves + a.n_tokens - 1) / a.n_tokens;
    slices = slices < 1 ? 1 : slices > most ? most : slices;
    // (a launch holds fewer than 2^32 threads)
    for (uint64_t first = 0; first < a.n_tokens; first += kMostTokens) {
        const uint64_t tokens = a.n_tokens - first < kMostTokens ? a.n_tokens - first : kMostTokens;
        const uint64_t groups = (tokens * slices + kWavesPerGroup - 1) / kWavesPerGroup;
        k_turn<LANES, VEC, MODE, APPEND><<<dim3((uint32_t)groups), dim3(kThreads), 0, stream>>>(
            a, cache, batch, (uint32_t)slices, (uint32_t)first);
        if (hipError_t e = hipGetLastError()) return e;
    }
    return hipSuccess;
}

// Lanes per row: the least power of two that holds it.  A lane's elements
// must not straddle the halves: 8 a lane where rotary_dim / 2 is a multiple
// of 8 (or pairs are interleaved), else 4.
template <int MODE, bool APPEND>
hipError_t pick(const TurnRows& a, const Cache& cache, const Batch& batch, hipStream_t stream) {
    const uint32_t d = a.head_dim;
    if constexpr (MODE == kHalves) {
        if (a.turn.dims % 16 != 0) {
            if (d <= 64) return go<16, 4, MODE, APPEND>(a, cache, batch, stream);
            if (d <= 128) return go<32, 4, MODE, APPEND>(a, cache, batch, stream);
            return go<64, 4, MODE, APPEND>(a, cache, batch, stream);
        }
    }
    if (d <= 64) return go<8, 8, MODE, APPEND>(a, cache, batch, stream);
    if (d <= 128) return go<16, 8, MODE, APPEND>(a, cache, batch, stream);
    return go<32, 8, MODE, APPEND>(a, cache, batch, stream);
}

template <bool APPEND>
hipError_t launch(const TurnRows& a, const Cache& cache, const Batch& batch, hipStream_t stream) {
    if (a.n_tokens == 0) return hipSuccess;
    if (a.turn.dims == 0) return pick<kNoTurn, APPEND>(a, cache, batch, stream);
    if (a.turn.interleaved) return pick<kInterleaved, APPEND>(a, cache, batch, stream);
    return pick<kHalves, APPEND>(a, cache, batch, stream);
}

// Sequences are found by a search over their starts, which finds one's rows
// for certain where no start before its own lies above it and none after
// lies below its end.  A wave takes `each` (at most 32) sequences: it reads
// all starts once, 64 at a time, and compares its own among themselves.
__global__ __launch_bounds__(kWave) void k_check_seqs(SeqCheck c, uint32_t each) {
    const uint32_t lane = threadIdx.x, s0 = blockIdx.x * each, n = c.batch.n_seqs;
    const uint32_t s1 = n - s0 < each ? n : s0 + each;
    int32_t top = INT32_MIN, low = INT32_MAX;
    for (uint32_t i = lane; i <= n; i += kWave) {
        const int32_t x = c.batch.starts[i];
        if (i < s0) top = x > top ? x : top;
        if (i > s1) low = x < low ? x : low;
    }
    const int32_t own = s0 + lane <= s1 ? c.batch.starts[s0 + lane] : 0;
    for (uint32_t s = s0; s < s1; s++) {
        const Seq q = load_seq(c.batch, s, c.max_len);
        bool good = q.good && top <= q.begin && low >= q.end;
        if (s0 + lane <= s1) good = good && (s0 + lane <= s ? own <= q.begin : own >= q.end);
        if (good) {
            const int64_t first_new = (int64_t)q.len - (q.end - q.begin);
            int64_t from = 0;
            if (c.append) {
                if (first_new < 0) good = false;
                from = first_new;
            } else if (c.causal && c.window != 0 && (uint64_t)first_new + 1 > c.window &&
                       first_new >= 0) {
                from = first_new + 1 - (int64_t)c.window;
            }
            if (good && q.begin < q.end && from < q.len) {
                const uint64_t row = (uint64_t)s * c.cache.table_pitch;
                const uint64_t last = (uint64_t)(q.len - 1) >> c.cache.page_log2;
                for (uint64_t p = ((uint64_t)from >> c.cache.page_log2) + lane; p <= last;
                     p += kWave)
                    good = good && good_page(c.cache.k_pages[row + p]) &&
                           good_page(c.cache.v_pages[row + p]);
            }
        }
        const bool all = __ballot(!good) == 0;
        if (lane == 0) c.status[s] = all ? kSeqGood : kBlockInvalid;
    }
}

}  // namespace

hipError_t launch_turn(const TurnRows& a, hipStream_t stream) {
    return launch<false>(a, Cache{}, Batch{}, stream);
}

hipError_t launch_append(const TurnRows& a, const Cache& cache, const Batch& batch,
                         hipStream_t stream) {
    if (batch.n_seqs == 0) return hipSuccess;
    return launch<true>(a, cache, batch, stream);
}

hipError_t launch_check_seqs(const SeqCheck& c, hipStream_t stream) {
    if (c.batch.n_seqs == 0) return hipSuccess;
    const uint32_t each = (c.batch.n_seqs + 2047) / 2048;
    k_check_seqs<<<dim3((c.batch.n_seqs + each - 1) / each), dim3(kWave), 0, stream>>>(c, each);
    return hipGetLastError();
}

}  // namespace sz
