// latent.hip -- attention over a paged cache of latents, the absorbed form.
//
// A cached token j is one row c_j of latent_dim + rotary_dim elements, a key
// of every query head, and its first latent_dim elements are the value:
//   s_j = scale * q.c_j,  p_j = exp(s_j - m),  o = sum p_j c_j[:latent_dim] / sum p_j
// for the keys j that a row sees.  All heads of a token read the same rows, so
// the rows of a sequence are (token, head) pairs, cut into tiles as in
// attend_parts.h with one KV head.
//
// Both products run on the matrix cores, S^T = C Q^T and O^T = C^T P^T, from
// the same copy of the keys in LDS: what is loaded once is read as keys and,
// transposed by the LDS reads, as values.
#include "attend_parts.h"

namespace sz {
namespace {

constexpr int kKeys = 64;  // of a step
constexpr uint64_t kCus = 256;

// A workgroup's four waves: RW groups of 32 rows, each KW waves that share
// its keys (in blocks of 32) and its elements of the output.
template <int DL, int DT, int RW>
struct Shape {
    static constexpr int kKw = 4 / RW;
    static constexpr uint32_t kRow = 2 * DT;              // bytes of a row in LDS
    static constexpr uint32_t kBuffer = kKeys * kRow;     // of a step's keys
    static constexpr int kLoads = DT / 32;                // KB that a wave fetches of them
    static constexpr int kSlices = DT / 16;               // of the first product
    static constexpr int kParts = DL / 32 / kKw;          // of the second, a wave's
    static constexpr int kBlocks = kKw == 1 ? 2 : 1;      // of 32 keys, a wave's scores
    static constexpr uint32_t kWeights = 2 * kBuffer;     // LDS: weights [RW][2][2][64 lanes][16 B]
    static constexpr uint32_t kTops = kWeights + (kKw > 1 ? RW * 4096 : 0);  // [RW][2][32] floats
    static constexpr uint32_t kLds = kTops + (kKw > 1 ? RW * 256 : 0);
    static_assert(kRow % 256 == 128, "rows start at alternating halves of the banks");
    static_assert(kLds <= 160 * 1024, "");
};

// 16-byte piece c of a step's key j lies at c ^ mix(j).  Rows being an odd
// multiple of 128 bytes, 16 keys' same piece then fall on 16 different places of
// the 256 bytes that LDS serves at once, and 64 consecutive bytes of four keys
// on four different quarters.
__device__ __forceinline__ constexpr uint32_t mix(uint32_t j) {
    return (j >> 1 & 1) << 2 | (j >> 2 & 1) << 1 | (j >> 3 & 1);
}

template <int N>
__device__ __forceinline__ void fetch_rows(__amdgpu_buffer_rsrc_t from, const uint32_t* at,
                                           uint32_t lds) {
    if constexpr (N >= 8) {
        load_to_lds<8>(from, at, lds);
        if constexpr (N > 8) fetch_rows<N - 8>(from, at + 8, lds + 8 * 1024);
    } else {
        load_to_lds<N>(from, at, lds);
    }
}

__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

template <int DL, int DT, int RW>
__device__ __forceinline__ void latent_part(const Attend& a, const AttendPlan& p, float by,
                                            uint8_t* ws, const Part& part, uint8_t* lds) {
    using S = Shape<DL, DT, RW>;
    constexpr int kKw = S::kKw, kParts = S::kParts, kBlocks = S::kBlocks;
    constexpr uint32_t kRow = S::kRow;
    const uint32_t lane = threadIdx.x % kWave, n = lane % 32, h = lane / 32;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t rw = wave / kKw, kw = wave % kKw;
    const Tile& t = part.t;
    const int32_t first = part.first, last = part.last;
    const uint32_t dim = a.cache.head_dim;

    // the row's query
    const Row mine = find_row(a, p, t, (int32_t)(32 * rw + n));
    bf16x8 q[S::kSlices];
    {
        const uint16_t* row = static_cast<const uint16_t*>(a.q.data) +
                              (uint64_t)mine.token * a.q.token_stride +
                              (uint64_t)mine.head * a.q.head_stride;
#pragma unroll
        for (int s = 0; s < S::kSlices; s++) {
            u32x4 v = {0, 0, 0, 0};
            if (mine.on && 16 * s + 8 * h < dim)
                v = *(const SZ_GLOBAL u32x4*)(row + 16 * s + 8 * h);
            q[s] = __builtin_bit_cast(bf16x8, v);
        }
    }
    const bool works = 32 * (int32_t)rw < t.rows;

    // this wave's part of a step: 16 keys
    constexpr uint32_t kPast = 0x80000000u;
    const uint32_t step = 2 * (uint32_t)a.cache.token_stride;
    uint32_t off[S::kLoads];
#pragma unroll
    for (int i = 0; i < S::kLoads; i++) {
        const uint32_t at = 1024 * i + 16 * lane, row = at / kRow;
        const uint32_t piece = at % kRow / 16 ^ mix(row);
        off[i] = 8 * piece < dim ? row * step + 16 * piece : kPast;
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)(SZ_LDS uint8_t*)lds;
    const uint64_t table_row = (uint64_t)t.seq * a.cache.table_pitch;
    const auto page_at = [&](int32_t j) {
        const int32_t jb = j + 16 * (int32_t)wave;
        return jb < last ? a.cache.k_pages[table_row + ((uint32_t)jb >> a.cache.page_log2)] : 0;
    };
    uint64_t next_page = page_at(first);
    const auto fetch = [&](int32_t j, uint32_t buffer) {
        const int32_t jb = j + 16 * (int32_t)wave;
        const uint32_t slot = (uint32_t)jb & ((1u << a.cache.page_log2) - 1);
        const uint64_t at =
            (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(next_page >> 32)) << 32 |
            (uint32_t)__builtin_amdgcn_readfirstlane((int)next_page);
        const auto rows = block_rows(a.cache, at, slot, 0, last - jb);
        fetch_rows<S::kLoads>(rows, off, lds0 + buffer * S::kBuffer + wave * 16 * kRow);
        next_page = page_at(j + kKeys);
    };

    // LDS addresses of this lane's reads.  Slice s of the keys: the first
    // one's address with bits 5 and 6 turned over by s % 4, and s / 4 times 128
    // bytes on; part d of the values with bit 6 by d % 2, and d / 2 times 128.
    const uint32_t k_lane = lds0 + n * kRow + (h ^ mix(n)) * 16;
    const uint32_t v_key = lane % 16 / 4;
    const uint32_t v_lane = lds0 + (4 * h + v_key) * kRow +
                            ((2 * (lane / 16 % 2) + lane % 4 / 2) ^ mix(4 * h + v_key)) * 16 +
                            lane % 2 * 8;
    const auto keys_at = [&](uint32_t at, int s) {
        return *(const SZ_LDS bf16x8*)(uintptr_t)((at ^ 32 * (s % 4)) + 128 * (s / 4));
    };
    // (keys 8 and more on have the lowest bit of the permutation set)
    const auto value_words = [&](uint32_t at, int t16, int d) {
        const uint32_t x0 = (at ^ 64 * (d % 2)) + 128 * (d / 2) + 16 * t16 * kRow;
        const uint32_t y0 = (at ^ (64 * (d % 2) + 16)) + 128 * (d / 2) + (16 * t16 + 8) * kRow;
        const u32x2 x = __builtin_bit_cast(
            u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((SZ_LDS s16x4*)(uintptr_t)x0));
        const u32x2 y = __builtin_bit_cast(
            u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((SZ_LDS s16x4*)(uintptr_t)y0));
        return u32x4{x.x, x.y, y.x, y.y};
    };

    float m = kNoKey, l = 0;
    f32x16 o[kParts];
#pragma unroll
    for (int d = 0; d < kParts; d++)
#pragma unroll
        for (int i = 0; i < 16; i++) o[d][i] = 0;

    const auto follow = [&](float top) {  // (the same top in both of a row's lanes)
        if (__ballot(top > m + kLag) == 0) return;
        top = fmaxf(top, m);
        const float keep = __builtin_amdgcn_exp2f(m - top);
        m = top;
        l *= keep;
#pragma unroll
        for (int d = 0; d < kParts; d++)
#pragma unroll
            for (int i = 0; i < 16; i++) o[d][i] *= keep;
    };

    const uint32_t my_weights = lds0 + S::kWeights + rw * 4096 + 16 * lane;
    const uint32_t my_tops = lds0 + S::kTops + rw * 256 + 4 * n;

    const auto compute = [&](int32_t j, uint32_t buffer) {
        const bool edge = j + kKeys > t.all_hi;
        const uint32_t ka = k_lane + buffer * S::kBuffer;
        f32x16 s[kBlocks];
        float top = -INFINITY;
        const uint32_t block0 = kKw == 1 ? 0 : kw % 2;
        if (works) {
#pragma unroll
            for (int b = 0; b < kBlocks; b++) {
#pragma unroll
                for (int i = 0; i < 16; i++) s[b][i] = 0;
#pragma unroll
                for (int c = 0; c < S::kSlices; c++) {
                    s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        keys_at(ka + (block0 + b) * 32 * kRow, c), q[c], s[b], 0, 0, 0);
                    if (c % 6 == 5) __builtin_amdgcn_sched_barrier(0);
                }
                if (edge) {
                    const Sees sees(0, mine.high, j + 32 * (int32_t)(block0 + b) + 4 * (int32_t)h);
#pragma unroll
                    for (int i = 0; i < 16; i++)
                        if (!sees(8 * (i / 4) + i % 4)) s[b][i] = -INFINITY;
                }
#pragma unroll
                for (int i = 0; i < 16; i++) top = fmaxf(top, s[b][i]);
            }
            top *= by;
            top = fmaxf(top, __shfl_xor(top, 32));
        }
        if constexpr (kKw > 1) {
            if (works && kw < 2 && h == 0)
                *(SZ_LDS float*)(uintptr_t)(my_tops + 128 * kw) = top;
            lds_barrier();
            if (works) top = fmaxf(top, *(const SZ_LDS float*)(uintptr_t)(my_tops + 128 * (1 - block0)));
        }
        u32x4 w[4];  // weights of 16 keys each
        if (works) {
            follow(top);
#pragma unroll
            for (int b = 0; b < kBlocks; b++) {
                uint32_t x[8];
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float u = __builtin_amdgcn_exp2f(fmaf(s[b][i], by, -m));
                    const float v = __builtin_amdgcn_exp2f(fmaf(s[b][i + 1], by, -m));
                    l += u + v;
                    x[i / 2] = pack_bf16(u, v);
                }
                w[2 * b] = u32x4{x[0], x[1], x[2], x[3]};
                w[2 * b + 1] = u32x4{x[4], x[5], x[6], x[7]};
            }
        }
        if constexpr (kKw > 1) {
            if (works && kw < 2) {
                *(SZ_LDS u32x4*)(uintptr_t)(my_weights + 2048 * kw) = w[0];
                *(SZ_LDS u32x4*)(uintptr_t)(my_weights + 2048 * kw + 1024) = w[1];
            }
            lds_barrier();
            if (works) {
#pragma unroll
                for (int i = 0; i < 4; i++)
                    w[i] = *(const SZ_LDS u32x4*)(uintptr_t)(my_weights + 1024 * i);
            }
        }
        if (!works) return;
        const uint32_t va = v_lane + buffer * S::kBuffer + kw * kParts * 64;
        // keys that some row of the tile sees and another does not: an
        // infinity or a NaN among them must not reach the rows that do not
        // see it, where 0 times it would be NaN.  The values go in without it;
        // rows that see it get NaN for it (their score with it is infinite or
        // NaN, and so is its weight times it), by a product of ones in its
        // place with what each row sees.
        const bool rim = edge && t.all_hi < last;
        uint32_t halves = 0;
#pragma unroll
        for (int t16 = 0; t16 < 4; t16++)
#pragma unroll
            for (int d = 0; d < kParts; d++) {
                u32x4 x = value_words(va, t16, d);
                if (rim) {
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        halves |= odd_halves(x[i]);
                        x[i] = plain_pair(x[i]);
                    }
                }
                o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                    __builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, w[t16]), o[d], 0, 0,
                    0);
                // (or operands are read far ahead, into registers that are not there)
                if (d % 4 == 3) __builtin_amdgcn_sched_barrier(0);
            }
        if (__ballot(any_odd(halves)) == 0) return;
        const Sees sees(0, mine.high, j + 4 * (int32_t)h);
#pragma unroll 1
        for (int t16 = 0; t16 < 4; t16++) {
            u32x4 seen;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint32_t key = 16 * t16 + 8 * (i / 2) + 2 * (i % 2);
                seen[i] = (sees(key) ? 0x3F80u : 0u) | (sees(key + 1) ? 0x3F800000u : 0u);
            }
#pragma unroll
            for (int d = 0; d < kParts; d++) {
                u32x4 x = value_words(va, t16, d);
#pragma unroll
                for (int i = 0; i < 4; i++)
                    x[i] = ((odd_halves(x[i]) >> 15) & 0x00010001u) * 0x3F80u;  // ones
                if (__ballot((x.x | x.y | x.z | x.w) != 0) == 0) continue;
                f32x16 z;
#pragma unroll
                for (int i = 0; i < 16; i++) z[i] = 0;
                z = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x),
                                                            __builtin_bit_cast(bf16x8, seen), z, 0,
                                                            0, 0);
#pragma unroll
                for (int i = 0; i < 16; i++) o[d][i] += z[i] > 0 ? NAN : 0.0f;
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };

    const auto arrived = [&] {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    };
    const int32_t steps = first < last ? (last - first + kKeys - 1) / kKeys : 0;
    arrived();  // (every wave is done with the part before)
    if (steps > 0) fetch(first, 0);
    for (int32_t x = 0; x < steps; x++) {
        arrived();
        if (x + 1 < steps) fetch(first + (x + 1) * kKeys, (x + 1) & 1);
        compute(first + x * kKeys, x & 1);
    }

    float total = l + __shfl_xor(l, 32);
    if constexpr (kKw > 1) {
        // each of two waves has the sum over its block of every step's keys
        lds_barrier();
        if (kw < 2 && h == 0) *(SZ_LDS float*)(uintptr_t)(my_tops + 128 * kw) = total;
        lds_barrier();
        total += *(const SZ_LDS float*)(uintptr_t)(my_tops + 128 * (1 - kw % 2));
    }
    if (!mine.on) return;
    if (part.alone) {
        const float inv = inverse(total);
        const uint64_t at = (uint64_t)mine.token * a.out.token_stride +
                            (uint64_t)mine.head * a.out.head_stride;
#pragma unroll
        for (int d = 0; d < kParts; d++)
#pragma unroll
            for (int g = 0; g < 4; g++) {
                const uint32_t e = 32 * (kw * kParts + d) + 8 * g + 4 * h;
                const float x[4] = {o[d][4 * g] * inv, o[d][4 * g + 1] * inv,
                                    o[d][4 * g + 2] * inv, o[d][4 * g + 3] * inv};
                if (e < a.value_dim) store_out<4>(a.out, at + e, x);
            }
        if (h == 0 && kw == 0 && a.lse != nullptr)
            a.lse[(uint64_t)mine.token * a.q.heads + mine.head] = log_sum(m, total);
    } else {
        const Partial u = partial_of(ws, a, p, 0, part.slot);
        const uint32_t r = 32 * rw + n;
#pragma unroll
        for (int d = 0; d < kParts; d++)
#pragma unroll
            for (int g = 0; g < 4; g++) {
                const uint32_t e = 32 * (kw * kParts + d) + 8 * g + 4 * h;
                if (e < a.value_dim)
                    store_global(reinterpret_cast<uint4*>(u.o + (uint64_t)r * a.value_dim + e),
                                 make_uint4(__float_as_uint(o[d][4 * g]),
                                            __float_as_uint(o[d][4 * g + 1]),
                                            __float_as_uint(o[d][4 * g + 2]),
                                            __float_as_uint(o[d][4 * g + 3])));
            }
        if (h == 0 && kw == 0) {
            u.ml[2 * r] = m;
            u.ml[2 * r + 1] = total;
        }
    }
}

template <int DL, int DT, int RW, bool SHARED>
__global__ __launch_bounds__(kThreads, 1) void k_attend_latent(Attend a, AttendPlan p, float by,
                                                               uint8_t* ws) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[Shape<DL, DT, RW>::kLds];
    const uint32_t index = blockIdx.x;
    Walk<SHARED> walk(a, p);
    Part part;
    if (!walk.first(a, p, SHARED ? index : p.tiles - 1 - index, part)) return;
    do {
        latent_part<DL, DT, RW>(a, p, by, ws, part, lds);
    } while (walk.next(a, p, index, part));
}

// Joins the parts of the tiles that were cut: a wave a row, eight elements a
// lane; the parts' maxima and sums 64 at a time, one a lane.
__global__ __launch_bounds__(kThreads) void k_latent_join(Attend a, AttendPlan p, uint8_t* ws) {
    const uint32_t lane = threadIdx.x % kWave;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t pieces = (1u << p.tile_log2) / kWaves;
    const uint32_t number = blockIdx.x / pieces;
    const Shares shares(a, p);
    if (number >= Shares::from_lane(shares.tiles1, kWave - 1)) return;
    const Shares::Found f = shares.find(a, p, true, number);
    const uint32_t at = number - f.tiles0;
    const uint32_t step = f.steps0 + at * f.x.steps;
    const uint32_t from = step / shares.quota, upto = (step + f.x.steps - 1) / shares.quota;
    if (from == upto) return;
    const Tile t = make_tile(a, p, f.seq, number, f.x.q, (int64_t)at << p.tile_log2);
    const int32_t r = (int32_t)(blockIdx.x % pieces * kWaves + wave);
    if (r >= t.rows) return;
    const Row w = find_row(a, p, t, r);
    const uint32_t e = 8 * lane;
    const bool on = e < a.value_dim;
    const uint64_t stride = (uint64_t)a.value_dim << p.tile_log2;
    float top = kNoKey, total = 0, x[8] = {};
    for (uint32_t i0 = from; i0 <= upto; i0 += kWave) {
        const uint32_t parts = upto - i0 + 1 < kWave ? upto - i0 + 1 : kWave;
        const Partial u = partial_of(ws, a, p, 0, i0 + number);
        float m = kNoKey, l = 0;
        if (lane < parts) {
            m = u.ml[2 * (((uint64_t)lane << p.tile_log2) + r)];
            l = u.ml[2 * (((uint64_t)lane << p.tile_log2) + r) + 1];
        }
        const float most = wave_max(fmaxf(m, top));
        const float weight = __builtin_amdgcn_exp2f(m - most);
        const float keep = __builtin_amdgcn_exp2f(top - most);
        top = most;
        total = total * keep + wave_sum(l * weight);
#pragma unroll
        for (int i = 0; i < 8; i++) x[i] *= keep;
        const float* o = u.o + (uint64_t)r * a.value_dim + e;
        constexpr uint32_t kBatch = 4;
        for (uint32_t s0 = 0; s0 < parts; s0 += kBatch) {
            f32x4 v[kBatch][2];
#pragma unroll
            for (uint32_t k = 0; k < kBatch; k++)
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    v[k][i] = f32x4{0, 0, 0, 0};
                    if (on && s0 + k < parts)
                        v[k][i] = *(const SZ_GLOBAL f32x4*)(o + (s0 + k) * stride + 4 * i);
                }
#pragma unroll
            for (uint32_t k = 0; k < kBatch; k++) {
                const float by = __int_as_float(
                    __builtin_amdgcn_readlane(__float_as_int(weight), (s0 + k) % kWave));
#pragma unroll
                for (int i = 0; i < 8; i++)
                    if (s0 + k < parts) x[i] = fmaf(v[k][i / 4][i % 4], by, x[i]);
            }
        }
    }
    const float inv = inverse(total);
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] *= inv;
    if (on)
        store_out<8>(a.out, (uint64_t)w.token * a.out.token_stride +
                                (uint64_t)w.head * a.out.head_stride + e, x);
    if (lane == 0 && a.lse != nullptr)
        a.lse[(uint64_t)w.token * a.q.heads + w.head] = log_sum(top, total);
}

// Tiles of 32 or 64 rows by what sequences have on average; whole where
// they fill the chip or have few keys, shared out among one workgroup a CU
// otherwise (attend_parts.h).
constexpr uint64_t kManyTiles = 1024;
constexpr uint64_t kWholeKeys = 256;
constexpr uint64_t kShareSeqs = 1024;
constexpr uint64_t kMostSteps = uint64_t{1} << 30;

AttendPlan plan_latent(uint32_t heads, uint64_t n_seqs, uint64_t n_tokens, uint64_t max_len) {
    AttendPlan p{};
    p.group = heads;
    const uint64_t rows = n_tokens * heads;
    p.tile_log2 = rows <= 32 * n_seqs ? 5 : 6;
    p.tiles = (uint32_t)((rows >> p.tile_log2) + n_seqs);
    const uint64_t full = rows >> p.tile_log2;
    const bool whole = n_seqs > kShareSeqs || (full > n_seqs ? full : n_seqs) >= kManyTiles ||
                       p.tiles * (max_len / kStep + 2) >= kMostSteps || max_len <= kWholeKeys;
    p.shares = whole ? 0 : (uint32_t)kCus;
    p.alone = (uint32_t)kCus;
    return p;
}

template <int DL, int DT, int RW>
void go(const Attend& a, const AttendPlan& p, float by, uint8_t* ws, hipStream_t stream) {
    const dim3 block(kThreads);
    if (p.shares != 0)
        k_attend_latent<DL, DT, RW, true><<<dim3(p.shares), block, 0, stream>>>(a, p, by, ws);
    else
        k_attend_latent<DL, DT, RW, false><<<dim3(p.tiles), block, 0, stream>>>(a, p, by, ws);
}

template <int DL, int DT>
void go(const Attend& a, const AttendPlan& p, float by, uint8_t* ws, hipStream_t stream) {
    if (p.tile_log2 == 5) go<DL, DT, 1>(a, p, by, ws, stream);
    else go<DL, DT, 2>(a, p, by, ws, stream);
}

}  // namespace

uint64_t attend_latent_workspace(uint32_t heads, const Cache&, uint32_t latent_dim,
                                 uint64_t n_seqs, uint64_t n_tokens, uint64_t max_len) {
    const AttendPlan p = plan_latent(heads, n_seqs, n_tokens, max_len);
    if (p.shares == 0) return 0;
    const uint64_t rows = partial_slots(p) << p.tile_log2;
    return (rows * (latent_dim + 2) * 4 + 255) / 256 * 256;
}

hipError_t launch_attend_latent(const Attend& a, uint8_t* ws, hipStream_t stream) {
    if (a.batch.n_seqs == 0 || a.batch.n_tokens == 0) return hipSuccess;
    const AttendPlan p =
        plan_latent(a.q.heads, a.batch.n_seqs, a.batch.n_tokens, (uint64_t)a.max_len);
    const float by = a.scale * kLog2e;
    if (a.value_dim <= 256 && a.cache.head_dim <= 320) go<256, 320>(a, p, by, ws, stream);
    else go<512, 576>(a, p, by, ws, stream);
    if (hipError_t e = hipGetLastError()) return e;
    if (p.shares == 0) return hipSuccess;
    const dim3 grid(p.tiles * ((1u << p.tile_log2) / kWaves));
    k_latent_join<<<grid, dim3(kThreads), 0, stream>>>(a, p, ws);
    return hipGetLastError();
}

}  // namespace sz
