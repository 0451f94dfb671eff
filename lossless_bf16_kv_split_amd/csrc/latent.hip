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
//
// 48 tokens of 128 heads on 100 to 8192 keys (196 MB of rows): 86 to 103 us
// by card, of which the join 10 to 12.  A step of 64 keys takes about 4800
// cycles: 1900 for the scores, bound by LDS (their reads 1152, the next step's
// rows arriving 576), 1060 for the output, 1200 for the softmax and its barrier,
// 600 waiting for the rows.  LDS holds two steps' keys and one workgroup a CU, so nothing runs
// beside a wave's wait.
//
// What beginning a tile costs, in steps, so that it is shared out with them
// (48 tokens of 128 heads: 104 us with 0, 96 with 2, 94 with 3; drafts of 3 tokens
// 37, 31, 31; 32 tokens of one sequence on 8192 keys 89, 101, 94)
#define SZ_TILE_EXTRA 3
#include "attend_parts.h"

namespace sz {
namespace {

constexpr int kKeys = 64;  // of a step
constexpr uint64_t kCus = 256;
constexpr int kAhead = 6;  // products that operands are read from LDS ahead of

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
    static constexpr uint32_t kWeights = 2 * kBuffer;     // LDS: weights [RW][2][2][64 lanes][16 B]
    static constexpr uint32_t kTops = kWeights + RW * 4096;  // [RW][2][32] floats
    static constexpr uint32_t kFlags = kTops + RW * 256;     // of each wave
    static constexpr uint32_t kLds = kFlags + 16;
    static_assert(RW <= 2 && kRow % 256 == 128, "rows start at alternating halves of the banks");
    static_assert(2 * kLoads <= kSlices, "a load for every other product");
    static_assert(kLds <= 160 * 1024, "");
};

// 16-byte piece c of a step's key j lies at c ^ mix(j).  Rows being an odd
// multiple of 128 bytes, 16 keys' same piece then fall on 16 different places of
// the 256 bytes that LDS serves at once, and 64 consecutive bytes of four keys
// on four different quarters.
__device__ __forceinline__ constexpr uint32_t mix(uint32_t j) {
    return (j >> 1 & 1) << 2 | (j >> 2 & 1) << 1 | (j >> 3 & 1);
}

// 64 lanes' 16 bytes each from offsets of a buffer to consecutive bytes of LDS
// (load_to_lds, one load, to stand between products: issuing one takes as long
// as half a product).
__device__ __forceinline__ void load_piece(__amdgpu_buffer_rsrc_t from, uint32_t at, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %2, %1, 0 offen lds"
                 :
                 : "s"(lds), "s"(from), "v"(at)
                 : "memory");
}

template <int DL, int DT, int RW>
__device__ __forceinline__ void latent_part(const Attend& a, const AttendPlan& p, float by,
                                            uint8_t* ws, const Part& part, uint32_t half,
                                            uint8_t* lds) {
    using S = Shape<DL, DT, RW>;
    constexpr int kKw = S::kKw, kParts = S::kParts;
    constexpr uint32_t kRow = S::kRow;
    const uint32_t lane = threadIdx.x % kWave, n = lane % 32, h = lane / 32;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t rw = wave / kKw, kw = wave % kKw, block = kw % 2;
    const uint32_t r = 32 * (RW * half + rw) + n;  // the lane's row of the tile
    const Tile& t = part.t;
    const int32_t first = part.first, last = part.last;
    const uint32_t dim = a.cache.head_dim;

    const Row mine = find_row(a, p, t, (int32_t)r);
    const bool works = 32 * (int32_t)(RW * half + rw) < t.rows;

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

    // the row's query, asked for before anything is waited for
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

    // A step's fetch: the rows of this wave's block (none past the last step),
    // and their loads, one at a time
    struct Fetch {
        __amdgpu_buffer_rsrc_t rows;
        uint32_t to;
    };
    const auto begin_fetch = [&](int32_t j, uint32_t buffer) {
        const int32_t jb = j + 16 * (int32_t)wave;
        const uint32_t slot = (uint32_t)jb & ((1u << a.cache.page_log2) - 1);
        const uint64_t at =
            (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(next_page >> 32)) << 32 |
            (uint32_t)__builtin_amdgcn_readfirstlane((int)next_page);
        next_page = page_at(j + kKeys);
        return Fetch{block_rows(a.cache, at, slot, 0, last - jb),
                     lds0 + buffer * S::kBuffer + wave * 16 * kRow};
    };
    const auto fetch = [&](const Fetch& f, int i) { load_piece(f.rows, off[i], f.to + 1024 * i); };

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

    const uint32_t my_weights = lds0 + S::kWeights + rw * 4096 + 16 * lane;
    const uint32_t my_tops = lds0 + S::kTops + rw * 256 + 4 * n;
    const uint32_t flags = lds0 + S::kFlags;
    enum { kRise = 1, kOdd = 2 };

    // A step, with the next one's fetch.  EDGE: some row does not see some key.
    const auto compute = [&](int32_t j, uint32_t buffer, const Fetch& next, auto edge_step) {
        constexpr bool edge = decltype(edge_step)::value;
        const uint32_t ka = k_lane + buffer * S::kBuffer + block * 32 * kRow;
        const uint32_t va = v_lane + buffer * S::kBuffer + kw * kParts * 64;
        f32x16 s;
        float top = -INFINITY;
        bool odd = false;  // an infinity or a NaN among the keys: no score is a number
        if (works) {
            bf16x8 f[kAhead];
#pragma unroll
            for (int c = 0; c < kAhead; c++) f[c] = keys_at(ka, c);
#pragma unroll
            for (int i = 0; i < 16; i++) s[i] = 0;
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int c = 0; c < S::kSlices; c++) {
                s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[c % kAhead], q[c], s, 0, 0, 0);
                if (c + kAhead < S::kSlices) f[c % kAhead] = keys_at(ka, c + kAhead);
                if (c % 2 == 0 && c / 2 < S::kLoads) fetch(next, c / 2);
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
#pragma unroll
            for (int i = 0; i < S::kLoads; i++) fetch(next, i);
        }
        u32x4 f[kAhead];
        const auto words = [&](int g) { return value_words(va, g / kParts, g % kParts); };
        // weights of this wave's 32 keys, and their sum
        u32x4 w[4];
        float sum = 0;
        const auto weigh = [&] {
            uint32_t x[8];
            sum = 0;
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float u = __builtin_amdgcn_exp2f(fmaf(s[i], by, -m));
                const float v = __builtin_amdgcn_exp2f(fmaf(s[i + 1], by, -m));
                sum += u + v;
                x[i / 2] = pack_bf16(u, v);
            }
            if (kw < 2) {
                *(SZ_LDS u32x4*)(uintptr_t)(my_weights + 2048 * kw) = u32x4{x[0], x[1], x[2], x[3]};
                *(SZ_LDS u32x4*)(uintptr_t)(my_weights + 2048 * kw + 1024) =
                    u32x4{x[4], x[5], x[6], x[7]};
            }
        };
        if (works) {
            if constexpr (edge) {
                const Sees sees(0, mine.high, j + 32 * (int32_t)block + 4 * (int32_t)h);
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    odd = odd || !(fabsf(s[i]) <= FLT_MAX);
                    if (!sees(8 * (i / 4) + i % 4)) s[i] = -INFINITY;
                }
                odd = __ballot(odd) != 0;
            }
#pragma unroll
            for (int g = 0; g < kAhead; g++) f[g] = words(g);  // (under way meanwhile)
#pragma unroll
            for (int i = 0; i < 16; i++) top = fmaxf(top, s[i]);
            top *= by;
            weigh();
        }
        // The maximum belongs to all the waves of a row group: where a score
        // rises above it too far, all take part in moving it, and weigh again.
        const bool rise = __ballot(top > m + kLag) != 0;
        if (lane == 0)
            *(SZ_LDS uint32_t*)(uintptr_t)(flags + 4 * wave) = (rise ? kRise : 0) | (odd ? kOdd : 0);
        lds_barrier();
        const u32x4 any = *(const SZ_LDS u32x4*)(uintptr_t)flags;
        const uint32_t all = __builtin_amdgcn_readfirstlane((int)(any.x | any.y | any.z | any.w));
        if (all & kRise) {
            if (works) {
                top = fmaxf(top, __shfl_xor(top, 32));
                if (kw < 2 && h == 0) *(SZ_LDS float*)(uintptr_t)(my_tops + 128 * kw) = top;
            }
            lds_barrier();
            if (works) {
                top = fmaxf(top, *(const SZ_LDS float*)(uintptr_t)(my_tops + 128 * (1 - block)));
                // (each row by its own scores: none depends on another's)
                top = top > m + kLag ? top : m;
                const float keep = __builtin_amdgcn_exp2f(m - top);
                m = top;
                l *= keep;
#pragma unroll
                for (int d = 0; d < kParts; d++)
#pragma unroll
                    for (int i = 0; i < 16; i++) o[d][i] *= keep;
                weigh();
            }
            lds_barrier();
        }
        if (!works) return;
        odd = edge && (all & kOdd) != 0;
        l += sum;
#pragma unroll
        for (int i = 0; i < 4; i++) w[i] = *(const SZ_LDS u32x4*)(uintptr_t)(my_weights + 1024 * i);
        // At an edge an infinity or a NaN must not reach the rows that do not
        // see it, where 0 times it would be NaN.  The values go in without it;
        // rows that see it get NaN for it (their score with it is infinite or
        // NaN, and so is its weight times it), by a product of ones in its
        // place with what each row sees.
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int g = 0; g < 4 * kParts; g++) {
            u32x4 x = f[g % kAhead];
            if (edge && odd) {
#pragma unroll
                for (int i = 0; i < 4; i++) x[i] = plain_pair(x[i]);
            }
            o[g % kParts] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                __builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, w[g / kParts]),
                o[g % kParts], 0, 0, 0);
            if (g + kAhead < 4 * kParts) f[g % kAhead] = words(g + kAhead);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (!edge || !odd) return;
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
    lds_barrier();  // (every wave is done with the part before)
    if (steps > 0) {
        const Fetch f = begin_fetch(first, 0);
#pragma unroll
        for (int i = 0; i < S::kLoads; i++) fetch(f, i);
    }
    // (in accumulation registers, which the product reads as well: the output's
    // sums have the others, where they can be scaled)
#pragma unroll
    for (int s = 0; s < S::kSlices; s++) asm volatile("" : "+a"(q[s]));
    // (the steps that every row sees all of come first)
    int32_t inner = t.all_hi > first ? (t.all_hi - first) / kKeys : 0;
    inner = inner < steps ? inner : steps;
    const auto begin_step = [&](int32_t x) {
        arrived();
        return begin_fetch(first + (x + 1) * kKeys, (x + 1) & 1);
    };
    int32_t x = 0;
#pragma unroll 1
    for (; x < inner; x++) {
        const Fetch f = begin_step(x);
        compute(first + x * kKeys, x & 1, f, std::false_type{});
    }
#pragma unroll 1
    for (; x < steps; x++) {
        const Fetch f = begin_step(x);
        compute(first + x * kKeys, x & 1, f, std::true_type{});
    }
    // nothing may still be on its way to this workgroup's LDS when it ends
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

    float total = l + __shfl_xor(l, 32);
    // each of two waves has the sum over its block of every step's keys
    lds_barrier();
    if (kw < 2 && h == 0) *(SZ_LDS float*)(uintptr_t)(my_tops + 128 * kw) = total;
    lds_barrier();
    total += *(const SZ_LDS float*)(uintptr_t)(my_tops + 128 * (1 - block));
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
        const Partial u = partial_of(ws, a, p, 0, part.slot, a.value_dim);
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

// HALVES workgroups have a tile's rows between them and read the same keys at
// the same time: numbers that differ by eight, which share an L2, so that the
// keys come from memory once (246 MB for the 48 tokens above; tiles of 64 rows
// read 460).  Tiles of 64 rows, pairs of them: 48 tokens 99 and 97 us, drafts of
// 3 tokens of 64 heads 32.9 and 31.3, 32 tokens of one sequence 108 and 100, 128 of
// one 151 and 152.
template <int DL, int DT, int RW, int HALVES, bool SHARED>
__global__ __launch_bounds__(kThreads, 1) void k_attend_latent(Attend a, AttendPlan p, float by,
                                                               uint8_t* ws) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[Shape<DL, DT, RW>::kLds];
    const uint32_t index =
        HALVES == 1 ? blockIdx.x : blockIdx.x / (8 * HALVES) * 8 + blockIdx.x % 8;
    const uint32_t half = HALVES == 1 ? 0 : blockIdx.x / 8 % HALVES;
    if (!SHARED && index >= p.tiles) return;
    Walk<SHARED> walk(a, p);
    Part part;
    if (!walk.first(a, p, SHARED ? index : p.tiles - 1 - index, part)) return;
    do {
        if (32 * RW * (int32_t)half < part.t.rows)
            latent_part<DL, DT, RW>(a, p, by, ws, part, half, lds);
    } while (walk.next(a, p, index, part));
}

// Joins the parts of the tiles that were cut, eight elements a lane; the parts'
// maxima and sums 64 at a time, one a lane.  A row is one wave's, or (TOGETHER,
// where tiles have many parts) the four waves of a workgroup take a quarter
// of its parts each.  Latency bound: 4 us of a short call, 10 of the 48 tokens'.
template <bool TOGETHER>
__global__ __launch_bounds__(kThreads) void k_latent_join(Attend a, AttendPlan p, uint8_t* ws) {
    constexpr uint32_t kRows = TOGETHER ? 1 : kWaves;
    __shared__ float sums[TOGETHER ? kWaves : 1][8][kWave];
    __shared__ float ml[TOGETHER ? kWaves : 1][2];
    const uint32_t lane = threadIdx.x % kWave;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t pieces = (1u << p.tile_log2) / kRows;
    const uint32_t number = blockIdx.x / pieces;
    const Shares shares(a, p);
    if (number >= Shares::from_lane(shares.tiles1, kWave - 1)) return;
    const Shares::Found f = shares.find(a, p, true, number);
    const uint32_t at = number - f.tiles0;
    const uint32_t step = f.steps0 + at * f.x.steps;
    uint32_t from = (step + kExtra) / shares.quota, upto = (step + f.x.steps - 1) / shares.quota;
    if (from == upto) return;
    const Tile t = make_tile(a, p, f.seq, number, f.x.q, (int64_t)at << p.tile_log2);
    const int32_t r = (int32_t)(blockIdx.x % pieces * kRows + (TOGETHER ? 0 : wave));
    if (r >= t.rows) return;
    if (TOGETHER) {
        const uint32_t each = (upto - from + kWaves) / kWaves, past = upto + 1;
        from += wave * each;
        upto = from + each < past ? from + each : past;  // (from here: past the last)
    } else {
        upto++;
    }
    const Row w = find_row(a, p, t, r);
    const uint32_t e = 8 * lane;
    const bool on = e < a.value_dim;
    const uint64_t stride = (uint64_t)a.value_dim << p.tile_log2;
    float top = kNoKey, total = 0, x[8] = {};
    for (uint32_t i0 = from; i0 < upto; i0 += kWave) {
        const uint32_t parts = upto - i0 < kWave ? upto - i0 : kWave;
        const Partial u = partial_of(ws, a, p, 0, i0 + number, a.value_dim);
        const float* o = u.o + (uint64_t)r * a.value_dim + e;
        constexpr uint32_t kBatch = 8;
        f32x4 v[kBatch][2];
        const auto read = [&](uint32_t s0) {
#pragma unroll
            for (uint32_t k = 0; k < kBatch; k++)
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    v[k][i] = f32x4{0, 0, 0, 0};
                    if (on && s0 + k < parts)
                        v[k][i] = *(const SZ_GLOBAL f32x4*)(o + (s0 + k) * stride + 4 * i);
                }
        };
        float m = kNoKey, l = 0;
        if (lane < parts) {
            m = u.ml[2 * (((uint64_t)lane << p.tile_log2) + r)];
            l = u.ml[2 * (((uint64_t)lane << p.tile_log2) + r) + 1];
        }
        read(0);  // (under way while the weights are made)
        const float most = wave_max(fmaxf(m, top));
        const float weight = __builtin_amdgcn_exp2f(m - most);
        const float keep = __builtin_amdgcn_exp2f(top - most);
        top = most;
        total = total * keep + wave_sum(l * weight);
#pragma unroll
        for (int i = 0; i < 8; i++) x[i] *= keep;
        for (uint32_t s0 = 0; s0 < parts; s0 += kBatch) {
            if (s0 > 0) read(s0);
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
    if constexpr (TOGETHER) {
        ml[wave][0] = top;
        ml[wave][1] = total;
#pragma unroll
        for (int i = 0; i < 8; i++) sums[wave][i][lane] = x[i];
        __syncthreads();
        if (wave != 0) return;
        top = fmaxf(fmaxf(ml[0][0], ml[1][0]), fmaxf(ml[2][0], ml[3][0]));
        total = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) x[i] = 0;
#pragma unroll
        for (uint32_t k = 0; k < kWaves; k++) {
            const float weight = __builtin_amdgcn_exp2f(ml[k][0] - top);
            total = fmaf(ml[k][1], weight, total);
#pragma unroll
            for (int i = 0; i < 8; i++) x[i] = fmaf(sums[k][i][lane], weight, x[i]);
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

// Tiles of 32, 64 or 128 rows by what sequences have on average; whole, or shared
// out among one workgroup a CU (attend_parts.h).  Whole ones take as long as the
// longest sequence; of two workgroups for each CU, or of one with lengths that
// differ, about half would wait for it.  Sharing them out costs what 400 keys do
// and two for each workgroup (parts to store and to join).  Whole and shared
// out, us: one token of 16 heads on 256 keys 12.7 and 16.4, on 512 18.5 and 16.0;
// 8 on 700 23.6 and 16.0; 48 of 128 heads on 512 28 and 36, on 1024 42 and 45, on
// 2048 71 and 62, on 100 to 2048 69 and 47; 128 on 100 to 8192 493 and 242; 256
// of 32 heads on 100 to 2048 138 and 114; 300 of 16 on 100 to 1024 55 and 63, to
// 8192 372 and 297; 512 of 16 to 1024 93 and 182, to 8192 546 and 528; 1000 of 16
// to 1024 167 and 506; 256 tokens of one sequence, 128 heads, on 4096 271 and 283.
// Shares a tile from which on four waves join a row: one token of 16 heads on 32768
// keys, 256 shares, 26 us, by one wave 40; 32 tokens of 128 heads, four shares, 104
// and 98.
constexpr uint32_t kTogether = 8;
constexpr uint64_t kMostSteps = uint64_t{1} << 30;

uint32_t halves(const AttendPlan& p) { return p.tile_log2 == 7 ? 2 : 1; }

AttendPlan plan_latent(uint32_t heads, uint64_t n_seqs, uint64_t n_tokens, uint64_t max_len) {
    AttendPlan p{};
    p.group = heads;
    const uint64_t rows = n_tokens * heads;
    p.tile_log2 = rows <= 32 * n_seqs ? 5 : rows <= 64 * n_seqs ? 6 : 7;
    p.tiles = (uint32_t)((rows >> p.tile_log2) + n_seqs);
    const uint64_t full = rows >> p.tile_log2;
    const uint64_t units = (full > n_seqs ? full : n_seqs) * halves(p);
    const bool whole = units >= 2 * kCus ||
                       p.tiles * (max_len / kStep + 2 + kExtra) >= kMostSteps ||
                       max_len * (2 * kCus - units) <= 2 * kCus * (400 + 2 * units);
    p.shares = whole ? 0 : (uint32_t)(kCus / halves(p));
    p.alone = p.shares;
    return p;
}

template <int DL, int DT, int RW, int HALVES>
void go(const Attend& a, const AttendPlan& p, float by, uint8_t* ws, hipStream_t stream) {
    const dim3 block(kThreads);
    const uint32_t units = p.shares != 0 ? p.shares : p.tiles;
    const dim3 grid(HALVES == 1 ? units : (units + 7) / 8 * 8 * HALVES);
    if (p.shares != 0)
        k_attend_latent<DL, DT, RW, HALVES, true><<<grid, block, 0, stream>>>(a, p, by, ws);
    else
        k_attend_latent<DL, DT, RW, HALVES, false><<<grid, block, 0, stream>>>(a, p, by, ws);
}

template <int DL, int DT>
void go(const Attend& a, const AttendPlan& p, float by, uint8_t* ws, hipStream_t stream) {
    if (p.tile_log2 == 5) go<DL, DT, 1, 1>(a, p, by, ws, stream);
    else if (p.tile_log2 == 6) go<DL, DT, 2, 1>(a, p, by, ws, stream);
    else go<DL, DT, 2, 2>(a, p, by, ws, stream);
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
    const dim3 block(kThreads);
    if (p.shares >= kTogether * p.tiles)
        k_latent_join<true><<<dim3(p.tiles << p.tile_log2), block, 0, stream>>>(a, p, ws);
    else
        k_latent_join<false>
            <<<dim3((p.tiles << p.tile_log2) / kWaves), block, 0, stream>>>(a, p, ws);
    return hipGetLastError();
}

}  // namespace sz
