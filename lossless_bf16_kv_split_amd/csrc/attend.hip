// attend.hip -- attention of new tokens over a paged BF16 KV cache.
//
// For a query row q at position c and the keys j visible to it (j < len,
// causal j <= c, window j > c - W):
//   s_j = scale * q.k_j, or softcap * tanh(scale * q.k_j / softcap)
//   m = max s_j, l = sum exp(s_j - m), o = sum exp(s_j - m) v_j / l
// in one pass over the keys with a running m and l, in powers of two:
// t = s log2(e), weights 2^(t - m).
//
// The query heads of one KV head read the same keys, so a sequence's rows
// for a KV head are (token, head of the group) pairs, row r = token * G + g,
// cut into tiles.  Both products run on the matrix cores in the form
//   S^T = K Q^T,  O^T = V^T P^T
// whose results hold one query per lane: the softmax's statistics are
// lane-local but for one exchange, and since the order of a contraction's
// terms is free, the weights go from the first product's result registers
// into the second's operand without any exchange at all.
#include "attend_parts.h"

namespace sz {
namespace {

constexpr uint64_t kCus = 256;
// The work is shared out among as many workgroups as the chip holds at once:
// two a CU, one with 256-element heads.  Whole tiles where there are enough
// of them to even out (kManyFew, kManyTiles), or where a tile has so few keys
// that one workgroup is done with them in the time that the second launch
// would take.  Few rows: by the bytes, which one CU gets at about 50 GB/s (one
// token of 32 / 8 heads of 128, whole and shared out: 512 keys, 256 KB, 11.9 and
// 12.7 us; 640, 12.4 and 13.1; 704, 13.6 and 13.4; 896, 14.8 and 13.0; of 64
// elements: 1152 keys, 288 KB, 11.8 and 12.7; 1280, 13.5 and 12.3.  More
// sequences stay better whole for longer: 32 of 768 keys 21 and 29; 9 of 5
// tokens, 64 elements, 1536 keys 14.7 and 16.7).
// Where they are many: 256 sequences of 1024 keys, 8 KV heads: 199 us whole,
// 237 shared out; 128 of 2048: 210 and 198.
// Tiles of 128 rows: 128 elements, 896 keys: 23.7 us whole, 30.1 shared out;
// 1500: 35.5 and 22.5; 256 elements, 319 keys: 22.7 and 30.4; 565: 32.1 and
// 29.5; 64 elements (whose steps cost nearly what 128 do), 1100: 20.9, 19.4.
// Long chunks, four tiles a sequence and more, fill the CUs evenly with whole
// tiles from one a CU on, and every cut of theirs costs 128 KB of sums written
// and read: 32 / 8 heads of 128, 256 tiles, 1024 keys 27 us whole, 42 shared
// out; 4096: 84 and 92; 16384: 323 and 298; 128 tiles, 1024 keys: 26 and 34;
// 2048: 45 and 43.
constexpr uint64_t kManyFew = 2048, kManyTiles = 512;
constexpr uint64_t kWholeFew = 288 * 1024, kWholeTiles = 480 * 1024;
constexpr uint64_t kWholeHalf = 700 * 1024, kWholeOneEach = 4096 * 1024;
// Sharing out looks at every sequence in every workgroup, 64 at a time.
constexpr uint64_t kShareSeqs = 1024;
// and counts steps in 32 bits.
constexpr uint64_t kMostSteps = uint64_t{1} << 30;
// Shares of one step only where all of them find a CU for themselves, of a
// 128-row tile never: twice the parts to join and to write cost more (32 / 8
// heads of 128 elements, one token: 4096 keys 13.6 us in shares of one step,
// 14.4 of two; 8192 keys 18.1 and 15.8; 64 tokens on 4096: 32.0 and 26.3).

AttendPlan plan_attend(uint32_t q_heads, const Cache& c, uint64_t n_seqs, uint64_t n_tokens,
                       uint64_t max_len, uint64_t window) {
    AttendPlan p;
    p.group = q_heads / c.kv_heads;
    const uint64_t rows = n_tokens * p.group;
    p.tile_log2 = rows <= 16 * n_seqs ? 4 : 7;
    // 256 rows where even they are many and sequences fill 16 of them on average
    // (8 with 64 elements): half the reads of LDS and L2 for the same products,
    // but one workgroup a CU, not two, and more rows that a sequence's last tile
    // lacks (32 / 8 heads of 128, tiles of 128 and of 256 rows: 2 chunks of 2048
    // tokens 198 us and 192, 4 of 1000 206 and 205, 8 of 512 116 and 130, 32 of
    // 128 120 and 149; 4096 tokens beside 200 single ones 484 and 700; of 64: 8
    // of 512 81 and 73, 16 of 256 79 and 78, 32 of 128 73 and 82, but 8 of 1024
    // beside 8 single ones 199 and 249)
    if (p.tile_log2 == 7 && c.head_dim <= 128 &&
        rows >> (c.head_dim <= 64 ? 11 : 12) >= n_seqs && (rows >> 8) * c.kv_heads >= kManyTiles)
        p.tile_log2 = 8;
    p.tiles = (uint32_t)((rows >> p.tile_log2) + n_seqs);
    // keys of a tile: a window shows its rows' tokens' own keys and those of
    // a window before
    uint64_t keys = max_len;
    const uint64_t tokens = ((1u << p.tile_log2) - 1) / p.group + 2;
    if (window < keys && window != 0 && window + tokens < keys) keys = window + tokens;
    // workgroups with whole tiles, as far as can be told here: numbers of
    // tiles are mostly free where sequences have few rows each
    const uint64_t full = rows >> p.tile_log2;
    const uint64_t groups = (full > n_seqs ? full : n_seqs) * c.kv_heads;
    const uint64_t resident = c.head_dim > 128 ? kCus : 2 * kCus;
    const uint64_t width = p.few() || c.head_dim > 128 ? c.head_dim : 128;
    uint64_t most_bytes = p.few() ? kWholeFew : kWholeTiles;
    if (!p.few() && full >= 4 * n_seqs && groups >= kCus / 2)
        most_bytes = groups >= kCus ? kWholeOneEach : kWholeHalf;
    const bool whole = n_seqs > kShareSeqs || c.kv_heads > resident ||
                       groups >= (p.few() ? kManyFew : kManyTiles) || p.tile_log2 == 8 ||
                       p.tiles * (max_len / kStep + 2) >= kMostSteps ||
                       keys * width * 4 <= most_bytes;
    p.shares = whole ? 0 : (uint32_t)(resident / c.kv_heads);
    p.alone = p.few() ? (uint32_t)(kCus / c.kv_heads) : 0;
    p.wide = p.few() && whole && groups <= kCus && c.head_dim <= 128;
    return p;
}

// ---- few rows: a decode step, drafted tokens ------------------------------
//
// One workgroup takes a tile of 16 rows and a part of its keys; each wave
// streams every fourth (or eighth) block of 32 keys straight from the pages
// into registers, with the next block's loads in flight, and the waves'
// results are joined in LDS at the end.  Bound by the bytes of the cache: 48
// sequences of 130 to 8192 keys, 908 MB, take 168 us (5.4 TB/s; a large copy
// moves 4.8), two of 32768, 264 MB, 55 us with the join.  A short cache is
// bound by the chain of loads (lengths, page addresses, keys): about 7 us,
// and 3 for the join.
//
// Matrix operands of 16x16x32: lane (n = lane % 16, h = lane / 16) holds
// eight of 32 contraction terms of row n.
//  - K: row n of a block of 16 keys, elements 32 s + 8 h .. + 7: one 16-byte
//    load a slice, a key's four lanes together 64 contiguous bytes.
//  - S^T's result: lane (query n, h) has the scores of keys 4 h + i of each
//    block.  These eight are what the lane feeds the second product as its
//    contraction terms,
//  - so V's operand needs, in lane (n, h), eight keys 4 h + i of both blocks
//    for one element.  A lane loads those eight keys' rows at elements
//    8 n .. 8 n + 7 (16 lanes read a whole contiguous row) and transposes
//    8 x 8 words in registers (32 byte permutes); product i takes the
//    elements 8 n + i as its rows.
//  - O^T's result: lane (query n, h) then has, for r < 4, elements
//    32 h + 8 r + i: 32 consecutive ones.
template <int DP, int WAVES>
struct FewLds {
    float o[WAVES][16][DP + 4];
    float m[WAVES][16], l[WAVES][16];
};

template <int DP, int WAVES, bool SHARED>
__device__ __forceinline__ void few_part(const Attend& a, const AttendPlan& p, const Score& score,
                                         uint8_t* ws, const Part& part, uint32_t kv,
                                         FewLds<DP, WAVES>& join) {
    constexpr int kStride = 32 * WAVES;    // keys that the workgroup takes at a time
    // the loads' nt bit: shared out work is more than the caches hold (2 x
    // 32768 keys: 58 us without; but 12.1 us with, 10.6 without, for tiles of
    // 1024 keys that stay in them)
    constexpr int kAux = SHARED ? 2 : 0;
    constexpr int kSlices = DP / 32;       // of K, 32 elements each
    constexpr int kVec = DP < 128 ? 4 : 8; // elements of a V row per load
    constexpr int kVLoads = DP / (16 * kVec);
    constexpr int kProducts = DP / 16;     // of 16 elements of the output
    const uint32_t lane = threadIdx.x % kWave, n = lane % 16, h = lane / 16;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const Tile& t = part.t;
    const int32_t first = part.first, last = part.last;

    // the rows, their queries (slices of 32 elements, zeros past head_dim)
    const uint32_t dim = a.cache.head_dim;
    bf16x8 q[kSlices];
    const Row mine = find_row(a, p, t, (int32_t)n);
    const int32_t low = mine.low, high = mine.high;
    {
        const uint16_t* row = static_cast<const uint16_t*>(a.q.data) +
                              (uint64_t)mine.token * a.q.token_stride +
                              (uint64_t)(kv * p.group + mine.head) * a.q.head_stride;
#pragma unroll
        for (int s = 0; s < kSlices; s++) {
            u32x4 v = {0, 0, 0, 0};
            if (mine.on && 32 * s + 8 * h < dim)
                v = *(const SZ_GLOBAL u32x4*)(row + 32 * s + 8 * h);
            q[s] = __builtin_bit_cast(bf16x8, v);
        }
    }

    // byte offsets of the lane's loads within a block of 16 keys
    constexpr uint32_t kPast = 0x80000000u;
    const uint32_t step = 2 * (uint32_t)a.cache.token_stride;
    uint32_t k_off[kSlices], v_off[4][kVLoads];
#pragma unroll
    for (int s = 0; s < kSlices; s++)
        k_off[s] = 32 * s + 8 * h < dim ? n * step + 64 * s + 16 * h : kPast;
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int u = 0; u < kVLoads; u++)
            v_off[i][u] = kVec * n + 128 * u < dim ? (4 * h + i) * step + 2 * (kVec * n + 128 * u)
                                                   : kPast;

    struct Block {
        u32x4 k[2][kSlices];
        u32x4 v[8][kVLoads];
    };
    const uint64_t table_row = (uint64_t)t.seq * a.cache.table_pitch;
    const auto load = [&](Block& x, int32_t j) {
#pragma unroll
        for (int b = 0; b < 2; b++) {
            const int32_t jb = j + 16 * b;
            uint64_t k_page = 0, v_page = 0;
            if (jb < last && jb + 16 > t.lo) {
                const uint64_t entry = table_row + ((uint32_t)jb >> a.cache.page_log2);
                k_page = page_address(a.cache.k_pages, entry);
                v_page = page_address(a.cache.v_pages, entry);
            }
            const uint32_t slot = (uint32_t)jb & ((1u << a.cache.page_log2) - 1);
            const auto kr = block_rows(a.cache, k_page, slot, kv, last - jb);
            const auto vr = block_rows(a.cache, v_page, slot, kv, last - jb);
#pragma unroll
            for (int s = 0; s < kSlices; s++)
                x.k[b][s] = __builtin_amdgcn_raw_buffer_load_b128(kr, k_off[s], 0, kAux);
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int u = 0; u < kVLoads; u++) {
                    if constexpr (kVec == 8) {
                        x.v[4 * b + i][u] =
                            __builtin_amdgcn_raw_buffer_load_b128(vr, v_off[i][u], 0, kAux);
                    } else {
                        const u32x2 w = __builtin_amdgcn_raw_buffer_load_b64(vr, v_off[i][u], 0, kAux);
                        x.v[4 * b + i][u] = u32x4{w.x, w.y, 0, 0};
                    }
                }
        }
    };

    float m = kNoKey, l = 0;
    f32x4 o[kProducts];
#pragma unroll
    for (int d = 0; d < kProducts; d++) o[d] = f32x4{0, 0, 0, 0};

    // operand i of the transposed values
    const auto values = [&](const Block& x, int d) {
        const int u = d / kVec, i = d % kVec;
        const uint32_t pick = i & 1 ? 0x07060302u : 0x05040100u;
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; k++)
            w[k] = __builtin_amdgcn_perm(x.v[2 * k + 1][u][i / 2], x.v[2 * k][u][i / 2], pick);
        return words8(w[0], w[1], w[2], w[3]);
    };

    const auto compute = [&](Block& x, int32_t j) {
        // keys that some row does not see
        const bool edge = j < t.all_lo || j + 32 > t.all_hi;
        bool odd = false;
        if (edge) {
#pragma unroll
            for (int k = 0; k < 8; k++) {
                const int32_t key = j + 16 * (k / 4) + 4 * (int32_t)h + k % 4;
#pragma unroll
                for (int u = 0; u < kVLoads; u++)
#pragma unroll
                    for (int i = 0; i < kVec / 2; i++) {
                        if (key < t.lo) x.v[k][u][i] = 0;
                        odd = odd || any_odd(odd_halves(x.v[k][u][i]));
                    }
            }
            odd = __ballot(odd) != 0;
        }
        uint32_t weights[4], seen[4];
        {
            float s[8];
#pragma unroll
            for (int k = 0; k < 2; k++) {
                f32x4 z = {0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < kSlices; c++)
                    z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8, x.k[k][c]), q[c], z, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; i++) s[4 * k + i] = z[i];
            }
            if (score.cap > 0) {
#pragma unroll
                for (int i = 0; i < 8; i++) s[i] = capped(score, s[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++) s[i] *= score.by;
            }
            if (edge) {
                const Sees sees(low, high, j + 4 * (int32_t)h);
#pragma unroll
                for (int i = 0; i < 8; i++)
                    if (!sees(16 * (i / 4) + i % 4)) s[i] = -INFINITY;
            }
            float top = s[0];
#pragma unroll
            for (int i = 1; i < 8; i++) top = fmaxf(top, s[i]);
            if (__ballot(top > m + kLag) != 0) {
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                top = fmaxf(top, m);
                const float keep = __builtin_amdgcn_exp2f(m - top);
                m = top;
                l *= keep;
#pragma unroll
                for (int d = 0; d < kProducts; d++) o[d] *= keep;
            }
#pragma unroll
            for (int i = 0; i < 8; i++) {
                s[i] = __builtin_amdgcn_exp2f(s[i] - m);
                l += s[i];
            }
#pragma unroll
            for (int i = 0; i < 4; i++) weights[i] = pack_bf16(s[2 * i], s[2 * i + 1]);
            if (odd) {
                const Sees sees(low, high, j + 4 * (int32_t)h);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const uint32_t key = 16 * (i / 2) + 2 * (i % 2);
                    seen[i] = (sees(key) ? 0x3F80u : 0u) | (sees(key + 1) ? 0x3F800000u : 0u);
                }
            }
        }
        if (odd) {
            // an infinity or a NaN must reach the rows that see it and no
            // other: 0 times it would be NaN.  The values go in without it,
            // and a product of marks with what each row sees brings it in.
            Block y;
#pragma unroll
            for (int k = 0; k < 8; k++)
#pragma unroll
                for (int u = 0; u < kVLoads; u++)
#pragma unroll
                    for (int i = 0; i < kVec / 2; i++) {
                        y.v[k][u][i] = mark_pair(x.v[k][u][i]);
                        x.v[k][u][i] = plain_pair(x.v[k][u][i]);
                    }
#pragma unroll
            for (int d = 0; d < kProducts; d++) {
                f32x4 z = {0, 0, 0, 0};
                z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    values(y, d), words8(seen[0], seen[1], seen[2], seen[3]), z, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; i++) o[d][i] += unmark(z[i]);
            }
        }
#pragma unroll
        for (int d = 0; d < kProducts; d++) {
            o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                values(x, d), words8(weights[0], weights[1], weights[2], weights[3]), o[d], 0, 0, 0);
        }
    };

    int32_t j = first + 32 * (int32_t)wave;
    Block even, odd;
    load(even, j);
    for (; j < last; j += 2 * kStride) {
        load(odd, j + kStride);
        compute(even, j);
        load(even, j + 2 * kStride);
        if (j + kStride < last) compute(odd, j + kStride);
    }

    // join the waves: row by row in LDS
    if (SHARED) __syncthreads();  // (the part before has been read)
    constexpr int kRun = 4 * kVec;  // consecutive elements of a lane's result, per 16 kVec
    {
        float sum = l;
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (h == 0) {
            join.m[wave][n] = m;
            join.l[wave][n] = sum;
        }
#pragma unroll
        for (int u = 0; u < kVLoads; u++)
#pragma unroll
            for (int r = 0; r < 4; r++)
#pragma unroll
                for (int i = 0; i < kVec; i++)
                    join.o[wave][n][16 * kVec * u + kRun * h + kVec * r + i] =
                        o[kVec * u + i][r];
        __syncthreads();
        constexpr int kPer = DP / 16;  // elements of a thread, of the first 256
        const uint32_t r = threadIdx.x / 16 % 16, e = threadIdx.x % 16 * kPer;
        const Row w = find_row(a, p, t, (int32_t)r);
        if (w.on && threadIdx.x < kThreads) {
            float top = join.m[0][r];
#pragma unroll
            for (int i = 1; i < WAVES; i++) top = fmaxf(top, join.m[i][r]);
            float total = 0, x[kPer] = {};
#pragma unroll
            for (int i = 0; i < WAVES; i++) {
                const float keep = __builtin_amdgcn_exp2f(join.m[i][r] - top);
                total += join.l[i][r] * keep;
#pragma unroll
                for (int k = 0; k < kPer; k++) x[k] = fmaf(join.o[i][r][e + k], keep, x[k]);
            }
            const uint32_t head = kv * p.group + w.head;
            if (!SHARED || part.alone) {
                const float inv = inverse(total);
#pragma unroll
                for (int k = 0; k < kPer; k++) x[k] *= inv;
                const uint64_t at = (uint64_t)w.token * a.out.token_stride +
                                    (uint64_t)head * a.out.head_stride + e;
                constexpr int kPiece = kPer < 8 ? kPer : 8;
#pragma unroll
                for (int k = 0; k < kPer; k += kPiece) {
                    float y[kPiece];
#pragma unroll
                    for (int i = 0; i < kPiece; i++) y[i] = x[k + i];
                    if (e + k < dim) store_out<kPiece>(a.out, at + k, y);
                }
                if (e == 0 && a.lse != nullptr)
                    a.lse[(uint64_t)w.token * a.q.heads + head] = log_sum(top, total);
            } else {
                const Partial u = partial_of(ws, a, p, kv, part.slot, a.cache.head_dim);
#pragma unroll
                for (int k = 0; k < kPer; k += 4)
                    if (e + k < dim)
                        store_global(reinterpret_cast<uint4*>(
                                         u.o + (uint64_t)r * dim + e + k),
                                     make_uint4(__float_as_uint(x[k]), __float_as_uint(x[k + 1]),
                                                __float_as_uint(x[k + 2]),
                                                __float_as_uint(x[k + 3])));
                if (e == 0) {
                    u.ml[2 * r] = top;
                    u.ml[2 * r + 1] = total;
                }
            }
        }
    }
}

template <int DP, int WAVES, bool SHARED>
__global__ __launch_bounds__(WAVES * kWave, DP > 128 || WAVES > 4 ? 1 : 2) void k_attend_few(
    Attend a, AttendPlan p, Score score, uint8_t* ws) {
    const uint32_t kv = blockIdx.x % a.cache.kv_heads, index = blockIdx.x / a.cache.kv_heads;
    __shared__ FewLds<DP, WAVES> join;
    Walk<SHARED> walk(a, p);
    Part part;
    if (!walk.first(a, p, index, part)) return;
    do {
        few_part<DP, WAVES, SHARED>(a, p, score, ws, part, kv, join);
    } while (walk.next(a, p, index, part));
}

// ---- chunks: a part of a prompt, or all of it -----------------------------
//
// One workgroup of four waves takes a tile of 128 (or 256) rows, each wave 32
// (or 64) of them, and walks the tile's keys 64 at a time.  The keys and values
// of a step go from the pages straight to LDS (each wave fetches a block of
// 16 keys) while the step before is worked on, with one barrier a step.
//
// Bound by power: at 1.0 PFLOP/s under the counters the matrix cores are busy
// 50% of the cycles, the vector units 42%, and the clock falls from 2.4 to
// 2.0 GHz (1.73 with a kernel that kept the former busy 55%), so what counts
// is fewer instructions and fewer reads for the same products.  Measured:
// 2048 tokens of 64 heads on 32768 keys 1.89 to 1.93 ms (1.11 to 1.13 PFLOP/s),
// a prompt of 8192 tokens of 32 heads 0.53 ms (1.04); a library product of
// 8192^3: 1.40.  With a cap on the scores, two more transcendental instructions
// each, 15 to 30% slower.  The tile of 128 rows leaves room for two
// workgroups a CU (which take all of its 160 KB of LDS, with 128 elements, and
// up to 256 registers a lane each), which hide each other's barriers and
// latencies; the one of 256 reads LDS and L2 half as often for the same products
// and is 3% faster where sequences fill many of them.  Heads of 256 elements have one workgroup of 128 rows a CU: 0.89
// PFLOP/s on 2048 tokens of 16 heads over 8192 keys.
//
// Matrix operands of 32x32x16: lane (n = lane % 32, h = lane / 32) holds eight
// of 16 contraction terms of row n.
//  - K: key n of 32, elements 16 s + 8 h .. + 7: 16 bytes of LDS.
//  - S^T's result i: query n, key 8 (i / 4) + 4 h + i % 4 of the 32.
//  - V: keys 16 t + 4 h + .. and 16 t + 8 + 4 h + .. (four each) for element
//    32 d + n: LDS reads that transpose four rows of 16 words.
//  - O^T's result i: query n, element 32 d + 8 (i / 4) + 4 h + i % 4.
//
// LDS holds rows of DP words in 16-byte pieces, permuted so that both kinds
// of reads spread over the banks: piece c of key j lies at c ^ k_mix(j) (16
// keys' same piece: 16 places) and c ^ v_mix(j) (four keys' 64 consecutive
// bytes: four places).  No bank conflicts are counted.

template <int DP>
__device__ __forceinline__ constexpr uint32_t k_mix(uint32_t j) {
    return DP == 64 ? j >> 1 & 7 : j & 15;
}
template <int DP>
__device__ __forceinline__ constexpr uint32_t v_mix(uint32_t j) {
    return DP == 64 ? (j >> 1 & 1) << 2 : (j & 3) << 2;
}

// Where a step's keys and values come from.  Paged: from the cache's pages,
// looked up a step ahead.
struct Paged {
    static constexpr bool kRotary = false;
    const Attend& a;
    uint64_t table_row, k_page, v_page;
    uint32_t kv;
    int32_t last;

    __device__ __forceinline__ Paged(const Attend& attend, const Part& part, uint32_t head)
        : a(attend), table_row((uint64_t)part.t.seq * attend.cache.table_pitch), kv(head),
          last(part.last) {}
    __device__ __forceinline__ uint32_t k_step() const { return 2 * (uint32_t)a.cache.token_stride; }
    __device__ __forceinline__ uint32_t v_step() const { return 2 * (uint32_t)a.cache.token_stride; }
    __device__ __forceinline__ uint32_t k_dim() const { return a.cache.head_dim; }
    // the block of 16 keys at jb (a load that nothing waits for: the step's
    // own wait covers it)
    __device__ __forceinline__ void look_up(int32_t jb, int32_t lo) {
        const bool seen = jb < last && jb + 16 > lo;
        const uint64_t entry = table_row + ((uint32_t)jb >> a.cache.page_log2);
        k_page = seen ? a.cache.k_pages[entry] : 0;
        v_page = seen ? a.cache.v_pages[entry] : 0;
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows(uint64_t page, int32_t jb) const {
        const uint32_t slot = (uint32_t)jb & ((1u << a.cache.page_log2) - 1);
        const uint64_t at = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(page >> 32))
                                << 32 | (uint32_t)__builtin_amdgcn_readfirstlane((int)page);
        return block_rows(a.cache, at, slot, kv, last - jb);
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t keys(int32_t jb) const {
        return rows(k_page, jb);
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t values(int32_t jb) const {
        return rows(v_page, jb);
    }
};

// Ragged: from tensors of rows, sequence after sequence, every head with keys
// and values of its own and a rotary part of the key beside them.
struct Ragged {
    static constexpr bool kRotary = true;
    const Expanded& e;
    int64_t start;
    uint32_t head;
    int32_t last;

    __device__ __forceinline__ Ragged(const Expanded& expanded, int64_t key_start, uint32_t h,
                                      int32_t past)
        : e(expanded), start(key_start), head(h), last(past) {}
    __device__ __forceinline__ uint32_t k_step() const { return 2 * (uint32_t)e.k.token_stride; }
    __device__ __forceinline__ uint32_t v_step() const { return 2 * (uint32_t)e.v.token_stride; }
    __device__ __forceinline__ uint32_t r_step() const { return 2 * (uint32_t)e.r.token_stride; }
    __device__ __forceinline__ uint32_t k_dim() const { return e.key_dim; }
    __device__ __forceinline__ void look_up(int32_t, int32_t) {}
    // (row numbers come from the device: uniform, but not to the compiler)
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows(const Rows& r, uint32_t h, uint32_t dim,
                                                           int32_t jb) const {
        const bool some = jb < last;
        const uint64_t at = reinterpret_cast<uint64_t>(r.data) +
                            2 * ((uint64_t)(start + jb) * r.token_stride + h * r.head_stride);
        const uint64_t to = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(at >> 32))
                                << 32 | (uint32_t)__builtin_amdgcn_readfirstlane((int)at);
        const uint32_t n = last - jb > 16 ? 15 : (uint32_t)(last - jb) - 1;
        const uint32_t bytes = __builtin_amdgcn_readfirstlane(
            some ? 2 * (n * (uint32_t)r.token_stride + dim) : 0);
        return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(bytes != 0 ? to : 0), 0,
                                                 bytes, kBufferFlags);
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t keys(int32_t jb) const {
        return rows(e.k, head, e.key_dim, jb);
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t values(int32_t jb) const {
        return rows(e.v, head, e.value_dim, jb);
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t rotary(int32_t jb) const {
        return rows(e.r, e.r.heads == 1 ? 0 : head, e.rotary_dim, jb);
    }
};

// Bytes of LDS: K of two steps of 64 keys, V of three (or two), and of two
// steps 64 elements of the keys' rotary part, in rows of their own.
template <int DP, bool ROTARY, int VS>
constexpr uint32_t kChunkLds = (2 + VS) * 64 * 2 * DP + (ROTARY ? 2 * 64 * 128 : 0);
static_assert(2 * kChunkLds<128, false, 3> <= 160 * 1024, "two workgroups a CU");
static_assert(kChunkLds<256, false, 3> <= 160 * 1024, "");
static_assert(2 * kChunkLds<128, true, 2> <= 160 * 1024, "two workgroups a CU");

template <int DP, int QB, int CAP, bool SHARED, class Source>
__device__ __forceinline__ void chunk_part(const Attend& a, const AttendPlan& p,
                                           const Score& score, uint8_t* ws, const Part& part,
                                           uint32_t kv, uint8_t* lds, Source source) {
    constexpr bool kRotary = Source::kRotary;
    // With the rotary part there is room for two workgroups only if V has two
    // buffers.  A step's values are then asked for when it begins, into those
    // of the step before the last, and waited for in its middle, a barrier more
    // (a prompt of 8192 tokens of 32 heads 618 us, 753 with three buffers and one
    // workgroup, 638 with 256 rows; shared out, 1024 tokens of 16 heads on 8192
    // keys 102, 123 with one workgroup).
    constexpr bool kLate = kRotary;
    constexpr uint32_t kVs = kLate ? 2 : 3;
    constexpr int kKeys = 64;
    constexpr uint32_t kRow = 2 * DP;             // bytes of a row in LDS
    constexpr uint32_t kBuffer = kKeys * kRow;    // K or V of a step
    constexpr int kLoads = DP / 32;               // per wave, of K or V
    constexpr int kMain = DP / 16, kParts = DP / 32;
    constexpr int kSlices = kMain + (kRotary ? 4 : 0);  // those of the rotary part last
    const uint32_t lane = threadIdx.x % kWave, n = lane % 32, h = lane / 32;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const Tile& t = part.t;
    const int32_t first = part.first, last = source.last;

    const uint32_t dim = source.k_dim(), v_dim = a.cache.head_dim;
    bf16x8 q[QB][kSlices];
    int32_t low[QB], high[QB];
#pragma unroll
    for (int b = 0; b < QB; b++) {
        const Row w = find_row(a, p, t, (int32_t)(32 * QB * wave + 32 * b + n));
        low[b] = w.low;
        high[b] = w.high;
        const uint16_t* row = static_cast<const uint16_t*>(a.q.data) +
                              (uint64_t)w.token * a.q.token_stride +
                              (uint64_t)(kv * p.group + w.head) * a.q.head_stride;
#pragma unroll
        for (int s = 0; s < kSlices; s++) {
            u32x4 v = {0, 0, 0, 0};
            uint32_t e = 16 * s + 8 * h, past = dim;
            if constexpr (kRotary) {
                if (s >= kMain) {
                    e = dim + 16 * (s - kMain) + 8 * h;
                    past = dim + source.e.rotary_dim;
                }
            }
            if (w.on && e < past) v = *(const SZ_GLOBAL u32x4*)(row + e);
            q[b][s] = __builtin_bit_cast(bf16x8, v);
        }
    }
    // keys visible to some row of this wave
    int32_t w_lo = t.lo, w_hi = t.hi;
    {
        const int32_t r0 = 32 * QB * (int32_t)wave;
        const Row x = find_row(a, p, t, r0), y = find_row(a, p, t, r0 + 32 * QB - 1);
        if (x.on) w_lo = x.low;
        else w_hi = w_lo;  // no rows: nothing to do
        if (y.on) w_hi = y.high;
    }

    // this wave's part of a step: 16 keys, kLoads KB of K and of V
    constexpr uint32_t kPast = 0x80000000u;
    uint32_t k_off[kLoads], v_off[kLoads], r_off[2];
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
        const uint32_t at = 1024 * i + 16 * lane, row = at / kRow, piece = at % kRow / 16;
        const uint32_t kp = piece ^ k_mix<DP>(row), vp = piece ^ v_mix<DP>(row);
        k_off[i] = 8 * kp < dim ? row * source.k_step() + 16 * kp : kPast;
        v_off[i] = 8 * vp < v_dim ? row * source.v_step() + 16 * vp : kPast;
    }
    if constexpr (kRotary) {
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const uint32_t at = 1024 * i + 16 * lane, row = at / 128;
            const uint32_t piece = at % 128 / 16 ^ k_mix<64>(row);
            r_off[i] = 8 * piece < source.e.rotary_dim ? row * source.r_step() + 16 * piece : kPast;
        }
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)(SZ_LDS uint8_t*)lds;
    constexpr uint32_t kRotaryAt = (2 + kVs) * kBuffer;  // of LDS
    source.look_up(first + 16 * (int32_t)wave, t.lo);
    // K and V of the step at j to their buffers
    const auto fetch_keys = [&](int32_t j, uint32_t buffer) {
        const int32_t jb = j + 16 * (int32_t)wave;
        load_to_lds<kLoads>(source.keys(jb), k_off, lds0 + buffer * kBuffer + wave * 16 * kRow);
        if constexpr (kRotary)
            load_to_lds<2>(source.rotary(jb), r_off,
                           lds0 + kRotaryAt + buffer * 8192 + wave * 2048);
    };
    const auto fetch_values = [&](int32_t j, uint32_t buffer) {
        load_to_lds<kLoads>(source.values(j + 16 * (int32_t)wave), v_off,
                            lds0 + (2 + buffer) * kBuffer + wave * 16 * kRow);
    };
    // both, and the next step's block looked up
    const auto fetch_step = [&](int32_t j, uint32_t k_buffer, uint32_t v_buffer) {
        fetch_keys(j, k_buffer);
        fetch_values(j, v_buffer);
        source.look_up(j + kKeys + 16 * (int32_t)wave, t.lo);
    };

    // LDS addresses of this lane's reads.  Slice s of K is at its first
    // slice's address with 32 s exclusive-or-ed in, part d of V at the first
    // part's with 64 d (the permutations only touch bits that a row's start
    // has as zeros).
    const uint32_t k_lane = lds0 + n * kRow + (h ^ k_mix<DP>(n)) * 16;
    const uint32_t v_key = lane % 16 / 4;
    const uint32_t v_lane = lds0 + 2 * kBuffer + (4 * h + v_key) * kRow +
                            ((2 * (lane / 16 % 2) + lane % 4 / 2) ^ v_mix<DP>(v_key)) * 16 +
                            lane % 2 * 8;
    // K of 32 keys (block of a buffer) at `at`, V of 16 keys
    const uint32_t r_lane = lds0 + kRotaryAt + n * 128 + (h ^ k_mix<64>(n)) * 16;
    const auto keys_at = [&](uint32_t at, int s) {
        if constexpr (kRotary) {  // (rows of 128 bytes, half of those of 128 elements)
            static_assert(!kRotary || kRow == 256, "");
            if (s >= kMain)
                return *(const SZ_LDS bf16x8*)(uintptr_t)((r_lane + (at - k_lane) / 2) ^
                                                          32 * (s - kMain));
        }
        return *(const SZ_LDS bf16x8*)(uintptr_t)(at ^ 32 * s);
    };
    const auto value_words = [&](uint32_t at, int t16, int d) {
        const uint32_t from = (at ^ 64 * d) + 16 * t16 * kRow;
        const u32x2 x = __builtin_bit_cast(
            u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((SZ_LDS s16x4*)(uintptr_t)from));
        const u32x2 y = __builtin_bit_cast(
            u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                       (SZ_LDS s16x4*)(uintptr_t)(from + 8 * kRow)));
        return u32x4{x.x, x.y, y.x, y.y};
    };

    float m[QB], l[QB];
    f32x16 o[QB][kParts];
#pragma unroll
    for (int b = 0; b < QB; b++) {
        m[b] = kNoKey;
        l[b] = 0;
#pragma unroll
        for (int d = 0; d < kParts; d++)
#pragma unroll
            for (int i = 0; i < 16; i++) o[b][d][i] = 0;
    }

    const float by = CAP != kUncapped ? 1.0f : score.by;
    const auto scored = [&](float x) {
        return CAP == kQuick ? capped_quickly(score, x) : CAP == kExact ? capped(score, x) : x;
    };
    // The running maximum of block b of 32 rows, and what hangs on it, where
    // a score of it (its largest in this lane: top, in powers of two) is too
    // far above it
    const auto follow = [&](int b, float top) {
        if (__ballot(top > m[b] + kLag) == 0) return;
        top = fmaxf(top, __shfl_xor(top, 32));
        top = fmaxf(top, m[b]);
        const float keep = __builtin_amdgcn_exp2f(m[b] - top);
        m[b] = top;
        l[b] *= keep;
#pragma unroll
        for (int d = 0; d < kParts; d++)
#pragma unroll
            for (int i = 0; i < 16; i++) o[b][d][i] *= keep;
    };

    // A step at the rim of what the wave's rows see, one block of 32 rows
    // at a time.  An infinity or a NaN among its values must reach the rows
    // that see it and no other, and 0 times it would be NaN: the product then
    // reads a copy of the values without them (in the buffer that no step is
    // using; every wave makes all of it, so none waits for another), and they
    // are added afterwards, key by key.
    const auto rim = [&](int32_t j, uint32_t k_buffer, uint32_t v_buffer, uint32_t spare) {
        const uint32_t ka = k_lane + k_buffer * kBuffer;
        const uint32_t values = lds0 + (2 + v_buffer) * kBuffer;
        uint32_t halves = 0;
#pragma unroll 8
        for (int i = 0; i < (int)(kBuffer / 1024); i++) {
            const u32x4 x = *(const SZ_LDS u32x4*)(uintptr_t)(values + 1024 * i + 16 * lane);
            halves |= odd_halves(x.x) | odd_halves(x.y) | odd_halves(x.z) | odd_halves(x.w);
        }
        const bool odd = __ballot(any_odd(halves)) != 0;
        if (odd) {
#pragma unroll 1
            for (int i = 0; i < (int)(kBuffer / 1024); i++) {
                const uint32_t at = 1024 * i + 16 * lane;
                const u32x4 x = *(const SZ_LDS u32x4*)(uintptr_t)(values + at);
                *(SZ_LDS u32x4*)(uintptr_t)(lds0 + (2 + spare) * kBuffer + at) =
                    u32x4{plain_pair(x.x), plain_pair(x.y), plain_pair(x.z), plain_pair(x.w)};
            }
        }
        const uint32_t va = v_lane + (odd ? spare : v_buffer) * kBuffer;
#pragma unroll
        for (int b = 0; b < QB; b++) {
            f32x16 s[2];
#pragma unroll
            for (int k = 0; k < 2; k++) {
#pragma unroll
                for (int i = 0; i < 16; i++) s[k][i] = 0;
#pragma unroll
                for (int c = 0; c < kSlices; c++) {
                    s[k] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        keys_at(ka + 32 * k * kRow, c), q[b][c], s[k], 0, 0, 0);
                    // (or all the operands are read at once, into registers
                    // that the other loop misses)
                    if (c % 8 == 7) __builtin_amdgcn_sched_barrier(0);
                }
            }
            const Sees sees(low[b], high[b], j + 4 * (int32_t)h);
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < 2; k++)
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    s[k][i] = sees(32 * k + 8 * (i / 4) + i % 4)
                                  ? (CAP != kUncapped ? capped(score, s[k][i]) : s[k][i])
                                  : -INFINITY;
                    top = fmaxf(top, s[k][i]);
                }
            follow(b, top * by);
            uint32_t weights[16];
#pragma unroll
            for (int k = 0; k < 2; k++)
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float x = __builtin_amdgcn_exp2f(fmaf(s[k][i], by, -m[b]));
                    const float y = __builtin_amdgcn_exp2f(fmaf(s[k][i + 1], by, -m[b]));
                    l[b] += x + y;
                    weights[8 * k + i / 2] = pack_bf16(x, y);
                }
#pragma unroll
            for (int t16 = 0; t16 < 4; t16++) {
#pragma unroll
                for (int d = 0; d < kParts; d++)
                    o[b][d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        __builtin_bit_cast(bf16x8, value_words(va, t16, d)),
                        words8(weights[4 * t16], weights[4 * t16 + 1], weights[4 * t16 + 2],
                               weights[4 * t16 + 3]),
                        o[b][d], 0, 0, 0);
                if (t16 % 2 == 1) __builtin_amdgcn_sched_barrier(0);
            }
            if (odd) {
#pragma unroll 1
                for (int k = 0; k < kKeys; k++) {
                    const bool seen = j + k >= low[b] && j + k < high[b];
#pragma unroll
                    for (int d = 0; d < kParts; d++)
#pragma unroll
                        for (int g = 0; g < 4; g++) {
                            const u32x2 w = *(const SZ_LDS u32x2*)(uintptr_t)(
                                values + k * kRow + ((4 * d + g) ^ v_mix<DP>(k)) * 16 + 8 * h);
                            if (__ballot(seen && any_odd(odd_halves(w.x) | odd_halves(w.y))) == 0)
                                continue;
#pragma unroll
                            for (int e = 0; e < 4; e++) {
                                const float x = __uint_as_float(
                                    e % 2 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
                                if (seen && !(fabsf(x) <= FLT_MAX)) o[b][d][4 * g + e] += x;
                            }
                        }
                }
            }
        }
    };

    // Steps that every row sees all of, in a pipeline of halves (32 keys):
    // while the softmax of one half's scores (now) runs on the vector units,
    // the matrix cores form the next half's (next); then they add the one
    // half's values.  The order is laid down instruction group by instruction
    // group, so that each product has its share of the softmax beside it and
    // its operand read some groups ahead.
    struct Half {
        f32x16 s[QB];
        float top[QB];
    };
    // groups: a slice of the first product, a part of 16 keys of the second
    constexpr int kGroups = kSlices, kGroups2 = 2 * kParts;
    constexpr int kUnits = 8 * QB;       // pairs of weights in a lane
    constexpr int kAhead = 3;            // groups that operands are read ahead
    const auto zero = [&](Half& x) {
#pragma unroll
        for (int b = 0; b < QB; b++)
#pragma unroll
            for (int i = 0; i < 16; i++) x.s[b][i] = 0;
    };
    // ka: the next half's keys; va: this half's values.  PRODUCT: there is a
    // next half.
    const auto inner = [&](Half& now, Half& next, uint32_t ka, uint32_t va, auto product) {
        constexpr bool kProduct = decltype(product)::value;
#pragma unroll
        for (int b = 0; b < QB; b++) follow(b, scored(now.top[b]) * by);
        uint32_t weights[QB][8];
        // two weights: of 16 keys u / (4 QB), rows' block u / 4 % QB
        const auto unit = [&](int u) {
            const int t16 = u / (4 * QB), b = u / 4 % QB, i = 8 * t16 + 2 * (u % 4);
            const float x = __builtin_amdgcn_exp2f(fmaf(scored(now.s[b][i]), by, -m[b]));
            const float y = __builtin_amdgcn_exp2f(fmaf(scored(now.s[b][i + 1]), by, -m[b]));
            l[b] += x + y;
            // (kept here: left to itself the compiler puts the additions off
            // and holds every weight in a register until then)
            asm volatile("" : "+v"(l[b]));
            weights[b][4 * t16 + u % 4] = pack_bf16(x, y);
        };
        constexpr int kFirst = kUnits * 3 / 4;  // units beside the first product
        bf16x8 kf[kAhead + 1];
        u32x4 vf[kAhead + 1];
        const auto read = [&](int g) {  // group g's operand
            if (g < kGroups) {
                if constexpr (kProduct) kf[g % (kAhead + 1)] = keys_at(ka, g);
            } else if (g < kGroups + kGroups2) {
                vf[g % (kAhead + 1)] =
                    value_words(va, (g - kGroups) / kParts, (g - kGroups) % kParts);
            }
        };
#pragma unroll
        for (int g = 0; g < kAhead; g++) read(g);
        if constexpr (kProduct) zero(next);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int g = 0; g < kGroups; g++) {
            read(g + kAhead);
            if constexpr (kProduct) {
#pragma unroll
                for (int b = 0; b < QB; b++)
                    next.s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        kf[g % (kAhead + 1)], q[b][g], next.s[b], 0, 0, 0);
            }
#pragma unroll
            for (int u = g * kFirst / kGroups; u < (g + 1) * kFirst / kGroups; u++) unit(u);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (kProduct) {
#pragma unroll
            for (int b = 0; b < QB; b++) next.top[b] = -INFINITY;
        }
#pragma unroll
        for (int g = 0; g < kGroups2; g++) {
            read(kGroups + g + kAhead);
            const int t16 = g / kParts, d = g % kParts;
#pragma unroll
            for (int b = 0; b < QB; b++)
                o[b][d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                    __builtin_bit_cast(bf16x8, vf[(kGroups + g) % (kAhead + 1)]),
                    words8(weights[b][4 * t16], weights[b][4 * t16 + 1], weights[b][4 * t16 + 2],
                           weights[b][4 * t16 + 3]),
                    o[b][d], 0, 0, 0);
            if (g < kParts) {
#pragma unroll
                for (int u = kFirst + g * (kUnits - kFirst) / kParts;
                     u < kFirst + (g + 1) * (kUnits - kFirst) / kParts; u++)
                    unit(u);
            } else if constexpr (kProduct) {
#pragma unroll
                for (int i = (g - kParts) * 16 / kParts; i < (g - kParts + 1) * 16 / kParts; i++)
#pragma unroll
                    for (int b = 0; b < QB; b++)
                        next.top[b] = fmaxf(next.top[b], next.s[b][i]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // The scores of the first half
    const auto ahead = [&](Half& x, uint32_t ka) {
        zero(x);
#pragma unroll
        for (int c = 0; c < kSlices; c++) {
            const bf16x8 f = keys_at(ka, c);
#pragma unroll
            for (int b = 0; b < QB; b++)
                x.s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, q[b][c], x.s[b], 0, 0, 0);
        }
#pragma unroll
        for (int b = 0; b < QB; b++) {
            x.top[b] = x.s[b][0];
#pragma unroll
            for (int i = 1; i < 16; i++) x.top[b] = fmaxf(x.top[b], x.s[b][i]);
        }
    };

    // What was fetched for a step has arrived from every wave, and every
    // wave is done with the step before: with its keys, and with the values
    // of the one before that, which the next fetch replaces.
    const auto arrived = [&] {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    };
    // Steps of 64 keys; step x has K's buffer x % 2 and V's x % 3.
    // [in0, in1): steps all of which every row sees.
    const int32_t steps = first < last ? (last - first + kKeys - 1) / kKeys : 0;
    int32_t in0 = t.all_lo > first ? (t.all_lo - first + kKeys - 1) / kKeys : 0;
    int32_t in1 = (t.all_hi < last ? t.all_hi : last) - first;
    in1 = in1 > 0 ? in1 / kKeys : 0;
    if (in1 > steps) in1 = steps;
    if (in0 >= in1) in0 = in1 = steps;
    if (SHARED) arrived();  // (every wave is done with the part before)
    if (kLate) fetch_keys(first, 0);
    else if (steps > 0) fetch_step(first, 0, 0);
    // (waves without rows, of a token among chunks, leave LDS to the others:
    // 24 tokens and two chunks of 833, 256 elements, capped, 137 -> 132 us;
    // whole tiles run 2% slower with the test)
    const bool works = !SHARED || 32 * QB * (int32_t)wave < t.rows;
    int32_t x = 0;
    uint32_t vb = 0;  // x % kVs
    const auto begin_step = [&] {
        arrived();
        if constexpr (kLate) {
            fetch_values(first + x * kKeys, vb);
            fetch_keys(first + (x + 1) * kKeys, (x + 1) & 1);
        } else {
            fetch_step(first + (x + 1) * kKeys, (x + 1) & 1, vb == kVs - 1 ? 0 : vb + 1);
        }
    };
    // the step's values have arrived from every wave (the next keys, whose
    // loads came last, may still be under way)
    const auto values_here = [&] {
        if constexpr (kLate) {
            static_assert(!kLate || kLoads + 2 == 6, "");
            asm volatile("s_waitcnt vmcnt(6) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
    };
    const auto end_step = [&] {
        x++;
        vb = vb == kVs - 1 ? 0 : vb + 1;
    };
    for (int pass = 0; pass < 2; pass++) {
        const int32_t stop = pass == 0 ? in0 : steps;
        while (x < stop) {
            const int32_t j = first + x * kKeys;
            begin_step();
            values_here();
            if (j < w_hi && j + kKeys > w_lo) rim(j, x & 1, vb, vb == 0 ? kVs - 1 : vb - 1);
            end_step();
        }
        if (pass == 1 || in0 == in1) continue;
        Half even, uneven;
        uint32_t va = v_lane + vb * kBuffer;
        begin_step();
        if (works) {
            ahead(even, k_lane + (x & 1) * kBuffer);
            values_here();
            inner(even, uneven, k_lane + (x & 1) * kBuffer + 32 * kRow, va, std::true_type{});
        } else {
            values_here();
        }
        end_step();
        while (x < in1) {
            const uint32_t ka = k_lane + (x & 1) * kBuffer;
            begin_step();
            if (works) {
                inner(uneven, even, ka, va + 32 * kRow, std::true_type{});
                values_here();
                va = v_lane + vb * kBuffer;
                inner(even, uneven, ka + 32 * kRow, va, std::true_type{});
            } else {
                values_here();
            }
            end_step();
        }
        if (works) inner(uneven, even, 0, va + 32 * kRow, std::false_type{});
    }
    // nothing may still be on its way to this workgroup's LDS when it ends
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

#pragma unroll
    for (int b = 0; b < QB; b++) {
        const uint32_t r = 32 * QB * wave + 32 * b + n;
        const Row w = find_row(a, p, t, (int32_t)r);
        const float total = l[b] + __shfl_xor(l[b], 32);
        if (!w.on) continue;
        const uint32_t head = kv * p.group + w.head;
        if (!SHARED || part.alone) {
            const float inv = inverse(total);
            const uint64_t at = (uint64_t)w.token * a.out.token_stride +
                                (uint64_t)head * a.out.head_stride;
#pragma unroll
            for (int d = 0; d < kParts; d++)
#pragma unroll
                for (int g = 0; g < 4; g++) {
                    const uint32_t e = 32 * d + 8 * g + 4 * h;
                    const float x[4] = {o[b][d][4 * g] * inv, o[b][d][4 * g + 1] * inv,
                                        o[b][d][4 * g + 2] * inv, o[b][d][4 * g + 3] * inv};
                    if (e < v_dim) store_out<4>(a.out, at + e, x);
                }
            if (h == 0 && a.lse != nullptr)
                a.lse[(uint64_t)w.token * a.q.heads + head] = log_sum(m[b], total);
        } else {
            const Partial u = partial_of(ws, a, p, kv, part.slot, a.cache.head_dim);
#pragma unroll
            for (int d = 0; d < kParts; d++)
#pragma unroll
                for (int g = 0; g < 4; g++) {
                    const uint32_t e = 32 * d + 8 * g + 4 * h;
                    if (e < v_dim)
                        store_global(reinterpret_cast<uint4*>(u.o + (uint64_t)r * v_dim + e),
                                     make_uint4(__float_as_uint(o[b][d][4 * g]),
                                                __float_as_uint(o[b][d][4 * g + 1]),
                                                __float_as_uint(o[b][d][4 * g + 2]),
                                                __float_as_uint(o[b][d][4 * g + 3])));
                }
            if (h == 0) {
                u.ml[2 * r] = m[b];
                u.ml[2 * r + 1] = total;
            }
        }
    }
}

template <int DP, int QB, int CAP, bool SHARED>
__global__ __launch_bounds__(kThreads, QB == 1 && DP <= 128 ? 2 : 1) void k_attend_chunk(
    Attend a, AttendPlan p, Score score, uint8_t* ws) {
    const uint32_t kv = blockIdx.x % a.cache.kv_heads, index = blockIdx.x / a.cache.kv_heads;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kChunkLds<DP, false, 3>];
    Walk<SHARED> walk(a, p);
    Part part;
    // whole tiles: the last ones of a prompt see the most keys and go first
    if (!walk.first(a, p, SHARED ? index : p.tiles - 1 - index, part)) return;
    do {
        chunk_part<DP, QB, CAP, SHARED>(a, p, score, ws, part, kv, lds, Paged(a, part, kv));
    } while (walk.next(a, p, index, part));
}

// The same over keys and values expanded from latents: 192 elements of keys,
// 128 of values.
template <bool SHARED>
__global__ __launch_bounds__(kThreads, 2) void k_attend_expanded(
    Attend a, Expanded e, AttendPlan p, Score score, uint8_t* ws) {
    const uint32_t head = blockIdx.x % a.cache.kv_heads, index = blockIdx.x / a.cache.kv_heads;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kChunkLds<128, true, 2>];
    Walk<SHARED> walk(a, p);
    Part part;
    if (!walk.first(a, p, SHARED ? index : p.tiles - 1 - index, part)) return;
    do {
        // (a sequence whose keys lie outside the tensors: none are read)
        const int64_t start = __builtin_amdgcn_readfirstlane(e.key_starts[part.t.seq]);
        const int32_t len = __builtin_amdgcn_readfirstlane(a.batch.lens[part.t.seq]);
        const bool good = start >= 0 && start + len <= e.n_keys;
        chunk_part<128, 1, kUncapped, SHARED>(a, p, score, ws, part, head, lds,
                                              Ragged(e, start, head, good ? part.last : part.first));
    } while (walk.next(a, p, index, part));
}

__host__ __device__ inline uint32_t join_pieces(const AttendPlan& p) {
    return (1u << p.tile_log2) / (p.few() ? kWaves : 4 * kWaves);
}

// Joins the parts of the tiles that were cut, a row to a wave at a time (of a
// 128-row tile four, one after the other: a workgroup's way to its tile takes
// longer than a row).  64 parts at a time, a lane holds one's maximum and sum;
// LANES lanes take four elements each of one's sums, so that a wave reads
// 64 / LANES of them at a time, and four times as many with nothing to wait
// for between them (16 times: no faster with 64 parts, 1 us slower with
// few).  Latency bound: 3 us of a short call, 6 where 48 sequences' tiles
// were cut.
template <int LANES>
__global__ __launch_bounds__(kThreads) void k_attend_join(Attend a, AttendPlan p, uint8_t* ws) {
    constexpr uint32_t kAtOnce = kWave / LANES, kBatch = 4;
    const uint32_t lane = threadIdx.x % kWave;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t pieces = join_pieces(p);
    const uint32_t kv = blockIdx.x % a.cache.kv_heads;
    const uint32_t rest = blockIdx.x / a.cache.kv_heads;
    const uint32_t number = rest / pieces;
    const Shares shares(a, p);
    if (number >= Shares::from_lane(shares.tiles1, kWave - 1)) return;
    const Shares::Found f = shares.find(a, p, true, number);
    const uint32_t at = number - f.tiles0;
    const uint32_t step = f.steps0 + at * f.x.steps;
    const uint32_t from = step / shares.quota, upto = (step + f.x.steps - 1) / shares.quota;
    const Tile t = make_tile(a, p, f.seq, number, f.x.q, (int64_t)at << p.tile_log2);
    if (from == upto) return;
    const uint32_t dim = a.cache.head_dim;
    const uint32_t e = 4 * (lane % LANES);
    const uint64_t stride = (uint64_t)dim << p.tile_log2;
    const int32_t rows = 1 << p.tile_log2;
    for (int32_t r = (int32_t)(rest % pieces * kWaves + wave); r < t.rows && r < rows;
         r += (int32_t)(pieces * kWaves)) {
        const Row w = find_row(a, p, t, r);
        float top = kNoKey, total = 0;
        f32x4 x = {0, 0, 0, 0};
        for (uint32_t i0 = from; i0 <= upto; i0 += kWave) {
            const uint32_t parts = upto - i0 + 1 < kWave ? upto - i0 + 1 : kWave;
            const Partial u = partial_of(ws, a, p, kv, i0 + number, a.cache.head_dim);
            float m = kNoKey, l = 0;
            if (lane < parts) {
                m = u.ml[2 * (((uint64_t)lane << p.tile_log2) + r)];
                l = u.ml[2 * (((uint64_t)lane << p.tile_log2) + r) + 1];
            }
            const float* o = u.o + (uint64_t)r * dim + e;
            f32x4 v[kBatch];
            const auto read = [&](uint32_t s0) {
#pragma unroll
                for (uint32_t k = 0; k < kBatch; k++) {
                    const uint32_t s = s0 + k * kAtOnce + lane / LANES;
                    v[k] = f32x4{0, 0, 0, 0};
                    if (s < parts && e < dim) v[k] = *(const SZ_GLOBAL f32x4*)(o + s * stride);
                }
            };
            read(0);  // (under way while the weights are made)
            const float most = wave_max(fmaxf(m, top));
            const float weight = __builtin_amdgcn_exp2f(m - most);
            const float keep = __builtin_amdgcn_exp2f(top - most);
            top = most;
            total = total * keep + wave_sum(l * weight);
            x *= keep;
            for (uint32_t s0 = 0; s0 < parts; s0 += kBatch * kAtOnce) {
                if (s0 > 0) read(s0);
#pragma unroll
                for (uint32_t k = 0; k < kBatch; k++)
                    x += v[k] * __shfl(weight, (s0 + k * kAtOnce + lane / LANES) % kWave);
            }
        }
#pragma unroll
        for (int d = LANES; d < (int)kWave; d *= 2)
#pragma unroll
            for (int i = 0; i < 4; i++) x[i] += __shfl_xor(x[i], d);
        const float inv = inverse(total);
        const float y[4] = {x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv};
        const uint32_t head = kv * p.group + w.head;
        if (lane < LANES && e < dim)
            store_out<4>(a.out, (uint64_t)w.token * a.out.token_stride +
                                    (uint64_t)head * a.out.head_stride + e, y);
        if (lane == 0 && a.lse != nullptr)
            a.lse[(uint64_t)w.token * a.q.heads + head] = log_sum(top, total);
    }
}

template <int DP, int CAP>
hipError_t go(const Attend& a, const AttendPlan& p, uint8_t* ws, hipStream_t stream) {
    const dim3 grid((p.shares != 0 ? p.shares : p.tiles) * a.cache.kv_heads);
    constexpr uint32_t block = kThreads;
    const Score score = score_of(a);
    if (p.few()) {
        if (p.shares != 0)
            k_attend_few<DP, 4, true><<<grid, block, 0, stream>>>(a, p, score, ws);
        else if (DP <= 128 && p.wide)
            k_attend_few<DP <= 128 ? DP : 128, 8, false>
                <<<grid, 2 * block, 0, stream>>>(a, p, score, ws);
        else
            k_attend_few<DP, 4, false><<<grid, block, 0, stream>>>(a, p, score, ws);
        return hipGetLastError();
    }
    if constexpr (DP <= 128) {
        if (p.tile_log2 == 8) {
            k_attend_chunk<DP, 2, CAP, false><<<grid, block, 0, stream>>>(a, p, score, ws);
            return hipGetLastError();
        }
    }
    if (p.shares != 0)
        k_attend_chunk<DP, 1, CAP, true><<<grid, block, 0, stream>>>(a, p, score, ws);
    else
        k_attend_chunk<DP, 1, CAP, false><<<grid, block, 0, stream>>>(a, p, score, ws);
    return hipGetLastError();
}

template <int CAP>
hipError_t go(const Attend& a, const AttendPlan& p, uint8_t* ws, hipStream_t stream) {
    const uint32_t dim = a.cache.head_dim;
    return dim <= 64    ? go<64, CAP>(a, p, ws, stream)
           : dim <= 128 ? go<128, CAP>(a, p, ws, stream)
                        : go<256, CAP>(a, p, ws, stream);
}

}  // namespace

uint64_t attend_workspace(uint32_t q_heads, const Cache& c, uint64_t n_seqs, uint64_t n_tokens,
                          uint64_t max_len) {
    // without a window: with one the work may stay in whole tiles, and is
    // shared out the same otherwise
    const AttendPlan p = plan_attend(q_heads, c, n_seqs, n_tokens, max_len, 0);
    if (p.shares == 0) return 0;
    const uint64_t rows = c.kv_heads * partial_slots(p) << p.tile_log2;
    return (rows * (c.head_dim + 2) * 4 + 255) / 256 * 256;
}

// Keys and values expanded from latents: a head is a KV head of its own.
// Tiles of 128 rows, whole where there is one for each CU (four chunks of 20
// heads, 340 tiles: 112 us whole, 129 shared out), or where the CUs without one
// would take too few keys off the others to pay for the join.  Whole and shared
// out, us: 1024 tokens of 16 heads (128 tiles) on 1024 keys 29 and 35, on 2048
// 50 and 42, on 8192 159 and 102; 1500 of 16 as a prompt (176) 40 and 47; on
// 1024 keys 512 of 5 (20) 27.3 and 24.7, 128 of 16 (16) 27.5 and 22.5.
AttendPlan plan_expanded(uint32_t heads, uint64_t n_seqs, uint64_t n_tokens, uint64_t max_len) {
    AttendPlan p{};
    p.group = 1;
    p.tile_log2 = 7;
    p.tiles = (uint32_t)((n_tokens >> p.tile_log2) + n_seqs);
    const uint64_t full = n_tokens >> p.tile_log2;
    const uint64_t groups = (full > n_seqs ? full : n_seqs) * heads;
    const bool whole = n_seqs > kShareSeqs || heads > kCus || groups >= kCus ||
                       p.tiles * (max_len / kStep + 2) >= kMostSteps ||
                       max_len * (kCus - groups) <= 768 * kCus;
    p.shares = whole ? 0 : (uint32_t)(2 * kCus / heads);
    return p;
}

uint64_t attend_expanded_workspace(uint32_t heads, uint32_t value_dim, uint64_t n_seqs,
                                   uint64_t n_tokens, uint64_t max_len) {
    // (0, of any length: one that is shared out if any is)
    const AttendPlan p =
        plan_expanded(heads, n_seqs, n_tokens, max_len == 0 ? uint64_t{1} << 18 : max_len);
    if (p.shares == 0) return 0;
    const uint64_t rows = heads * partial_slots(p) << p.tile_log2;
    return (rows * (value_dim + 2) * 4 + 255) / 256 * 256;
}

hipError_t launch_attend_expanded(const Attend& a, const Expanded& e, uint8_t* ws,
                                  hipStream_t stream) {
    if (a.batch.n_seqs == 0 || a.batch.n_tokens == 0) return hipSuccess;
    const AttendPlan p =
        plan_expanded(a.q.heads, a.batch.n_seqs, a.batch.n_tokens, (uint64_t)a.max_len);
    const Score score = score_of(a);
    const dim3 grid((p.shares != 0 ? p.shares : p.tiles) * a.cache.kv_heads), block(kThreads);
    if (p.shares != 0) k_attend_expanded<true><<<grid, block, 0, stream>>>(a, e, p, score, ws);
    else k_attend_expanded<false><<<grid, block, 0, stream>>>(a, e, p, score, ws);
    const hipError_t st = hipGetLastError();
    if (st != hipSuccess || p.shares == 0) return st;
    const dim3 join(p.tiles * a.cache.kv_heads * join_pieces(p));
    if (a.value_dim <= 64) k_attend_join<16><<<join, block, 0, stream>>>(a, p, ws);
    else k_attend_join<32><<<join, block, 0, stream>>>(a, p, ws);
    return hipGetLastError();
}

hipError_t launch_attend(const Attend& a, uint8_t* ws, hipStream_t stream) {
    if (a.batch.n_seqs == 0 || a.batch.n_tokens == 0) return hipSuccess;
    const AttendPlan p =
        plan_attend(a.q.heads, a.cache, a.batch.n_seqs, a.batch.n_tokens, (uint64_t)a.max_len,
                    a.window);
    const hipError_t e = !(a.softcap > 0)         ? go<kUncapped>(a, p, ws, stream)
                         : a.softcap <= kQuickCap ? go<kQuick>(a, p, ws, stream)
                                                  : go<kExact>(a, p, ws, stream);
    if (e != hipSuccess || p.shares == 0) return e;
    const dim3 grid(p.tiles * a.cache.kv_heads * join_pieces(p)), block(kThreads);
    if (a.cache.head_dim <= 64) k_attend_join<16><<<grid, block, 0, stream>>>(a, p, ws);
    else if (a.cache.head_dim <= 128) k_attend_join<32><<<grid, block, 0, stream>>>(a, p, ws);
    else k_attend_join<64><<<grid, block, 0, stream>>>(a, p, ws);
    return hipGetLastError();
}

}  // namespace sz
