// attend_parts.h -- what the attention kernels over a cache share
// (attend.hip, latent.hip): how a call's rows and keys are cut up, scores,
// and the care for infinities and NaN in what a row does not see.
#pragma once

#include "kv_internal.h"

#include <cfloat>
#include <cstdint>

// What beginning a tile costs, in steps of keys (a file that includes this may
// say so first).
#ifndef SZ_TILE_EXTRA
#define SZ_TILE_EXTRA 0
#endif

namespace sz {
namespace {

constexpr uint32_t kExtra = SZ_TILE_EXTRA;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
#define SZ_LDS __attribute__((address_space(3)))
constexpr uint32_t kThreads = 256;
constexpr uint32_t kWaves = kThreads / kWave;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A row's running maximum before any key: below every finite score, and
// finite itself, so that differences with it are never infinity - infinity.
constexpr float kNoKey = -FLT_MAX;
// The maximum follows the scores only when one exceeds it by more than
// this (in powers of two): weights then stay below 2^8, which neither FP32
// sums nor BF16's relative rounding notice, and most tiles need no exchange
// between lanes and no rescaling.
constexpr float kLag = 8.0f;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

__device__ __forceinline__ bf16x8 words8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const u32x4 v = {a, b, c, d};
    return __builtin_bit_cast(bf16x8, v);
}

// The largest value of a wave's lanes, and their sum, in every lane: along
// rows of 16 lanes, then across them, without a pass through LDS.
template <int CTRL, int ROWS>
__device__ __forceinline__ float moved(float x, float other) {
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(other), __float_as_int(x),
                                                      CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ float last_lane(float x) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), kWave - 1));
}
__device__ __forceinline__ float wave_max(float x) {
    x = fmaxf(x, moved<0x111, 0xF>(x, x));  // row_shr:1
    x = fmaxf(x, moved<0x112, 0xF>(x, x));
    x = fmaxf(x, moved<0x114, 0xF>(x, x));
    x = fmaxf(x, moved<0x118, 0xF>(x, x));
    x = fmaxf(x, moved<0x142, 0xA>(x, x));  // row_bcast:15 into rows 1 and 3
    x = fmaxf(x, moved<0x143, 0xC>(x, x));  // row_bcast:31 into rows 2 and 3
    return last_lane(x);
}
__device__ __forceinline__ float wave_sum(float x) {
    x += moved<0x111, 0xF>(x, 0);
    x += moved<0x112, 0xF>(x, 0);
    x += moved<0x114, 0xF>(x, 0);
    x += moved<0x118, 0xF>(x, 0);
    x += moved<0x142, 0xA>(x, 0);
    x += moved<0x143, 0xC>(x, 0);
    return last_lane(x);
}

// How a call is cut up.  Tiles: the rows of a sequence for one KV head,
// tile_rows at a time.  Either each tile is one workgroup's, with all its
// keys; tile number floor(starts[s] * G / tile_rows) + s is then the first
// of sequence s, which leaves room for every tile whatever the lengths and
// needs no sum over the sequences.  Or (shares > 0) the work is shared out:
// all tiles' keys, in steps of kStep, laid end to end and cut into equal
// parts, one for each workgroup of a KV head, so that uneven lengths leave
// no workgroup behind; a tile cut by such a border is joined by a second
// launch.  Tiles are then numbered without gaps.
struct AttendPlan {
    uint32_t group;      // G
    uint32_t tile_log2;
    uint32_t tiles;      // a bound of the tiles' numbers
    uint32_t shares;     // workgroups that share it out for a KV head; 0: whole tiles
    uint32_t alone;      // up to so many steps in all, shares of one step
    bool wide;           // few rows, whole tiles, a CU each: eight waves
    __host__ __device__ bool few() const { return tile_log2 == 4; }
};

constexpr uint32_t kStep = 128;  // keys

// A tile, all uniform.
struct Tile {
    uint32_t seq;
    uint32_t number;
    int32_t begin;      // first token of the sequence
    int32_t row0, rows; // rows row0 .. row0 + rows - 1 of the sequence
    int32_t c0;         // position of the sequence's first new token
    int32_t lo, hi;     // keys visible to any row of the tile: lo .. hi - 1
    int32_t all_lo, all_hi;  // keys visible to every row
    int32_t from;       // lo rounded down to a multiple of 32
};

// The tile of row row0 on, of a sequence that holds it.
__device__ __forceinline__ Tile make_tile(const Attend& a, const AttendPlan& p, uint32_t seq,
                                          uint32_t number, const Seq& q, int64_t row0) {
    Tile t;
    t.seq = seq;
    t.number = number;
    t.begin = q.begin;
    t.c0 = q.len - (q.end - q.begin);
    // (row numbers fit 32 bits: the host keeps n_tokens * q heads below 2^31)
    t.row0 = (int32_t)row0;
    const int64_t left = (int64_t)(q.end - q.begin) * p.group - row0, most = 1ll << p.tile_log2;
    t.rows = (int32_t)(left < most ? left : most);
    t.lo = t.all_lo = 0;
    t.hi = t.all_hi = q.len;
    if (a.causal) {
        const int32_t first_c = t.c0 + t.row0 / (int32_t)p.group;
        const int32_t last_c = t.c0 + (t.row0 + t.rows - 1) / (int32_t)p.group;
        t.hi = last_c + 1 < 0 ? 0 : last_c + 1;
        t.all_hi = first_c + 1 < 0 ? 0 : first_c + 1;
        if (a.window != 0) {
            if ((int64_t)first_c + 1 > (int64_t)a.window) t.lo = first_c + 1 - (int32_t)a.window;
            if ((int64_t)last_c + 1 > (int64_t)a.window) t.all_lo = last_c + 1 - (int32_t)a.window;
        }
    }
    t.from = t.lo & ~31;
    return t;
}

// Whole tiles: the tile of a number, if there is one.
__device__ __forceinline__ bool find_tile(const Attend& a, const AttendPlan& p, uint32_t tile,
                                          Tile& t) {
    const auto first = [&](uint32_t s) {
        return (((int64_t)a.batch.starts[s] * p.group) >> p.tile_log2) + s;
    };
    const uint32_t s = find_seq(a.batch.n_seqs, tile, first);
    const Seq q = load_seq(a.batch, s, a.max_len);
    if (!q.good) return false;
    const int64_t at = (int64_t)tile - ((((int64_t)q.begin * p.group) >> p.tile_log2) + s);
    const int64_t row0 = at << p.tile_log2;
    if (at < 0 || row0 >= (int64_t)(q.end - q.begin) * p.group) return false;
    t = make_tile(a, p, s, tile, q, row0);
    return true;
}

// Work shared out: worker i takes steps i * quota .. (i + 1) * quota - 1 of
// all tiles' steps laid end to end.  Every wave adds up the sequences' steps
// for itself: lane i takes `each` consecutive sequences (one, up to 64 of
// them), a scan over the lanes gives where each lane's begin, and a second
// one, over the sequences of one lane, where each of those does.  (The host
// keeps the sum below kMostSteps.)
struct Shares {
    struct Load {
        Seq q;
        uint32_t tiles;   // of the sequence, 0 where it is faulty or has no rows
        uint32_t steps;   // of each of its tiles, at least 1, kExtra ones first
        int32_t from;     // the key of step 0
    };
    uint32_t each;
    uint32_t total;       // steps
    uint32_t quota;
    // this lane's sequences: steps and tiles before them, and with them
    uint32_t steps0, steps1, tiles0, tiles1;
    int32_t before;       // the largest start before them
    Load own;             // each == 1: the lane's sequence

    // (no sequence begins before an earlier one's start: those that remain
    // lie apart from each other, whatever the starts, so that their tiles and
    // steps stay within what the host counted on)
    static __device__ __forceinline__ int32_t start(const Attend& a, uint32_t s) {
        return s < a.batch.n_seqs ? a.batch.starts[s] : INT32_MIN;
    }
    static __device__ __forceinline__ Load load(const Attend& a, const AttendPlan& p, uint32_t s,
                                                int32_t begin, int32_t before) {
        Load x{};
        if (s >= a.batch.n_seqs) return x;
        x.q.begin = begin;
        x.q.end = a.batch.starts[s + 1];
        x.q.len = a.batch.lens[s];
        x.q.good = x.q.begin >= 0 && x.q.begin >= before && x.q.begin < x.q.end &&
                   x.q.end <= (int64_t)a.batch.n_tokens && x.q.len >= 0 && x.q.len <= a.max_len;
        if (!x.q.good) return x;
        const int64_t rows = (int64_t)(x.q.end - x.q.begin) * p.group;
        x.tiles = (uint32_t)((rows + (1 << p.tile_log2) - 1) >> p.tile_log2);
        const int32_t c0 = x.q.len - (x.q.end - x.q.begin);
        if (a.causal && a.window != 0 && (int64_t)c0 + 1 > (int64_t)a.window)
            x.from = (c0 + 1 - (int32_t)a.window) & ~31;
        x.steps = (uint32_t)(x.q.len - x.from + kStep - 1) / kStep;
        x.steps = (x.steps == 0 ? 1 : x.steps) + kExtra;
        return x;
    }

    // running sums over the lanes (rows of 16 lanes, then across the rows)
    template <int CTRL, int ROWS>
    static __device__ __forceinline__ uint32_t plus(uint32_t x) {
        return x + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, false);
    }
    static __device__ __forceinline__ uint32_t scan(uint32_t x) {
        x = plus<0x111, 0xF>(x);  // row_shr:1
        x = plus<0x112, 0xF>(x);
        x = plus<0x114, 0xF>(x);
        x = plus<0x118, 0xF>(x);
        x = plus<0x142, 0xA>(x);  // row_bcast:15 into rows 1 and 3
        x = plus<0x143, 0xC>(x);  // row_bcast:31 into rows 2 and 3
        return x;
    }

    // the largest value up to a lane
    template <int CTRL, int ROWS>
    static __device__ __forceinline__ int32_t most(int32_t x) {
        const int32_t y = __builtin_amdgcn_update_dpp(INT32_MIN, x, CTRL, ROWS, 0xF, false);
        return x > y ? x : y;
    }
    static __device__ __forceinline__ int32_t scan_most(int32_t x) {
        x = most<0x111, 0xF>(x);
        x = most<0x112, 0xF>(x);
        x = most<0x114, 0xF>(x);
        x = most<0x118, 0xF>(x);
        x = most<0x142, 0xA>(x);
        x = most<0x143, 0xC>(x);
        return x;
    }

    static __device__ __forceinline__ uint32_t from_lane(uint32_t x, uint32_t lane) {
        return (uint32_t)__builtin_amdgcn_readlane((int)x, lane);
    }

    __device__ __forceinline__ Shares(const Attend& a, const AttendPlan& p) {
        const uint32_t lane = threadIdx.x % kWave;
        each = (a.batch.n_seqs + kWave - 1) / kWave;
        uint32_t steps = 0, tiles = 0;
        before = INT32_MIN;
        if (each == 1) {
            const int32_t begin = start(a, lane);
            own = load(a, p, lane, begin, scan_most(begin));
            steps = own.tiles * own.steps;
            tiles = own.tiles;
        } else {
            int32_t top = INT32_MIN;
            for (uint32_t i = 0; i < each; i++) {
                const int32_t begin = start(a, lane * each + i);
                top = begin > top ? begin : top;
            }
            top = scan_most(top);
            before = __shfl_up(top, 1);
            if (lane == 0) before = INT32_MIN;
            top = before;
            for (uint32_t i = 0; i < each; i++) {
                const int32_t begin = start(a, lane * each + i);
                const Load x = load(a, p, lane * each + i, begin, top);
                top = begin > top ? begin : top;
                steps += x.tiles * x.steps;
                tiles += x.tiles;
            }
        }
        steps1 = scan(steps);
        tiles1 = scan(tiles);
        steps0 = steps1 - steps;
        tiles0 = tiles1 - tiles;
        total = from_lane(steps1, kWave - 1);
        quota = (total + p.shares - 1) / p.shares;
        if (quota == 1 && total > p.alone) quota = 2;
    }

    // A sequence: by one of its steps, or one of its tiles
    struct Found {
        uint32_t seq;
        Load x;
        uint32_t steps0, tiles0;  // steps and tiles before the sequence's
    };
    __device__ __forceinline__ Found find(const Attend& a, const AttendPlan& p, bool by_tile,
                                          uint32_t number) const {
        const auto first_past = [&](uint32_t steps, uint32_t tiles) {
            return (uint32_t)__builtin_ctzll(__ballot((by_tile ? tiles : steps) > number) |
                                             1ull << (kWave - 1));
        };
        uint32_t lane = first_past(steps1, tiles1);
        Found f;
        f.seq = lane;
        f.steps0 = from_lane(steps0, lane);
        f.tiles0 = from_lane(tiles0, lane);
        Load x = own;
        if (each > 1) {
            const uint32_t mine = threadIdx.x % kWave, first = lane * each;
            const uint32_t s = mine < each ? first + mine : a.batch.n_seqs;
            const int32_t begin = start(a, s), top = scan_most(begin);
            const int32_t base = (int32_t)from_lane((uint32_t)before, lane);
            x = load(a, p, s, begin, top > base ? top : base);
            const uint32_t steps = x.tiles * x.steps;
            const uint32_t s1 = scan(steps) + f.steps0, t1 = scan(x.tiles) + f.tiles0;
            lane = first_past(s1, t1);
            f.seq = first + lane;
            f.steps0 = from_lane(s1 - steps, lane);
            f.tiles0 = from_lane(t1 - x.tiles, lane);
        }
        f.x.q.begin = (int32_t)from_lane((uint32_t)x.q.begin, lane);
        f.x.q.end = (int32_t)from_lane((uint32_t)x.q.end, lane);
        f.x.q.len = (int32_t)from_lane((uint32_t)x.q.len, lane);
        f.x.q.good = true;
        f.x.tiles = from_lane(x.tiles, lane);
        f.x.steps = from_lane(x.steps, lane);
        f.x.from = (int32_t)from_lane((uint32_t)x.from, lane);
        return f;
    }
};

// What a workgroup works on at a time: a tile and a range of its keys, first
// .. last - 1 (first a multiple of 32, last - first one of kStep unless last
// is the tile's last key's; none where last <= first).
struct Part {
    Tile t;
    int32_t first, last;
    bool alone;      // the tile's only part
    uint32_t slot;   // of the results otherwise
};

// A workgroup's parts, one after the other.  Shared out, worker i's part of
// tile T has slot i + T: both only grow, so no two parts have the same one.
template <bool SHARED>
struct Walk;
template <>
struct Walk<false> {
    __device__ __forceinline__ Walk(const Attend&, const AttendPlan&) {}
    __device__ __forceinline__ bool first(const Attend& a, const AttendPlan& p, uint32_t index,
                                          Part& part) {
        if (!find_tile(a, p, index, part.t)) return false;
        part.first = part.t.from;
        part.last = part.t.hi;
        part.alone = true;
        part.slot = 0;
        return true;
    }
    __device__ __forceinline__ bool next(const Attend&, const AttendPlan&, uint32_t, Part&) {
        return false;
    }
};
// A tile begins with kExtra steps that have no keys, which stand for what it
// costs to begin one: a border among them counts as one before the tile.
template <>
struct Walk<true> {
    uint32_t step, end;
    __device__ __forceinline__ Walk(const Attend&, const AttendPlan&) {}
    __device__ __forceinline__ bool first(const Attend& a, const AttendPlan& p, uint32_t index,
                                          Part& part) {
        const Shares shares(a, p);
        step = index * shares.quota;
        end = step + shares.quota < shares.total ? step + shares.quota : shares.total;
        if (step >= end) return false;
        return take(shares, a, p, index, part);
    }
    // (the sums are made anew: they would hold registers through the part)
    __device__ __forceinline__ bool next(const Attend& a, const AttendPlan& p, uint32_t index,
                                         Part& part) {
        if (step >= end) return false;
        return take(Shares(a, p), a, p, index, part);
    }
    __device__ __forceinline__ bool take(const Shares& shares, const Attend& a,
                                         const AttendPlan& p, uint32_t index, Part& part) {
        const Shares::Found f = shares.find(a, p, false, step);
        const uint32_t at = (step - f.steps0) / f.x.steps;
        const uint32_t base = f.steps0 + at * f.x.steps, stop = base + f.x.steps;
        if constexpr (kExtra != 0)
            if (end < stop && end - base <= kExtra) return false;
        const uint32_t upto = stop < end ? stop : end;
        const uint32_t done = step - base <= kExtra ? 0 : step - base - kExtra;
        part.t = make_tile(a, p, f.seq, f.tiles0 + at, f.x.q, (int64_t)at << p.tile_log2);
        // (a part begins at one of the steps, even where a window shows the
        // tile's rows fewer keys than the sequence's first one: whole steps
        // up to the part's end, which masks nothing)
        const uint32_t skip = (uint32_t)(part.t.from - f.x.from) / kStep;
        part.first = f.x.from + (int32_t)((done > skip ? done : skip) * kStep);
        const int32_t last = f.x.from + (int32_t)((upto - base - kExtra) * kStep);
        part.last = last < part.t.hi ? last : part.t.hi;
        part.alone = done == 0 && upto == stop;
        part.slot = index + part.t.number;
        step = upto;
        return true;
    }
};

// Keys that a row sees: low .. high - 1.  Rows past the tile's end are given
// all of the tile's (nothing of them is stored).
struct Row {
    int32_t token, head;  // head within the group
    int32_t low, high;
    bool on;
};
__device__ __forceinline__ Row find_row(const Attend& a, const AttendPlan& p, const Tile& t,
                                        int32_t r) {
    Row w;
    w.on = r < t.rows;
    const int32_t row = t.row0 + (w.on ? r : 0);
    const int32_t i = row / (int32_t)p.group;
    w.token = t.begin + i;
    w.head = row - i * (int32_t)p.group;
    w.low = t.lo;
    w.high = t.hi;
    if (w.on && a.causal) {
        const int32_t c = t.c0 + i;
        w.high = c + 1;
        if (a.window != 0 && (int64_t)c + 1 > (int64_t)a.window)
            w.low = c + 1 - (int32_t)a.window;
    }
    return w;
}

// t of a raw score: score * (scale log2 e), or the capped form, whose tanh
// is 1 - 2 / (1 + e^2x), and for |x| < 1/2, where that difference leaves few
// bits, x (1 + c1 x^2 + c2 x^4 + c3 x^6 + c4 x^8), off by less than 3e-8 of it
// (least squares on Chebyshev nodes, reweighted until the error was even).
struct Score {
    float by;    // scale log2 e; capped: 2 scale log2 e / softcap
    float cap;   // softcap log2 e, 0 for none
    float odd[5];  // capped: the polynomial in the score times `by`
};
inline Score score_of(const Attend& a) {
    static const double kTanh[5] = {1.0, -0.33333143895419826, 0.1332587893917483,
                                    -0.05304549308250774, 0.01724148911923954};
    Score s{};
    s.cap = a.softcap * kLog2e;
    s.by = a.softcap > 0 ? 2 * kLog2e * (a.scale / a.softcap) : a.scale * kLog2e;
    const double half = 0.5 * 0.69314718055994531;  // x = half * (score * by)
    double power = half * a.softcap * 1.4426950408889634;
    for (int i = 0; i < 5; i++, power *= half * half) s.odd[i] = (float)(kTanh[i] * power);
    return s;
}
__device__ __forceinline__ float capped(const Score& s, float x) {
    const float y = x * s.by, e = __builtin_amdgcn_exp2f(y), z = y * y;
    const float far = s.cap * (1.0f - 2.0f * __builtin_amdgcn_rcpf(1.0f + e));
    const float near =
        y * fmaf(z, fmaf(z, fmaf(z, fmaf(z, s.odd[4], s.odd[3]), s.odd[2]), s.odd[1]), s.odd[0]);
    return fabsf(y) < kLog2e ? near : far;
}
// Off by up to 1.5e-7 of the cap instead, whatever the score: in steps that
// every row sees all of, for caps up to kQuickCap, where that is at most 1e-5 of
// a score, a 400th of a weight's rounding to BF16 (2048 tokens of 32 heads of
// 128 on 8192 keys: 308 us, 399 with the other).  It rounds small scores
// all the same way, so no number of keys evens it out: with a cap of 1e5
// weights would be a hundredth off, with 1e8 the scores would be gone.
constexpr float kQuickCap = 64.0f;
enum { kUncapped = 0, kQuick = 1, kExact = 2 };  // what such steps compute
__device__ __forceinline__ float capped_quickly(const Score& s, float x) {
    const float e = __builtin_amdgcn_exp2f(x * s.by);
    return s.cap * (1.0f - 2.0f * __builtin_amdgcn_rcpf(1.0f + e));
}

// Infinities and NaN among BF16 word pairs: bits 15 and 31 of the result are
// set where a half's exponent is all ones (results may be or-ed together)
__device__ __forceinline__ uint32_t odd_halves(uint32_t w) {
    return (w & 0x7F807F80u) + 0x00800080u;
}
__device__ __forceinline__ bool any_odd(uint32_t halves) { return (halves & 0x80008000u) != 0; }

// Whether a row sees a key, by the key's offset: the row's keys are low ..
// high - 1, offsets are from `base`
struct Sees {
    uint32_t first, count;
    __device__ __forceinline__ Sees(int32_t low, int32_t high, int32_t base)
        : first((uint32_t)(low - base)), count(high > low ? (uint32_t)(high - low) : 0u) {}
    __device__ __forceinline__ bool operator()(uint32_t offset) const {
        return offset - first < count;
    }
};
// Such words taken out (0 in their place)
__device__ __forceinline__ uint32_t plain_pair(uint32_t w) {
    if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
    if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
    return w;
}
// Such words as marks, BF16 numbers: NaN 1, infinity 128, -infinity 16384.
// A sum of up to 127 marks of each kind is exact in FP32 and says which
// there were.
__device__ __forceinline__ uint32_t mark(uint32_t w) {
    if ((w & 0x7F80u) != 0x7F80u) return 0;
    if (w & 0x7Fu) return 0x3F80u;
    return w & 0x8000u ? 0x4680u : 0x4300u;
}
__device__ __forceinline__ uint32_t mark_pair(uint32_t w) {
    return mark(w & 0xFFFFu) | mark(w >> 16) << 16;
}
__device__ __forceinline__ float unmark(float marks) {
    const uint32_t n = (uint32_t)marks;
    float x = 0;
    if (n & 0x7Fu) x = NAN;
    if (n >> 7 & 0x7Fu) x += INFINITY;
    if (n >> 14) x -= INFINITY;
    return x;
}

// A page's address from a table, through the scalar cache: the tables do not
// change while a kernel runs, which the compiler cannot tell by itself in
// kernels that store inside a loop (a vector load there would wait for the
// loads of keys and values before it).
__device__ __forceinline__ uint64_t page_address(const uint64_t* table, uint64_t entry) {
    return *(const __attribute__((address_space(4))) uint64_t*)(uintptr_t)(table + entry);
}

// The resource of a block of 16 keys' rows in a page: rows from `skip` on
// (a page that no visible key lies in, or a bad page address: none) up to
// `rows`.  Offsets past the end read as zeros, so keys past the last visible
// one, elements past head_dim and unusable pages need no test at the loads.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t block_rows(const Cache& c, uint64_t page,
                                                             uint32_t slot, uint32_t head,
                                                             int32_t rows) {
    const uint64_t at = page + 2 * (slot * c.token_stride + head * c.head_stride);
    const bool good = good_page(page) && rows > 0;
    const uint32_t n = rows > 16 ? 15 : (uint32_t)rows - 1;
    const uint32_t bytes = good ? 2 * (n * (uint32_t)c.token_stride + c.head_dim) : 0;
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(good ? at : 0), 0, bytes,
                                             kBufferFlags);
}

// Results of a part: for (KV head, slot), tile_rows rows of dim sums and
// of (maximum, sum of weights).
struct Partial {
    float* o;
    float* ml;
};
__host__ __device__ inline uint64_t partial_slots(const AttendPlan& p) {
    return (uint64_t)p.tiles + p.shares;
}
__device__ __forceinline__ Partial partial_of(uint8_t* ws, const Attend& a, const AttendPlan& p,
                                              uint32_t kv, uint32_t slot, uint32_t dim) {
    const uint64_t slots = partial_slots(p);
    const uint64_t unit = kv * slots + slot;
    float* f = reinterpret_cast<float*>(ws);
    return Partial{f + 2 * (a.cache.kv_heads * slots << p.tile_log2) +
                       (unit << p.tile_log2) * dim,
                   f + 2 * (unit << p.tile_log2)};
}

// N finished elements of a row to the output, from element e on
template <int N>
__device__ __forceinline__ void store_out(const Rows& out, uint64_t at, const float (&x)[N]) {
    if (out.f32) {
        float* p = static_cast<float*>(out.data) + at;
#pragma unroll
        for (int i = 0; i < N; i += 4)
            store_global(reinterpret_cast<uint4*>(p + i),
                         make_uint4(__float_as_uint(x[i]), __float_as_uint(x[i + 1]),
                                    __float_as_uint(x[i + 2]), __float_as_uint(x[i + 3])));
        return;
    }
    uint16_t* p = static_cast<uint16_t*>(out.data) + at;
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; i++) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
#pragma unroll
    for (int i = 0; i + 4 <= N / 2; i += 4)
        store_global(reinterpret_cast<uint4*>(p + 2 * i),
                     make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]));
    if constexpr (N == 4) {
        const u32x2 v = {w[0], w[1]};
        *(SZ_GLOBAL u32x2*)p = v;
    }
}

// 1 / l; 0 where no key was seen
__device__ __forceinline__ float inverse(float l) { return l == 0 ? 0.0f : 1.0f / l; }
__device__ __forceinline__ float log_sum(float m, float l) {
    return l == 0 ? -INFINITY : (m + log2f(l)) * kLn2;
}

// A barrier after which every wave's writes to LDS are there; loads from
// memory that are under way stay so.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// N times 64 lanes' 16 bytes each, from offsets of a buffer to consecutive LDS
// bytes, 1024 a time; offsets past the buffer's end store zeros.  Completion is
// counted by vmcnt.  A load reads m0 and the resource's scalar registers, and
// the hardware waits for neither: one state must lie between a scalar write of
// m0 and the load, five between a vector instruction's write of a scalar
// register (a lane read back, a reload of a spilled one) and it.  The compiler
// keeps to that only around instructions that it knows, so the block itself
// waits: the move and four states after it, once for all loads (a block for
// every two or four of them: 2048 tokens of 64 heads of 128 on 32768 keys 2108
// us, not 1908; of 16 heads of 256 on 8192 296, not 267).
// (m0 is the compiler's to write just before an instruction that reads it and
// never holds a value across others: it refuses it as a clobber.)
template <int N>
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t from, const uint32_t* at,
                                            uint32_t lds) {
#define SZ_FIRST_LOAD "s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %2, %1, 0 offen lds\n\t"
#define SZ_NEXT_LOAD(at) \
    "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tbuffer_load_dwordx4 " at ", %1, 0 offen lds\n\t"
    static_assert(N == 2 || N == 4 || N == 8, "");
    if constexpr (N == 2) {
        asm volatile(SZ_FIRST_LOAD SZ_NEXT_LOAD("%3")
                     :
                     : "s"(lds), "s"(from), "v"(at[0]), "v"(at[1])
                     : "memory", "scc");
    } else if constexpr (N == 4) {
        asm volatile(SZ_FIRST_LOAD SZ_NEXT_LOAD("%3") SZ_NEXT_LOAD("%4") SZ_NEXT_LOAD("%5")
                     :
                     : "s"(lds), "s"(from), "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3])
                     : "memory", "scc");
    } else {
        asm volatile(SZ_FIRST_LOAD SZ_NEXT_LOAD("%3") SZ_NEXT_LOAD("%4") SZ_NEXT_LOAD("%5")
                         SZ_NEXT_LOAD("%6") SZ_NEXT_LOAD("%7") SZ_NEXT_LOAD("%8") SZ_NEXT_LOAD("%9")
                     :
                     : "s"(lds), "s"(from), "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]),
                       "v"(at[4]), "v"(at[5]), "v"(at[6]), "v"(at[7])
                     : "memory", "scc");
    }
#undef SZ_FIRST_LOAD
#undef SZ_NEXT_LOAD
}

}  // namespace
}  // namespace sz
