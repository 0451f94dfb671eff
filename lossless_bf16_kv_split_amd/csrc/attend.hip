// attend.hip -- attention of new tokens over a paged BF16 KV cache.
//
// For a query row q at position c and the keys j visible to it (j < len,
// causal j <= c, window j > c - W):
//   s_j = scale * q.k_j, or softcap * tanh(scale * q.k_j / softcap)
//   m = max s_j, l = sum exp(s_j - m), o = sum exp(s_j - m) v_j / l
// in one pass over the keys with a running m and l.
#include "kv_internal.h"

namespace sz {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

__device__ __forceinline__ void unpack(uint4 w, float (&x)[8]) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        x[2 * i] = __uint_as_float(v[i] << 16);
        x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
    }
}

// One wave per (token, query head).  LANES lanes share a key, 8 elements
// each, so a wave takes 64 / LANES keys a step, each group with its own
// running statistics, joined at the end.
template <int LANES>
__global__ __launch_bounds__(kWave) void k_attend_rows(Attend a) {
    const uint32_t lane = threadIdx.x, l = lane % LANES, g = lane / LANES;
    constexpr uint32_t kGroups = kWave / LANES;
    const uint64_t token = blockIdx.x / a.q.heads;
    const uint32_t h = blockIdx.x % a.q.heads;
    const uint32_t s = find_seq(a.batch.n_seqs, (int64_t)token,
                                [&](uint32_t i) { return (int64_t)a.batch.starts[i]; });
    const Seq q = load_seq(a.batch, s, a.max_len);
    if (!q.good || (int64_t)token < q.begin || (int64_t)token >= q.end) return;
    const uint32_t kv = h / (a.q.heads / a.cache.kv_heads);
    const int64_t c = (int64_t)q.len - q.end + (int64_t)token;
    int64_t from = 0, upto = q.len;
    if (a.causal) {
        upto = c + 1 < upto ? c + 1 : upto;
        if (a.window != 0 && c >= 0 && (uint64_t)c + 1 > a.window) from = c + 1 - (int64_t)a.window;
    }
    const bool live = l * 8 < a.cache.head_dim;
    float x[8] = {};
    if (live)
        unpack(load_global(reinterpret_cast<const uint4*>(
                   static_cast<const uint16_t*>(a.q.data) + token * a.q.token_stride +
                   h * a.q.head_stride + l * 8)), x);
    float m = -INFINITY, sum = 0, o[8] = {};
    const uint64_t row = (uint64_t)s * a.cache.table_pitch;
    for (int64_t j0 = from; j0 < upto; j0 += kGroups) {
        const int64_t j = j0 + g;
        const bool seen = j < upto;
        float k[8] = {}, v[8] = {};
        if (seen && live) {
            const uint64_t entry = row + ((uint64_t)j >> a.cache.page_log2);
            const uint64_t at = ((uint64_t)j & ((1u << a.cache.page_log2) - 1)) *
                                    a.cache.token_stride + kv * a.cache.head_stride + l * 8;
            const uint64_t kp = a.cache.k_pages[entry], vp = a.cache.v_pages[entry];
            if (good_page(kp))
                unpack(load_global(reinterpret_cast<const uint4*>(
                           reinterpret_cast<const uint16_t*>(kp) + at)), k);
            if (good_page(vp))
                unpack(load_global(reinterpret_cast<const uint4*>(
                           reinterpret_cast<const uint16_t*>(vp) + at)), v);
        }
        float dot = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) dot = fmaf(x[i], k[i], dot);
#pragma unroll
        for (int d = 1; d < LANES; d *= 2) dot += __shfl_xor(dot, d);
        float z = dot * a.scale;
        if (a.softcap > 0) z = a.softcap * tanhf(z / a.softcap);
        if (!seen) continue;
        const float top = fmaxf(m, z);
        const float keep = m == -INFINITY ? 0.0f : expf(m - top);
        const float p = top == -INFINITY ? 0.0f : expf(z - top);
        sum = sum * keep + p;
#pragma unroll
        for (int i = 0; i < 8; i++) o[i] = fmaf(p, v[i], o[i] * keep);
        m = top;
    }
#pragma unroll
    for (int d = LANES; d < (int)kWave; d *= 2) {
        const float other = __shfl_xor(m, d), top = fmaxf(m, other);
        const float mine = m == -INFINITY ? 0.0f : expf(m - top);
        const float theirs = other == -INFINITY ? 0.0f : expf(other - top);
        sum = sum * mine + __shfl_xor(sum, d) * theirs;
#pragma unroll
        for (int i = 0; i < 8; i++) o[i] = o[i] * mine + __shfl_xor(o[i], d) * theirs;
        m = top;
    }
    const float inv = sum > 0 ? 1.0f / sum : sum == 0 ? 0.0f : sum;
    if (g == 0 && live) {
        const uint64_t at = token * a.out.token_stride + h * a.out.head_stride + l * 8;
        if (a.out.f32) {
            float* p = static_cast<float*>(a.out.data) + at;
#pragma unroll
            for (int i = 0; i < 8; i++) p[i] = o[i] * inv;
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; i++) w[i] = pack_bf16(o[2 * i] * inv, o[2 * i + 1] * inv);
            store_global(reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out.data) + at),
                         make_uint4(w[0], w[1], w[2], w[3]));
        }
    }
    if (lane == 0 && a.lse != nullptr)
        a.lse[token * a.q.heads + h] = sum == 0 ? -INFINITY : m + logf(sum);
}

}  // namespace

uint64_t attend_workspace(uint32_t, const Cache&, uint64_t, uint64_t, uint64_t) { return 0; }

hipError_t launch_attend(const Attend& a, uint8_t*, hipStream_t stream) {
    if (a.batch.n_seqs == 0 || a.batch.n_tokens == 0) return hipSuccess;
    const dim3 grid((uint32_t)(a.batch.n_tokens * a.q.heads)), block(kWave);
    if (a.cache.head_dim <= 64) k_attend_rows<8><<<grid, block, 0, stream>>>(a);
    else if (a.cache.head_dim <= 128) k_attend_rows<16><<<grid, block, 0, stream>>>(a);
    else k_attend_rows<32><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace sz
