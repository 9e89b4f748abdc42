// Rotary positions of a ragged batch of new tokens and the append of their K/V
// rows to the pages, with the table of angles it reads.
//
//   (a, b) -> (a cos - b sin, b cos + a sin),  cos, sin = cs[position][i]
//
// over the pairs (i, i + rd/2) or (2i, 2i + 1) of the first rd values of every
// query and key head; the rest of the head and the values pass unchanged.
//
// The table is made once like weights, in 64 bits: an fp32 angle at position
// 100000 is off by up to 0.004 rad, more than the fp16 step of the result.
// Frequencies f_i = theta^(-2i/rd), divided by `factor` (linear), or blended
// between f_i and f_i / factor by how often pair i turns over the original
// context, with cos and sin scaled by 0.1 ln(factor) + 1 (YaRN, Peng et al. 2023).
#include <cmath>

#include "chunk.cuh"
#include "common.cuh"

namespace i4 {

struct RopeFreqs {
    double f[64];
    double scale;
};

__global__ void rope_chunk_table_kernel(float2 *cs, int max_pos, int half, const __grid_constant__ RopeFreqs fr) {
    const long long n = (long long)max_pos * half;
    for (long long idx = blockIdx.x * (long long)blockDim.x + threadIdx.x; idx < n;
         idx += (long long)gridDim.x * blockDim.x) {
        double s, c;
        sincos((double)(idx / half) * fr.f[idx % half], &s, &c);
        cs[idx] = make_float2((float)(c * fr.scale), (float)(s * fr.scale));
    }
}

constexpr int kRopeHeads = 4;

struct RopeChunkParams {
    const uint16_t *qkv;
    long long qkv_stride;
    const int32_t *q_start, *ctx_len, *page_table;
    const float2 *cs;
    uint16_t *q_out, *k_pool, *v_pool;
    int max_pos, T, B, Hq, Hkv, rd, page_size, max_pages, num_pages;
};

// One CTA per token. Sixteen lanes take one head, eight values (16 bytes) each, and a lane's partner values come
// from the lane rd/16 away by shuffles (half layout) or are its own neighbours (interleaved). The angles of a lane are
// the same for every head, so they are read once. Bound by HBM for many tokens and by the chain of dependent loads
// (sequence, position, page and angles) for few: the first heads' values, which depend on none of it, are loaded first.
// A thread takes kHeads heads at once; finding the token's place costs it as much as two or three of them (16397 tokens of
// 36 heads, half of each rotated, 306 MB: 56 us with two, issue slots 77 % busy; 50 us with four, 6.2 TB/s, 95 % of the copy
// rate). Eight single tokens take 3.4 us with the launch, a prompt of 512 5.1.
template <bool kInterleaved, int kHeads>
__global__ void __launch_bounds__(512) rope_append_chunk_kernel(const RopeChunkParams p) {
    grid_dep_wait();
    grid_dep_launch();
    const int t = blockIdx.x;
    const int c = threadIdx.x & 15;  // 16-byte chunk of the head
    const int heads = p.Hq + 2 * p.Hkv, step = blockDim.x >> 4, h_first = threadIdx.x >> 4;
    const uint16_t *src = p.qkv + (size_t)t * p.qkv_stride + 8 * c;
    uint4 v[kHeads];
    auto load = [&](int h0) {
#pragma unroll
        for (int k = 0; k < kHeads; ++k) {
            v[k] = make_uint4(0, 0, 0, 0);
            if (h0 + k * step < heads) v[k] = __ldcs(reinterpret_cast<const uint4 *>(src + (size_t)(h0 + k * step) * 128));
        }
    };
    load(h_first);
    const int b = chunk_find(p.q_start, p.B, t);
    if (b >= p.B) return;  // a row behind the last sequence
    const int2 rows = chunk_rows(p.q_start, b, p.T);
    const int pos = max(p.ctx_len[b], 0) - rows.y + (t - rows.x);
    const int in_row = (int)((unsigned)pos / (unsigned)p.page_size), slot = pos - in_row * p.page_size;
    if (t < rows.x || pos < 0 || pos >= p.max_pos || in_row >= p.max_pages) return;
    const int page = p.page_table[(size_t)b * p.max_pages + in_row];
    const bool page_ok = page >= 0 && page < p.num_pages;

    const int h16 = p.rd / 16;           // chunks of one half of the rotated part
    const bool turn = c < 2 * h16;
    const bool low = c < h16;
    const int partner = !turn ? c : (low ? c + h16 : c - h16);
    // angles: half layout, values 8c.. of the head are pairs 8c.. (low) or 8(c - h16).. (high); interleaved, pairs 4c..
    float2 cs[8];
    const float2 *row = p.cs + (size_t)pos * (p.rd / 2);
#pragma unroll
    for (int i = 0; i < (kInterleaved ? 4 : 8); i += 2) {
        float4 a = make_float4(1.f, 0.f, 1.f, 0.f);
        if (turn)
            a = *reinterpret_cast<const float4 *>(row + (kInterleaved ? 4 * c : 8 * (low ? c : c - h16)) + i);
        cs[i] = make_float2(a.x, a.y);
        cs[i + 1] = make_float2(a.z, a.w);
    }
    // the same trips for every thread: the shuffles need whole warps
    for (int h0 = h_first; h0 - h_first < heads; h0 += kHeads * step) {
        if (h0 != h_first) load(h0);
#pragma unroll
        for (int k = 0; k < kHeads; ++k) {
            const int h = h0 + k * step;
            uint32_t x[4] = {v[k].x, v[k].y, v[k].z, v[k].w}, y[4];
            if (kInterleaved) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x[i]));
                    const __half2 r = __floats2half2_rn(fmaf(f.x, cs[i].x, -f.y * cs[i].y), fmaf(f.y, cs[i].x, f.x * cs[i].y));
                    y[i] = *reinterpret_cast<const uint32_t *>(&r);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t o = __shfl_sync(0xffffffffu, x[i], partner, 16);
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x[i]));
                    const float2 g = __half22float2(*reinterpret_cast<const __half2 *>(&o));
                    const float s0 = low ? -cs[2 * i].y : cs[2 * i].y, s1 = low ? -cs[2 * i + 1].y : cs[2 * i + 1].y;
                    const __half2 r =
                        __floats2half2_rn(fmaf(f.x, cs[2 * i].x, g.x * s0), fmaf(f.y, cs[2 * i + 1].x, g.y * s1));
                    y[i] = *reinterpret_cast<const uint32_t *>(&r);
                }
            }
            if (h >= heads) continue;
            if (!turn || h >= p.Hq + p.Hkv)  // not rotated: the bits as they are
                for (int i = 0; i < 4; ++i) y[i] = x[i];
            uint16_t *dst;
            if (h < p.Hq) {
                dst = p.q_out + ((size_t)t * p.Hq + h) * 128;
            } else {
                if (!page_ok) continue;
                const int g = h < p.Hq + p.Hkv ? h - p.Hq : h - p.Hq - p.Hkv;
                dst = (h < p.Hq + p.Hkv ? p.k_pool : p.v_pool) + (((size_t)page * p.Hkv + g) * p.page_size + slot) * 128;
            }
            *reinterpret_cast<uint4 *>(dst + 8 * c) = make_uint4(y[0], y[1], y[2], y[3]);
        }
    }
}

}  // namespace i4

using namespace i4;

extern "C" int i4_rope_table(float *cs, int max_pos, int rotary_dim, double theta, int scaling, double factor,
                             int original_ctx, void *stream) {
    if (!cs) return fail(I4_EINVAL, "i4_rope_table: null pointer");
    if (max_pos < 1 || !(theta > 1.0) || !std::isfinite(theta))
        return fail(I4_EINVAL, "i4_rope_table: max_pos %d, theta %g", max_pos, theta);
    if (rotary_dim < 16 || rotary_dim > 128 || rotary_dim % 16)
        return fail(I4_EUNSUPPORTED, "i4_rope_table: rotary_dim %d (a multiple of 16 up to 128)", rotary_dim);
    if (scaling < I4_ROPE_NONE || scaling > I4_ROPE_YARN) return fail(I4_EINVAL, "i4_rope_table: scaling %d", scaling);
    if (scaling != I4_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
        return fail(I4_EINVAL, "i4_rope_table: factor %g must be at least 1", factor);
    if (scaling == I4_ROPE_YARN && original_ctx < 1)
        return fail(I4_EINVAL, "i4_rope_table: original_ctx %d", original_ctx);
    if (!aligned(cs, 16)) return fail(I4_EALIGN, "i4_rope_table: cs must be 16-byte aligned");
    RopeFreqs fr = {};
    const int half = rotary_dim / 2;
    fr.scale = scaling == I4_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
    double lo = 0, hi = 0;
    if (scaling == I4_ROPE_YARN) {
        // the pairs that turn 32 times and once over the original context
        const double per = rotary_dim / (2 * std::log(theta)), two_pi = 6.283185307179586;
        lo = std::floor(per * std::log(original_ctx / (32 * two_pi)));
        hi = std::ceil(per * std::log(original_ctx / two_pi));
        lo = lo < 0 ? 0 : lo;
        hi = hi > rotary_dim - 1 ? rotary_dim - 1 : hi;
        if (hi <= lo) hi = lo + 0.001;
    }
    for (int i = 0; i < half; ++i) {
        const double f = std::pow(theta, -2.0 * i / rotary_dim);
        fr.f[i] = f;
        if (scaling == I4_ROPE_LINEAR) fr.f[i] = f / factor;
        if (scaling == I4_ROPE_YARN) {
            double r = (i - lo) / (hi - lo);
            r = r < 0 ? 0 : (r > 1 ? 1 : r);
            fr.f[i] = f / factor * r + f * (1 - r);
        }
    }
    rope_chunk_table_kernel<<<8 * kNumSMs, 256, 0, (cudaStream_t)stream>>>(reinterpret_cast<float2 *>(cs), max_pos, half,
                                                                         fr);
    return launch_check("i4_rope_table");
}

extern "C" int i4_rope_append_chunk(const i4_rope_chunk_args *args, void *stream) {
    if (!args) return fail(I4_EINVAL, "i4_rope_append_chunk: null args");
    const auto [qkv, qkv_stride, q_start, ctx_len, cs, q_out, k_pool, v_pool, page_table, max_pos, rotary_dim, interleaved, T, B,
                Hq, Hkv, D, page_size, max_pages_per_seq, num_pages] = *args;
    if (!qkv || !q_start || !ctx_len || !cs || !q_out || !k_pool || !v_pool || !page_table)
        return fail(I4_EINVAL, "i4_rope_append_chunk: null pointer");
    if (D != 128) return fail(I4_EUNSUPPORTED, "i4_rope_append_chunk: head_dim %d (only 128)", D);
    if (rotary_dim < 16 || rotary_dim > 128 || rotary_dim % 16)
        return fail(I4_EUNSUPPORTED, "i4_rope_append_chunk: rotary_dim %d (a multiple of 16 up to 128)", rotary_dim);
    if (T < 1 || B < 1 || Hq < 1 || Hkv < 1 || max_pos < 1 || page_size < 1 || max_pages_per_seq < 1 || num_pages < 1 ||
        Hq > 4096 || Hkv > 4096)
        return fail(I4_EINVAL, "i4_rope_append_chunk: bad sizes T=%d B=%d Hq=%d Hkv=%d", T, B, Hq, Hkv);
    if (qkv_stride < (long long)(Hq + 2 * Hkv) * D || qkv_stride % 8)
        return fail(I4_EINVAL, "i4_rope_append_chunk: qkv_stride %lld must be >= (Hq + 2 Hkv) D and a multiple of 8",
                    qkv_stride);
    if (!aligned(qkv, 16) || !aligned(cs, 16) || !aligned(q_out, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) ||
        !aligned(q_start, 4) || !aligned(ctx_len, 4) || !aligned(page_table, 4))
        return fail(I4_EALIGN, "i4_rope_append_chunk: qkv, cs, q_out and the pools must be 16-byte aligned");
    const RopeChunkParams p = {qkv,    qkv_stride, q_start, ctx_len, page_table, reinterpret_cast<const float2 *>(cs),
                               q_out,  k_pool,     v_pool,  max_pos, T,          B,
                               Hq,     Hkv,        rotary_dim, page_size, max_pages_per_seq, num_pages};
    // four heads per sixteen lanes, whole warps, at most 512 threads
    int threads = 16 * ((Hq + 2 * Hkv + kRopeHeads - 1) / kRopeHeads);
    threads = (threads + 31) / 32 * 32;
    threads = threads > 512 ? 512 : threads;
    return cuda_check(launch(interleaved ? rope_append_chunk_kernel<true, kRopeHeads> : rope_append_chunk_kernel<false, kRopeHeads>,
                             dim3(T), dim3(threads), 0, (cudaStream_t)stream, g_pdl, p),
                      "i4_rope_append_chunk");
}
