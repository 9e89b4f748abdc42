// Attention of a ragged batch of new tokens over a paged cache.
//
//   out[t][h] = sum_u softmax_u(scale q[t][h] . K[g][u]) V[g][u],  u in (p - window, p]
//
// for the token at position p, one pass over u with the running maximum and sum.
// One warp per (token, query head): every lane holds four of the 128 dims.
#include <cmath>

#include "chunk.cuh"
#include "common.cuh"

namespace i4 {

struct ChunkAttnParams {
    const uint16_t *q, *k_pool, *v_pool;
    long long q_stride;
    const int32_t *page_table, *q_start, *ctx_len;
    uint16_t *out;
    int T, B, Hq, Hkv, page_size, max_pages, num_pages, window;
    float scale;
};

__device__ __forceinline__ float4 load4(const uint16_t *p) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&v.x)), b = __half22float2(*reinterpret_cast<const __half2 *>(&v.y));
    return make_float4(a.x, a.y, b.x, b.y);
}

__global__ void __launch_bounds__(256) chunk_attn_kernel(const ChunkAttnParams p) {
    const int t = blockIdx.x, g = blockIdx.y, lane = threadIdx.x & 31, G = p.Hq / p.Hkv;
    const int h = g * G + (threadIdx.x >> 5);
    const int b = chunk_find(p.q_start, p.B, t);
    if (b >= p.B) return;
    const int2 rows = chunk_rows(p.q_start, b, p.T);
    if (t < rows.x) return;
    const int pos = p.ctx_len[b] - rows.y + (t - rows.x);
    const int hi = min(pos + 1, p.max_pages * p.page_size), lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
    const float4 q = load4(p.q + (size_t)t * p.q_stride + (size_t)h * 128 + 4 * lane);
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int u = lo; u < hi; ++u) {
        const int page = p.page_table[(size_t)b * p.max_pages + u / p.page_size];
        float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;  // a page that is not there reads as zeros
        if (page >= 0 && page < p.num_pages) {
            const size_t off = (((size_t)page * p.Hkv + g) * p.page_size + u % p.page_size) * 128 + 4 * lane;
            k = load4(p.k_pool + off);
            v = load4(p.v_pool + off);
        }
        const float s = warp_sum(q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w) * p.scale;
        const float mn = fmaxf(m, s), a = m == -INFINITY ? 0.f : expf(m - mn), e = expf(s - mn);
        l = l * a + e;
        o = make_float4(o.x * a + e * v.x, o.y * a + e * v.y, o.z * a + e * v.z, o.w * a + e * v.w);
        m = mn;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t *dst = p.out + ((size_t)t * p.Hq + h) * 128 + 4 * lane;
    dst[0] = float_to_half_bits(o.x * inv);
    dst[1] = float_to_half_bits(o.y * inv);
    dst[2] = float_to_half_bits(o.z * inv);
    dst[3] = float_to_half_bits(o.w * inv);
}

}  // namespace i4

using namespace i4;

extern "C" size_t i4_paged_gqa_chunk_ws_bytes(void) { return 256; }

extern "C" int i4_paged_gqa_chunk(const uint16_t *q, long long q_stride, const uint16_t *k_pool, const uint16_t *v_pool,
                                  const int32_t *page_table, const int32_t *q_start, const int32_t *ctx_len, uint16_t *out, int T,
                                  int B, int Hq, int Hkv, int D, int page_size, int max_pages_per_seq, int num_pages, int window,
                                  int max_q, float scale, void *ws, size_t ws_bytes, void *stream) {
    if (!q || !k_pool || !v_pool || !page_table || !q_start || !ctx_len || !out)
        return fail(I4_EINVAL, "i4_paged_gqa_chunk: null pointer");
    if (T < 1 || B < 1 || Hq < 1 || Hkv < 1 || max_pages_per_seq < 1 || num_pages < 1 || window < 0 || max_q < 0)
        return fail(I4_EINVAL, "i4_paged_gqa_chunk: bad sizes T=%d B=%d Hq=%d Hkv=%d window=%d", T, B, Hq, Hkv, window);
    if (D != 128) return fail(I4_EUNSUPPORTED, "i4_paged_gqa_chunk: head_dim %d (only 128)", D);
    if (Hq % Hkv || Hq / Hkv > 8) return fail(I4_EUNSUPPORTED, "i4_paged_gqa_chunk: Hq/Hkv must be an integer <= 8");
    if (page_size < 8 || page_size > 128 || (page_size & (page_size - 1)))
        return fail(I4_EUNSUPPORTED, "i4_paged_gqa_chunk: page_size %d must be a power of two in [8, 128]", page_size);
    if (T > (1 << 20) || B > 65536 || Hkv > 4096 || (long long)max_pages_per_seq * page_size > (1 << 20))
        return fail(I4_EUNSUPPORTED, "i4_paged_gqa_chunk: more than 2^20 tokens, 65536 sequences or 4096 kv heads");
    if (!(scale > 0.f) || std::isinf(scale)) return fail(I4_EINVAL, "i4_paged_gqa_chunk: scale %g must be positive", scale);
    if (q_stride < (long long)Hq * D || q_stride % 8)
        return fail(I4_EINVAL, "i4_paged_gqa_chunk: q_stride %lld must be >= Hq*D and a multiple of 8", q_stride);
    if (!aligned(q, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(out, 16) || !aligned(page_table, 4) ||
        !aligned(q_start, 4) || !aligned(ctx_len, 4))
        return fail(I4_EALIGN, "i4_paged_gqa_chunk: q, the pools and out must be 16-byte aligned");
    const size_t need = i4_paged_gqa_chunk_ws_bytes();
    if (!ws || ws_bytes < need) return fail(I4_EINVAL, "i4_paged_gqa_chunk: workspace of %zu bytes needed (got %zu)", need, ws_bytes);
    if (!aligned(ws, 256)) return fail(I4_EALIGN, "i4_paged_gqa_chunk: workspace must be 256-byte aligned");
    const ChunkAttnParams p = {q,   k_pool, v_pool, q_stride, page_table, q_start,           ctx_len,   out,    T,
                               B,   Hq,     Hkv,    page_size, max_pages_per_seq, num_pages, window, scale};
    chunk_attn_kernel<<<dim3(T, Hkv), 32 * (Hq / Hkv), 0, (cudaStream_t)stream>>>(p);
    return launch_check("i4_paged_gqa_chunk");
}
