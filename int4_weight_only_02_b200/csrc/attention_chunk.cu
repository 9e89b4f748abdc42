// Attention of a ragged batch of new tokens over a paged cache, on tcgen05.
//
//   out[t][h] = sum_u softmax_u(scale q[t][h] . K[g][u]) V[g][u],  u in (p - window, p]
//
// for the token at position p, in one pass over u with the running maximum and
// sum of the softmax.
//
//  * Rows. The G = Hq / Hkv query heads that share a kv head are rows of one
//    matrix: row r of a sequence is (token r / G, head r % G), so 128 rows (the M of an
//    MMA) are 128 / G consecutive tokens, every K/V tile is read once for all of them, and a
//    short chunk fills the rows better than one head's tokens would.
//  * Work. A unit is NQ * 128 rows of one sequence and one kv head; its cost is the
//    number of 128-position tiles that its rows see. The units stand in one line (kv heads
//    outermost) and every CTA, one or two per SM, takes an equal stretch of the line's tiles, whatever
//    unit borders lie in it: a prompt's long and short units balance, and a
//    single token's long context spreads over the GPU. A unit that is cut
//    leaves its parts (m, l, O) in the workspace and a second kernel joins them in order.
//    The lengths are read on the device: every CTA finds its stretch by itself with two block-wide scans.
//  * Data. One warp loads K and V tiles (32 KB) page by page with TMA into a ring, 128-byte
//    swizzled; a page outside the pools, or one that no row sees, is an
//    out-of-range coordinate, which fills zeros.
//  * Math. S = Q K^T (M = 128 rows, N = 128 positions, both operands K-major in
//    shared memory) into tensor memory; the 128 threads of a warpgroup own one row
//    each, so maximum and sum need no exchange; P = 2^(S - m), rounded to fp16 (the tensor cores' operand
//    type; 2^-11 of each weight), goes back over S's columns and is the A operand of O += P V (V MN-major). m only
//    follows the row's maximum when that is more than 2^8 ahead, so O is rarely rescaled: P then reaches
//    at most 2^8, far inside fp16. l and O are fp32.
//  * Overlap. With NQ = 2 two warpgroups hold 128 rows each and alternate: the tensor cores
//    run one's P V and next Q K^T while the other computes its exponentials. With NQ = 1 two CTAs share an SM.
#include <cmath>

#include "chunk.cuh"
#include "common.cuh"
#include "mma.cuh"
#include "tc.cuh"

namespace i4 {

constexpr int kRows = 128;                         // rows of a slot: the MMA's M
constexpr int kTile = 128;                         // positions of a K/V tile
constexpr unsigned kHalf = kTile * 128;            // 64 of the 128 dims of a tile, 128 bytes per row
constexpr unsigned kTileBytes = 2 * kHalf;         // 32 KB
constexpr int kMaxCtas = 2 * kNumSMs;
constexpr int kMinTiles = 2;                       // tiles that are worth a CTA of their own
constexpr float kGrow = 8.f;                       // powers of two that a row's maximum may run ahead of its m
constexpr float kLog2e = 1.4426950408889634f;

template <int NQ>
struct Cfg {
    static constexpr int kThreads = NQ * 128 + 64;  // softmax warpgroups, the MMA warp, the load warp
    static constexpr int kStages = NQ == 2 ? 5 : 2;
    static constexpr int kCtasPerSm = NQ == 2 ? 1 : 2;
    static constexpr int kUnitRows = NQ * kRows;
    static constexpr unsigned kTmemCols = NQ * 256;  // S / P and O of every slot
    static constexpr unsigned kSmem = 1024 + (NQ + kStages) * kTileBytes;
};

__device__ int g_chunk_error = 0;

// Where a unit is cut at the beginning of a CTA's stretch: what the joining kernel needs.
struct Cut {
    int valid, last, rows, row0, r0, g;  // parts: CTA c-1's last, then the first of c .. last; unit rows [r0, r0 + rows)
};

struct ChunkAttnParams {
    const uint16_t *q, *k_pool, *v_pool;
    long long q_stride;
    const int32_t *page_table, *q_start, *ctx_len;
    uint16_t *out;
    int T, B, Hq, Hkv, page_size, max_pages, num_pages, window;
    float scale;
    Cut *cuts;        // [kMaxCtas]
    float2 *part_ml;  // [2 * CTAs][unit rows]: (m in powers of two, l)
    float4 *part_o;   // [2 * CTAs][unit rows / 32][32 column quads][32 rows]
};

// ------------------------------------------------------------------ the line of units

// Positions that the rows [r, e) of a sequence with n tokens from position pos0 on may see: [x, y), empty when y <= x.
__device__ __forceinline__ int2 seen(const ChunkAttnParams &p, int pos0, int G, int r, int e) {
    const int hi = min(pos0 + (e - 1) / G + 1, p.max_pages * p.page_size);
    const int lo = p.window > 0 ? max(0, pos0 + r / G - p.window + 1) : 0;
    return make_int2(lo, hi);
}
__device__ __forceinline__ int2 tiles_of(int2 s) {
    return s.y > s.x ? make_int2(s.x / kTile, (s.y + kTile - 1) / kTile) : make_int2(0, 0);
}

// A CTA's stretch of the line.
struct Stretch {
    int g, b, i, off;  // first unit, and its tiles that belong to earlier CTAs
    int left;          // tiles of the stretch (a unit that sees nothing counts as one)
};

// One unit's part in a stretch.
struct Piece {
    int g, b, n, pos0, row0;  // kv head; sequence: tokens, first position, first row of q
    int r0, rows;             // the unit's rows of the sequence
    int2 see;                 // positions that the unit sees
    int t0, t1;               // the part's tiles
    int whole, slot;          // uncut, or the slot of its parts
};

// Walks the pieces of a stretch; every role of the CTA does so by itself.
template <int NQ>
struct Walker {
    const ChunkAttnParams &p;
    const int G;
    int g, b, i, off, left, n, pos0, row0, units;
    __device__ Walker(const ChunkAttnParams &p_, const Stretch &s)
        : p(p_), G(p_.Hq / p_.Hkv), g(s.g), b(s.b), i(s.i), off(s.off), left(s.left) {
        if (left > 0) load();
    }
    __device__ void load() {
        const int2 r = chunk_rows(p.q_start, b, p.T);
        row0 = r.x;
        n = r.y;
        pos0 = max(p.ctx_len[b], 0) - n;
        units = (n * G + Cfg<NQ>::kUnitRows - 1) / Cfg<NQ>::kUnitRows;
    }
    __device__ bool next(Piece &pc) {
        if (left <= 0) return false;
        pc.g = g;
        pc.b = b;
        pc.n = n;
        pc.pos0 = pos0;
        pc.row0 = row0;
        pc.r0 = i * Cfg<NQ>::kUnitRows;
        pc.rows = min(n * G - pc.r0, Cfg<NQ>::kUnitRows);
        pc.see = seen(p, pos0, G, pc.r0, pc.r0 + pc.rows);
        const int2 t = tiles_of(pc.see);
        const int cost = max(t.y - t.x, 1), take = min(cost - off, left);
        pc.t0 = t.x + off;
        pc.t1 = min(t.y, pc.t0 + take);
        pc.whole = take == cost;
        pc.slot = 2 * blockIdx.x + (off == 0);
        left -= take;
        off = 0;
        if (left > 0 && ++i == units) {
            i = 0;
            do {
                if (++b == p.B) {
                    b = 0;
                    ++g;
                }
                load();
            } while (units == 0);
        }
        return true;
    }
};

// Tiles of a piece that the rows of slot s see: [x, y), and how many rows it has.
__device__ __forceinline__ int3 slot_tiles(const ChunkAttnParams &p, int G, const Piece &pc, int s) {
    const int rows = min(max(pc.rows - s * kRows, 0), kRows);
    if (rows == 0) return make_int3(0, 0, 0);
    const int2 t = tiles_of(seen(p, pc.pos0, G, pc.r0 + s * kRows, pc.r0 + s * kRows + rows));
    const int x = max(t.x, pc.t0), y = min(t.y, pc.t1);
    return y > x ? make_int3(x, y, rows) : make_int3(0, 0, rows);
}

template <int NT>
__device__ __forceinline__ int scan_block(int v, int &total, int *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    __syncthreads();  // the sums of an earlier scan have been read
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        before += w < warp ? warp_sums[w] : 0;
        total += warp_sums[w];
    }
    return before + inc - v;
}

// This CTA's stretch (out, thread 0's view in shared memory) and the cut at its beginning. scratch: NT + 32 ints.
template <int NQ>
__device__ __forceinline__ void find_stretch(const ChunkAttnParams &p, Stretch *out, int *scratch) {
    constexpr int NT = Cfg<NQ>::kThreads, R = Cfg<NQ>::kUnitRows;
    const int tid = threadIdx.x, G = p.Hq / p.Hkv;
    int *sums = scratch, *first = scratch + 32;  // first[j]: units before sequence b0 + j
    if (tid == 0) *out = {0, 0, 0, 0, 0};
    long long W = 0, start = 0, end = 0;
    int n_ctas = 1, line = 0, target = 0;
    for (int pass = 0; pass < 2; ++pass) {  // the first measures the line, the second finds the place in it
        int run = 0;
        for (int b0 = 0; b0 < p.B; b0 += NT) {
            int nu = 0, total_units;
            if (b0 + tid < p.B) nu = (chunk_rows(p.q_start, b0 + tid, p.T).y * G + R - 1) / R;
            const int before = scan_block<NT>(nu, total_units, sums);
            first[tid] = before;
            __syncthreads();
            for (int u0 = 0; u0 < total_units; u0 += NT) {
                const int u = u0 + tid;
                int cost = 0, j = 0, i = 0;
                if (u < total_units) {
                    int len = min(NT, p.B - b0);  // the last sequence whose first unit is not behind u
                    while (len > 1) {
                        const int h = len >> 1;
                        if (first[j + h] <= u) {
                            j += h;
                            len -= h;
                        } else {
                            len = h;
                        }
                    }
                    i = u - first[j];
                    const int n = chunk_rows(p.q_start, b0 + j, p.T).y, r0 = i * R;
                    const int2 t = tiles_of(seen(p, max(p.ctx_len[b0 + j], 0) - n, G, r0, min(n * G, r0 + R)));
                    cost = max(t.y - t.x, 1);
                }
                int sum;
                const int at = run + scan_block<NT>(cost, sum, sums);
                if (pass == 1 && cost > 0 && target >= at && target < at + cost) {
                    const int g = (int)(start / line), off = target - at;
                    *out = {g, b0 + j, i, off, (int)(end - start)};
                    Cut cut = {0, 0, 0, 0, 0, 0};
                    const long long unit = start - off;  // where the unit begins
                    if (off > 0 && W * (blockIdx.x - 1) / n_ctas <= unit) {
                        // the first cut of this unit: its parts end in the CTA that holds its last tile
                        const int2 rows = chunk_rows(p.q_start, b0 + j, p.T);
                        cut = {1, (int)(((unit + cost) * n_ctas - 1) / W), min(rows.y * G - i * R, R), rows.x, i * R, g};
                    }
                    p.cuts[blockIdx.x] = cut;
                }
                run += sum;
            }
            __syncthreads();  // first[] is read no more
        }
        if (pass == 0) {
            line = run;
            W = (long long)line * p.Hkv;
            n_ctas = (int)min((long long)gridDim.x, max((W + kMinTiles - 1) / kMinTiles, 1ll));
            start = W * blockIdx.x / n_ctas;
            end = W * (blockIdx.x + 1) / n_ctas;
            if ((int)blockIdx.x >= n_ctas || start >= end) {
                if (tid == 0) p.cuts[blockIdx.x].valid = 0;
                break;
            }
            target = (int)(start % line);
        }
    }
    __syncthreads();
}

// ------------------------------------------------------------------ the kernel

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A wait that ends: on the barrier, when another role of the CTA gave up, or after ~2 s.
__device__ __forceinline__ bool wait_or_stop(uint64_t *bar, unsigned parity, volatile int *stop) {
    if (mbar_test(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_test(bar, parity)) {
        if (*stop) return false;
        if (clock64() - t0 > kWaitCycles) {
            *stop = 1;
            record_error(&g_chunk_error, 1);
            return false;
        }
    }
    return true;
}

// The sum over the positions [lo, hi) of one row by plain loads, for rows whose tensor-core sum met a NaN or an
// infinity: P = 0 times such a value of a position that other rows see is NaN, and must not count. Lane: dims 4 lane ..
// 4 lane + 3. The row's m and l are right already.
__device__ __noinline__ float4 plain_row(const ChunkAttnParams &p, int b, int g, const uint16_t *q, int lo, int hi, float qs,
                                         float m_scaled) {
    const int lane = threadIdx.x & 31;
    float o[4] = {0.f, 0.f, 0.f, 0.f}, x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = half_bits_to_float(q[4 * lane + i]);
    for (int u = lo; u < hi; ++u) {
        const int page = p.page_table[(size_t)b * p.max_pages + u / p.page_size];
        if (page < 0 || page >= p.num_pages) continue;  // zeros
        const size_t off = (((size_t)page * p.Hkv + g) * p.page_size + u % p.page_size) * 128 + 4 * lane;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) s = fmaf(x[i], half_bits_to_float(p.k_pool[off + i]), s);
        const float w = ex2(fmaf(warp_sum(s), qs, -m_scaled));
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = fmaf(w, half_bits_to_float(p.v_pool[off + i]), o[i]);
    }
    return make_float4(o[0], o[1], o[2], o[3]);
}

template <int NQ>
__global__ void __launch_bounds__(Cfg<NQ>::kThreads, Cfg<NQ>::kCtasPerSm)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ ChunkAttnParams p) {
    using C = Cfg<NQ>;
    constexpr int S = C::kStages, kMmaWarp = NQ * 4, kLoadWarp = NQ * 4 + 1;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t kv_full[S], kv_empty[S], q_full[NQ], s_full[NQ], p_full[NQ], o_full[NQ], o_free[NQ], all_done;
    __shared__ uint32_t tmem_base;
    __shared__ Stretch stretch;
    __shared__ int stop_flag;
    volatile int *stop = &stop_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = p.Hq / p.Hkv;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char *gbase = smem_raw + (base - smem_u32(smem_raw));
    const uint32_t ring = base + NQ * kTileBytes;

    find_stretch<NQ>(p, &stretch, reinterpret_cast<int *>(gbase));
    grid_dep_launch();  // the joining kernel may come up; it waits for this grid's end before it reads anything
    if (stretch.left <= 0) return;
    if (tid == 0) {
        stop_flag = 0;
        for (int i = 0; i < S; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 1);
        }
        for (int s = 0; s < NQ; ++s) {
            mbar_init(&q_full[s], 4);
            mbar_init(&s_full[s], 1);
            mbar_init(&p_full[s], 4);
            mbar_init(&o_full[s], 1);
            mbar_init(&o_free[s], 4);
        }
        mbar_init(&all_done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)),
                     "r"(C::kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = tmem_base;  // S / P of slot s at column 128 s, O of slot s at 128 (NQ + s)

    Walker<NQ> walk(p, stretch);
    Piece pc;
    if (warp == kLoadWarp) {
        // ---------------- K and V tiles: K0 V0 K1 V1 ...
        const int np = kTile / p.page_size;  // pages of a tile
        const int half = lane / np, pg = lane % np;
        const bool loads = lane < 2 * np;
        unsigned it = 0;
        bool ok = true;
        while (ok && walk.next(pc)) {
            for (int t = pc.t0; ok && t < pc.t1; ++t) {
                const int idx = t * np + pg;
                int page = p.num_pages;  // out of range: the copy fills zeros
                if (loads && idx * p.page_size < pc.see.y && (idx + 1) * p.page_size > pc.see.x) {
                    const int e = p.page_table[(size_t)pc.b * p.max_pages + idx];
                    if (e >= 0 && e < p.num_pages) page = e;
                }
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv, ++it) {
                    const unsigned st = it % S, use = it / S;
                    ok = use == 0 || wait_or_stop(&kv_empty[st], (use - 1) & 1, stop);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_expect_tx(&kv_full[st], kTileBytes);
                    __syncwarp();
                    if (loads)
                        tma_load_4d(ring + st * kTileBytes + half * kHalf + pg * p.page_size * 128, kv ? &tm_v : &tm_k, half * 64, 0,
                                    pc.g, page, &kv_full[st]);
                }
            }
        }
        if (!ok)  // let the copies in flight land before the CTA's memory goes
            for (unsigned k = it > S ? it - S : 0; k < it; ++k)
                if (lane == 0) mbar_wait(&kv_full[k % S], (k / S) & 1);
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ---------------- S = Q K^T and O += P V of every slot
        constexpr uint32_t idesc_qk = idesc_f16(kRows, kTile), idesc_pv = idesc_f16(kRows, 128) | kIdescBMajorMN;
        unsigned it = 0, uses[NQ], steps[NQ];  // pieces and tiles of every slot so far
#pragma unroll
        for (int s = 0; s < NQ; ++s) uses[s] = steps[s] = 0;
        bool ok = true;
        while (ok && walk.next(pc)) {
            int3 r[NQ];
#pragma unroll
            for (int s = 0; s < NQ; ++s) r[s] = slot_tiles(p, G, pc, s);
            for (int j = pc.t0 - 1; ok && j < pc.t1; ++j) {
                if (pc.t1 <= pc.t0) break;
                const unsigned iv = it + 2 * (j - pc.t0) + 1, ik = iv + 1, sv = iv % S, sk = ik % S;
                if (j >= pc.t0) {
                    ok = wait_or_stop(&kv_full[sv], (iv / S) & 1, stop);
                    const int t = j * kTile;
                    if (ok && (t < pc.see.x || t + kTile > pc.see.y)) {
                        // rows of V that the unit does not see may hold anything, NaN included: zero them
                        for (int e = lane; e < 2 * kTile * 8; e += 32) {
                            const int u = (e >> 3) & (kTile - 1);
                            if (t + u < pc.see.x || t + u >= pc.see.y)
                                *reinterpret_cast<uint4 *>(gbase + (NQ + sv) * kTileBytes + e * 16) = make_uint4(0, 0, 0, 0);
                        }
                        fence_async_smem();
                    }
                    __syncwarp();
                }
                if (ok && j + 1 < pc.t1) ok = wait_or_stop(&kv_full[sk], (ik / S) & 1, stop);
#pragma unroll
                for (int s = 0; s < NQ; ++s) {
                    if (ok && j >= r[s].x && j < r[s].y) {
                        ok = wait_or_stop(&p_full[s], steps[s] & 1, stop);
                        ++steps[s];
                        if (ok && j == r[s].x) {
                            if (uses[s] > 0) ok = wait_or_stop(&o_free[s], (uses[s] - 1) & 1, stop);
                            ++uses[s];
                        }
                        ok = __all_sync(0xffffffffu, ok);
                        fence_after_sync();
                        if (ok && lane == 0) {
                            const uint32_t tP = tmem + 128 * s, tO = tmem + 128 * (NQ + s), vb = ring + sv * kTileBytes;
#pragma unroll
                            for (int kk = 0; kk < kTile / 16; ++kk)
                                umma_f16_ta(tO, tP + 8 * kk, desc_sw128_mn(vb + kk * 2048, kHalf), idesc_pv,
                                            (j > r[s].x || kk > 0) ? 1 : 0);
                            if (j + 1 == r[s].y) umma_commit(&o_full[s]);
                        }
                        __syncwarp();
                    }
                    if (ok && j + 1 >= r[s].x && j + 1 < r[s].y) {
                        if (j + 1 == r[s].x) ok = wait_or_stop(&q_full[s], uses[s] & 1, stop);
                        ok = __all_sync(0xffffffffu, ok);
                        fence_after_sync();
                        if (ok && lane == 0) {
                            const uint32_t qb = base + s * kTileBytes, kb = ring + sk * kTileBytes;
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk) {
                                const uint32_t o = (kk >> 2) * kHalf + (kk & 3) * 32;
                                umma_f16(tmem + 128 * s, desc_sw128(qb + o), desc_sw128(kb + o), idesc_qk, kk > 0 ? 1 : 0);
                            }
                            umma_commit(&s_full[s]);
                        }
                        __syncwarp();
                    }
                }
                if (ok && lane == 0) {
                    if (j >= pc.t0) umma_commit(&kv_empty[sv]);
                    if (j + 1 < pc.t1) umma_commit(&kv_empty[sk]);
                }
                __syncwarp();
            }
            it += 2 * (pc.t1 > pc.t0 ? pc.t1 - pc.t0 : 0);
        }
        // nothing of this CTA is in flight on the tensor cores when it leaves
        if (lane == 0) {
            umma_commit(&all_done);
            if (!mbar_wait(&all_done, 0)) record_error(&g_chunk_error, 1);
        }
        __syncwarp();
    } else {
        // ---------------- softmax of slot s: thread = row
        const int s = warp >> 2, wq = warp & 3, row = tid & 127;
        const uint32_t lanes = (uint32_t)(32 * wq) << 16;
        const uint32_t tS = tmem + 128 * s + lanes, tO = tmem + 128 * (NQ + s) + lanes;
        const float qs = p.scale * kLog2e, grow = fminf(kGrow / qs, 1e30f);
        unsigned tiles = 0, pieces = 0;
        bool ok = true;

        // the last piece's results, stored once the next piece's rows of Q are on their way
        Piece last = {};
        int3 last_r = make_int3(0, 0, 0);
        float m = -INFINITY, l = 0.f;
        auto limits = [&](const Piece &c, int &lo, int &hi) {  // positions that this thread's row sees
            const int tok = (c.r0 + s * kRows + row) / G, pos = c.pos0 + tok;
            hi = min(pos + 1, p.max_pages * p.page_size);
            lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
        };
        auto finish = [&] {
            if (last_r.z == 0) return;  // the slot had no rows
            const bool mine = row < last_r.z, any = last_r.y > last_r.x;
            const int r = last.r0 + s * kRows + row, tok = r / G, head = last.g * G + r % G;
            const float l_inv = l == 0.f ? 0.f : 1.f / l;
            uint16_t *out = p.out + ((size_t)(last.row0 + tok) * p.Hq + head) * 128;
            const int slot_row = last.slot * C::kUnitRows + s * kRows + row;
            float4 *part = p.part_o + (((size_t)last.slot * (C::kUnitRows / 32) + s * 4 + wq) * 32) * 32 + lane;
            if (!last.whole && mine)  // an all-NaN row has l = NaN and no maximum: keep it from reading as empty
                p.part_ml[slot_row] = make_float2(l != l ? 0.f : (m == -INFINITY ? m : m * qs), l);
            if (any) {
                ok = __all_sync(0xffffffffu, wait_or_stop(&o_full[s], (pieces - 1) & 1, stop));
                if (!ok) return;
                fence_after_sync();
            }
            float bad = 0.f;  // stays 0 while every value of O is finite
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t o[32];
                if (any) {
                    tmem_ld32(tO + 32 * c, o);
                    tmem_wait_ld32(o);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0u;
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) bad = fmaf(__uint_as_float(o[i]), 0.f, bad);
                if (!mine) continue;
                if (last.whole) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t h[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            h[k] = h2_bits(__floats2half2_rn(__uint_as_float(o[8 * i + 2 * k]) * l_inv,
                                                             __uint_as_float(o[8 * i + 2 * k + 1]) * l_inv));
                        *reinterpret_cast<uint4 *>(out + 32 * c + 8 * i) = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                } else if (any) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        part[(8 * c + i) * 32] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                             __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
                }
            }
            if (any) {
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&o_free[s]);
            }
            // rows that met a NaN or an infinity, and whose own scores are fine, are summed again over what they see
            unsigned again = __ballot_sync(0xffffffffu, mine && any && !(bad == 0.f) && fabsf(l) < INFINITY);
            while (again) {
                const int k = __ffs(again) - 1;
                again &= again - 1;
                int lo, hi;
                limits(last, lo, hi);
                lo = max(__shfl_sync(0xffffffffu, lo, k), last_r.x * kTile);
                hi = min(__shfl_sync(0xffffffffu, hi, k), last_r.y * kTile);
                const float mk = __shfl_sync(0xffffffffu, m, k), inv = __shfl_sync(0xffffffffu, l_inv, k);
                const int tk = __shfl_sync(0xffffffffu, tok, k), hk = __shfl_sync(0xffffffffu, head, k);
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (mk > -INFINITY)
                    v = plain_row(p, last.b, last.g, p.q + (size_t)(last.row0 + tk) * p.q_stride + (size_t)hk * 128, lo, hi, qs, mk * qs);
                if (last.whole) {
                    uint16_t *d = p.out + ((size_t)(last.row0 + tk) * p.Hq + hk) * 128 + 4 * lane;
                    d[0] = float_to_half_bits(v.x * inv);
                    d[1] = float_to_half_bits(v.y * inv);
                    d[2] = float_to_half_bits(v.z * inv);
                    d[3] = float_to_half_bits(v.w * inv);
                } else {
                    p.part_o[(((size_t)last.slot * (C::kUnitRows / 32) + s * 4 + wq) * 32 + lane) * 32 + k] = v;
                }
            }
        };

        while (ok && walk.next(pc)) {
            const int3 r = slot_tiles(p, G, pc, s);
            if (r.y > r.x) {
                // this row of Q, or zeros, into the swizzled tile; every MMA that read the last one is done, since its
                // S has arrived
                const int rr = pc.r0 + s * kRows + row;
                const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (size_t)(pc.row0 + rr / G) * p.q_stride +
                                                                   (size_t)(pc.g * G + rr % G) * 128);
                unsigned char *dst = gbase + s * kTileBytes + row * 128;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint4 v[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c) v[c] = row < r.z ? src[8 * h + c] : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4 *>(dst + h * kHalf + ((c ^ (row & 7)) << 4)) = v[c];
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_full[s]);
            }
            finish();
            if (!ok) break;
            last = pc;
            last_r = r;
            m = -INFINITY;
            l = 0.f;
            if (r.y <= r.x) continue;
            ++pieces;
            int lo, hi;
            limits(pc, lo, hi);
            if (row >= r.z) {  // no row: anything goes, nothing is stored
                lo = 0;
                hi = 0x7fffffff;
            }
#pragma unroll 1
            for (int t = r.x; t < r.y; ++t, ++tiles) {
                ok = __all_sync(0xffffffffu, wait_or_stop(&s_full[s], tiles & 1, stop));
                if (!ok) break;
                fence_after_sync();
                uint32_t x[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, x + 32 * c);
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_wait_ld32(x + 32 * c);
                const int a = lo - t * kTile, e = hi - t * kTile;  // the row sees the tile's [a, e)
                if (__any_sync(0xffffffffu, a > 0 || e < kTile)) {
#pragma unroll
                    for (int i = 0; i < 128; ++i)
                        if (i < a || i >= e) x[i] = 0xff800000u;  // -inf
                }
                float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
                for (int i = 0; i < 128; i += 8) {
                    mx0 = fmaxf(mx0, fmaxf(__uint_as_float(x[i]), __uint_as_float(x[i + 1])));
                    mx1 = fmaxf(mx1, fmaxf(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])));
                    mx2 = fmaxf(mx2, fmaxf(__uint_as_float(x[i + 4]), __uint_as_float(x[i + 5])));
                    mx3 = fmaxf(mx3, fmaxf(__uint_as_float(x[i + 6]), __uint_as_float(x[i + 7])));
                }
                const float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3));
                const bool up = mx > m + grow;
                const float m_old = m;
                if (up) m = mx;
                const float alpha = up ? ex2((m_old - m) * qs) : 1.f;  // 0 for a row that had seen nothing
                l *= alpha;
                if (t > r.x && __any_sync(0xffffffffu, up)) {  // O is still: P V of the tile before precedes this S
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t o[32];
                        tmem_ld32(tO + 32 * c, o);
                        tmem_wait_ld32(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        tmem_st32(tO + 32 * c, o);
                    }
                }
                const float mm = m == -INFINITY ? 0.f : -m * qs;
                const float2 mm2 = make_float2(mm, mm), qs2 = make_float2(qs, qs);
                float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t h[16];
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        float2 u = ffma2(make_float2(__uint_as_float(x[32 * c + 2 * i]), __uint_as_float(x[32 * c + 2 * i + 1])), qs2, mm2);
                        float2 w =
                            ffma2(make_float2(__uint_as_float(x[32 * c + 2 * i + 2]), __uint_as_float(x[32 * c + 2 * i + 3])), qs2, mm2);
                        u = make_float2(ex2(u.x), ex2(u.y));
                        w = make_float2(ex2(w.x), ex2(w.y));
                        sum0 = fadd2(sum0, u);
                        sum1 = fadd2(sum1, w);
                        h[i] = h2_bits(__floats2half2_rn(u.x, u.y));
                        h[i + 1] = h2_bits(__floats2half2_rn(w.x, w.y));
                    }
                    tmem_st16(tS + 16 * c, h);
                }
                tmem_wait_st();
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[s]);
                l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
            }
        }
        if (ok) finish();
    }
    fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        fence_after_sync();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols) : "memory");
    }
}

// The parts of the units that the stretches cut: out = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k, in the order of k.
// Grid (CTAs of the main kernel, row blocks of 32); lane = row, warp = 16 columns.
__global__ void __launch_bounds__(256) chunk_join_kernel(const __grid_constant__ ChunkAttnParams p, int unit_rows) {
    grid_dep_wait();
    const Cut c = p.cuts[blockIdx.x];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.y * 32 + lane;
    if (!c.valid || (int)blockIdx.y * 32 >= c.rows || row >= c.rows) return;
    const int G = p.Hq / p.Hkv, first = blockIdx.x;
    auto slot = [&](int k) { return k < first ? 2 * k + 1 : 2 * k; };
    float M = -INFINITY;
    for (int k = first - 1; k <= c.last; ++k) M = fmaxf(M, p.part_ml[(size_t)slot(k) * unit_rows + row].x);
    float L = 0.f;
    float4 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = first - 1; k <= c.last; ++k) {
        const float2 ml = p.part_ml[(size_t)slot(k) * unit_rows + row];
        if (ml.x == -INFINITY) continue;  // this part saw nothing: its O was not written
        const float w = exp2f(ml.x - M);
        L = fmaf(w, ml.y, L);
        const float4 *src = p.part_o + (((size_t)slot(k) * (unit_rows / 32) + blockIdx.y) * 32 + 4 * warp) * 32 + lane;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = src[i * 32];
            o[i] = make_float4(fmaf(w, v.x, o[i].x), fmaf(w, v.y, o[i].y), fmaf(w, v.z, o[i].z), fmaf(w, v.w, o[i].w));
        }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const int r = c.r0 + row;
    uint16_t *out = p.out + ((size_t)(c.row0 + r / G) * p.Hq + c.g * G + r % G) * 128 + 16 * warp;
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[2 * i] = h2_bits(__floats2half2_rn(o[i].x * inv, o[i].y * inv));
        h[2 * i + 1] = h2_bits(__floats2half2_rn(o[i].z * inv, o[i].w * inv));
    }
    reinterpret_cast<uint4 *>(out)[0] = make_uint4(h[0], h[1], h[2], h[3]);
    reinterpret_cast<uint4 *>(out)[1] = make_uint4(h[4], h[5], h[6], h[7]);
}

// ------------------------------------------------------------------ host side

// [pages][Hkv][P][128] fp16 as boxes of one page, one kv head and 64 dims.
static int pool_map(CUtensorMap *m, const uint16_t *pool, int num_pages, int Hkv, int P) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return fail(I4_ECUDA, "i4_paged_gqa_chunk: cuTensorMapEncodeTiled is not available");
    const cuuint64_t dims[4] = {128, (cuuint64_t)P, (cuuint64_t)Hkv, (cuuint64_t)num_pages};
    const cuuint64_t strides[3] = {256, 256ull * P, 256ull * P * Hkv};
    const cuuint32_t box[4] = {64, (cuuint32_t)P, 1, 1}, step[4] = {1, 1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<uint16_t *>(pool), dims, strides, box, step,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(I4_ECUDA, "i4_paged_gqa_chunk: tensor map encode failed (%d)", (int)r);
    return I4_OK;
}

constexpr int kMaxDevices = 64;
struct DeviceState {
    std::once_flag once;
    cudaError_t err = cudaSuccess;
    int sms = 0;
};

// The current device's number of SMs, after its kernels' shared-memory limits have been raised (once per device).
static int device_sms(int *sms) {
    static DeviceState state[kMaxDevices];
    int dev = 0;
    int st = cuda_check(cudaGetDevice(&dev), "i4_paged_gqa_chunk: cudaGetDevice");
    if (st) return st;
    if (dev < 0 || dev >= kMaxDevices) return fail(I4_EUNSUPPORTED, "i4_paged_gqa_chunk: device %d", dev);
    DeviceState &d = state[dev];
    std::call_once(d.once, [&] {
        d.err = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
        if (d.err == cudaSuccess)
            d.err = cudaFuncSetAttribute(chunk_attn_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<1>::kSmem);
        if (d.err == cudaSuccess)
            d.err = cudaFuncSetAttribute(chunk_attn_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<2>::kSmem);
        d.sms = d.sms > kNumSMs ? kNumSMs : d.sms;
    });
    if (d.err != cudaSuccess) return cuda_check(d.err, "i4_paged_gqa_chunk smem attribute");
    *sms = d.sms;
    return I4_OK;
}

template <int NQ>
static int launch_chunk(const CUtensorMap &tk, const CUtensorMap &tv, const ChunkAttnParams &p, int sms, cudaStream_t stream) {
    const int grid = sms * Cfg<NQ>::kCtasPerSm;
    chunk_attn_kernel<NQ><<<grid, Cfg<NQ>::kThreads, Cfg<NQ>::kSmem, stream>>>(tk, tv, p);
    int st = launch_check("i4_paged_gqa_chunk");
    if (st) return st;
    return cuda_check(launch(chunk_join_kernel, dim3(grid, Cfg<NQ>::kUnitRows / 32), dim3(256), 0, stream, true, p,
                             (int)Cfg<NQ>::kUnitRows),
                      "i4_paged_gqa_chunk join");
}

int read_chunk_error(int reset) {
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_chunk_error, sizeof v);
    if (e != cudaSuccess) return cuda_check(e, "reading the chunk attention error flag");
    if (reset && v) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_chunk_error, &zero, sizeof zero);
        if (e != cudaSuccess) return cuda_check(e, "clearing the chunk attention error flag");
    }
    return v;
}

// Workspace: cuts | part_ml | part_o. Both variants have room for 2 * CTAs * unit rows = 4 * 148 * 128 rows.
constexpr size_t kWsRows = (size_t)2 * kMaxCtas * kRows;
constexpr size_t kWsMl = (kMaxCtas * sizeof(Cut) + 255) / 256 * 256;
constexpr size_t kWsO = kWsMl + kWsRows * sizeof(float2);
constexpr size_t kWsBytes = kWsO + kWsRows * 128 * sizeof(float);
static_assert(kWsO % 256 == 0, "parts are read 16 bytes at a time");
static_assert(Cfg<1>::kUnitRows * Cfg<1>::kCtasPerSm == Cfg<2>::kUnitRows * Cfg<2>::kCtasPerSm, "one workspace size");

}  // namespace i4

using namespace i4;

extern "C" size_t i4_paged_gqa_chunk_ws_bytes(void) { return kWsBytes; }

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
    if (!ws || ws_bytes < kWsBytes)
        return fail(I4_EINVAL, "i4_paged_gqa_chunk: workspace of %zu bytes needed (got %zu)", (size_t)kWsBytes, ws_bytes);
    if (!aligned(ws, 256)) return fail(I4_EALIGN, "i4_paged_gqa_chunk: workspace must be 256-byte aligned");
    int sms = 0;
    int st = device_sms(&sms);
    if (st) return st;
    CUtensorMap tk, tv;
    if ((st = pool_map(&tk, k_pool, num_pages, Hkv, page_size))) return st;
    if ((st = pool_map(&tv, v_pool, num_pages, Hkv, page_size))) return st;
    ChunkAttnParams p = {q,   k_pool, v_pool, q_stride,  page_table,        q_start,   ctx_len, out,  T,
                         B,   Hq,     Hkv,    page_size, max_pages_per_seq, num_pages, window,  scale};
    char *w = reinterpret_cast<char *>(ws);
    p.cuts = reinterpret_cast<Cut *>(w);
    p.part_ml = reinterpret_cast<float2 *>(w + kWsMl);
    p.part_o = reinterpret_cast<float4 *>(w + kWsO);
    // one slot of 128 rows when every chunk fits it: the other warpgroup would idle
    const int longest = max_q > 0 && max_q < T ? max_q : T;
    if (longest * (Hq / Hkv) <= kRows) return launch_chunk<1>(tk, tv, p, sms, (cudaStream_t)stream);
    return launch_chunk<2>(tk, tv, p, sms, (cudaStream_t)stream);
}
