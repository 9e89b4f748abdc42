// Attention of a ragged batch of new tokens over a paged cache, on tcgen05.
//
//   out[t][h] = sum_u softmax_u(scale q[t][h] . K[g][u]) V[g][u],  u in (p - window, p]
//
// for the token at position p, in one pass over u with the running maximum and
// sum of the softmax.
//
//  * Rows. The G = Hq / Hkv query heads that share a kv head are rows of one
//    matrix: row r of a slot is (token r / G, head r % G), so the 128 rows of an MMA are 128 / G (rounded down)
//    consecutive tokens, every K/V tile is read once for all of them, and a short chunk fills the rows better than one head's
//    tokens would. One TMA box of (64 dims, G heads, 128 / G tokens) brings half of a slot's Q in that order.
//  * Work. A unit is NQ slots' tokens of one sequence and one kv head; its cost is the
//    number of 128-position tiles that its rows see, and kUnitCost for beginning and ending it. The units stand in one line (kv
//    heads outermost) and every CTA, one per SM, takes an equal stretch of the line: a prompt's long and short units
//    balance, and a single token's long context spreads over the GPU. A unit that a border cuts leaves its parts
//    (m, l, O) in the workspace and a second kernel joins them in order; a unit of at most kWhole tiles is not cut, since
//    joining costs as much. The lengths are read on the device: every CTA finds its stretch by itself with two block-wide scans.
//  * Data. One warp loads K and V tiles (32 KB) page by page with TMA into a ring, 128-byte
//    swizzled (64 single tokens at 8000 positions, 28 heads on 4: 4.6-4.9 TB/s with pages of 64, 4.1-4.3 with pages of 16,
//    whose boxes of 2 KB are bound by the rate at which an SM's TMA takes them; the single-token kernel of attention.cu, which
//    gathers pages by cp.async, reads 6.0-6.3 at either); a page outside the pools, or one that no row sees, is an
//    out-of-range coordinate, which fills zeros.
//  * Math. S = Q K^T (M = 128 rows, both operands K-major in shared memory) into tensor memory; the 128 threads of a
//    warpgroup own one row each, so maximum and sum need no exchange; P = 2^(S - m + 7), rounded to fp16 (the tensor cores'
//    operand type), goes back over S's columns and is the A operand of O += P V (V MN-major). m only
//    follows the row's maximum when that is more than 2^8 ahead, so O is rarely rescaled (always following costs 20 %): P
//    then reaches at most 2^15, inside fp16. The rounding is 2^-11 of a weight down to 2^-21 of the row's largest, where P
//    becomes subnormal, and 2^-32 of the largest below that; without the 7, which costs nothing and cancels in O / l, a sink's
//    tail of 2^20 positions at 2^-25 of it would be lost to P V, though not to l. l and O are fp32. The exponent is one FMA,
//    s c - (m c - 7) with c = scale log2(e), whose second term is rounded: by 2^-15 at most while m c is below 1000, but by
//    more than any exponent for the largest scores. A row whose m passes that counts its scores from m on, in the branches that
//    mask and that move the maximum: one more for it costs 8 to 10 %.
//  * Overlap. A slot takes a tile in two halves of 64 positions: while its threads compute one half's exponentials, the tensor
//    cores run the other half's P V and the next tile's S over it. With NQ = 2 two slots share every tile; NQ = 1, for
//    chunks that fit one slot and for little work, has a deeper ring instead (two CTAs of one slot and two tiles of ring on an
//    SM: four single tokens 15.6 us against 14.7, one at 32768 positions 32 against 26, 16 chunks of 16 at 3000 positions 44
//    against 37; both slots of a CTA on every other tile of one slot's rows: 15.7, 27 and 41). Whole tiles of 128 with the slots
//    taking turns come out the same, 254 and 252 us on the case below: they load the tensor cores less but leave each slot
//    waiting for its own product.
//
// Bound by the tensor cores and their power: S of 64 positions is fed at the A operand's rate, so a tile of 2 x 128 rows
// costs 48 products of 64 cycles, 93 % of the 3300 cycles measured (32 products of twice the width would do the same work), and
// under a steady load the GPU's power limit holds the
// clock near 1.6 GHz. 512 tokens behind 32768 positions (28 heads on 4): 212-219 us in short runs, 1090-1130 TFLOP/s, 245-252 us
// under a steady load, 950-975 TFLOP/s (cuBLAS: 1421); a prompt of 8192: 437 and 498 us. Few rows are bound by the chain of dependent
// steps: four single tokens at up to 2049 positions take 14 us, 3.5 to the first tile (lengths, scans, first loads), 2 a
// tile, 1.2 to store a part and 3.5 to join them (attention.cu's kernel, whose parts meet inside a cluster, takes 8.8); a prompt
// of 512 takes 17 us where the page-table row ends at 1024 positions, else 19.5.
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
constexpr int kStep = kTile / 2;                   // positions that a slot's softmax takes at once
constexpr float kGrow = 8.f;                       // powers of two that a row's maximum may run ahead of its m
constexpr float kLift = 7.f;                       // powers of two that P, l and O are held above the weights: at most 2^15 for P
constexpr float kFar = 1000.f;                     // size of a row's m, in powers of two, from which scores count from there
constexpr float kLog2e = 1.4426950408889634f;

template <int NQ>
struct Cfg {
    static constexpr int kThreads = NQ == 2 ? 384 : 192;  // softmax warpgroups, an MMA warp each, the load warps
    static constexpr int kStages = NQ == 2 ? 5 : 6;
    static constexpr int kUnitRows = NQ * kRows;
    static constexpr int kUnitCost = 2;  // what beginning and ending a unit costs, in tiles
    static constexpr int kMinCost = 2;   // tiles that are worth a CTA of their own
    // rows of a warp of the joining kernel, out of eight loads in flight: the rows of short chunks come in many parts
    // (16 chunks of 16: 37.3 us with 2, 40.0 with 1), full tiles in two or three (a mixed batch: 49.5 us with 4, 52 with 2)
    static constexpr int kJoinRows = NQ == 2 ? 4 : 2;
    static constexpr int kWhole = 4;     // a unit of at most so many tiles is not cut: joining would take longer
    static constexpr unsigned kTmemCols = NQ * 256;  // S / P and O of every slot
    static constexpr unsigned kSmem = 1024 + (NQ + kStages) * kTileBytes;
};

__device__ int g_chunk_error = 0;

// Where a unit is cut at the beginning of a CTA's stretch: what the joining kernel needs.
struct Cut {
    // parts: CTA c - 1's last, then the first of c .. last; the unit's tokens begin at this row of q
    int valid, last, tokens, row, g;
};

struct ChunkAttnParams {
    const uint16_t *q, *k_pool, *v_pool;
    long long q_stride;
    const int32_t *page_table, *q_start, *ctx_len;
    uint16_t *out;
    int T, B, Hq, Hkv, page_size, max_pages, num_pages, window;
    float scale;
    int slot_tokens;      // 128 / G
    unsigned unit_inv;    // ceil(2^32 / (NQ * slot_tokens))
    Cut *cuts;        // [CTAs]
    float2 *part_ml;  // [2 * CTAs][unit rows]: (m, l), m a score before the scale
    float *part_o;    // [2 * CTAs][unit rows][128]
};

// ------------------------------------------------------------------ the line of units

// The first position that the token at pos sees.
__device__ __forceinline__ int first_seen(const ChunkAttnParams &p, int pos) {
    return p.window > 0 ? max(0, max(pos, 0) - (p.window - 1)) : 0;  // no overflow at positions below 0 and windows up to 2^31 - 1
}

// Positions that the tokens [a, e) of a sequence whose first new token stands at pos0 may see: [x, y), empty when y <= x.
__device__ __forceinline__ int2 seen(const ChunkAttnParams &p, int pos0, int a, int e) {
    const int hi = min(pos0 + e, p.max_pages * p.page_size);
    return make_int2(first_seen(p, pos0 + a), hi);
}
__device__ __forceinline__ int2 tiles_of(int2 s) {
    return s.y > s.x ? make_int2(s.x / kTile, (s.y + kTile - 1) / kTile) : make_int2(0, 0);
}

// Units of n tokens: ceil(n / unit). n < 2^21 and a unit has at most 256 tokens, so the product is exact.
template <int NQ>
__device__ __forceinline__ int units_of(const ChunkAttnParams &p, int n) {
    return (int)__umulhi((unsigned)(n + NQ * p.slot_tokens - 1), p.unit_inv);
}

// a * b / c; in 32 bits, which takes a tenth of the time, wherever the line is shorter than 2^23 tiles (b <= 2^9).
__device__ __forceinline__ long long share(long long a, int b, long long c) {
    return a < (1 << 23) ? (long long)((unsigned)a * (unsigned)b / (unsigned)c) : a * b / c;
}

// A CTA's stretch of the line.
struct Stretch {
    int g, b, i, off;  // first unit, and what of its cost belongs to earlier CTAs
    int left;          // cost of the stretch
    int n, pos0, row0; // the first unit's sequence
};

// One unit's part in a stretch.
struct Piece {
    int g, b, pos0, row0;     // kv head; sequence: first position, first row of q
    int tok0, tokens;         // the unit's tokens of the sequence
    int2 see;                 // positions that the unit sees
    int t0, t1;               // the part's tiles
    int whole, slot;          // uncut, or the slot of its parts
};

// Walks the pieces of a stretch; every role of the CTA does so by itself.
template <int NQ>
struct Walker {
    const ChunkAttnParams &p;
    const int unit;  // tokens of a unit
    int g, b, i, off, left, n, pos0, row0, units;
    __device__ Walker(const ChunkAttnParams &p_, const Stretch &s)
        : p(p_), unit(NQ * p_.slot_tokens), g(s.g), b(s.b), i(s.i), off(s.off), left(s.left), n(s.n), pos0(s.pos0),
          row0(s.row0) {
        units = units_of<NQ>(p, n);
    }
    __device__ void load() {
        const int2 r = chunk_rows(p.q_start, b, p.T);
        row0 = r.x;
        n = r.y;
        pos0 = max(p.ctx_len[b], 0) - n;
        units = units_of<NQ>(p, n);
    }
    __device__ bool next(Piece &pc) {
        constexpr int V = Cfg<NQ>::kUnitCost;  // a unit's cost lies on the line as V, then its tiles
        while (left > 0) {
            pc.g = g;
            pc.b = b;
            pc.pos0 = pos0;
            pc.row0 = row0;
            pc.tok0 = i * unit;
            pc.tokens = min(n - pc.tok0, unit);
            pc.see = seen(p, pos0, pc.tok0, pc.tok0 + pc.tokens);
            const int2 t = tiles_of(pc.see);
            const int tiles = t.y - t.x, take = min(tiles + V - off, left);
            const int x = max(off - V, 0), y = max(off + take - V, 0);
            const bool any = tiles > 0 ? y > x : off == 0;  // rows that see nothing are written by one CTA too
            pc.t0 = t.x + x;
            pc.t1 = t.x + y;
            pc.whole = y - x == tiles;
            pc.slot = 2 * blockIdx.x + (x == 0);
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
            if (any) return true;
        }
        return false;
    }
};

// Tiles of a piece that the tokens of slot s see: [x, y), and how many tokens it has.
__device__ __forceinline__ int3 slot_tiles(const ChunkAttnParams &p, const Piece &pc, int s) {
    const int a = pc.tok0 + s * p.slot_tokens, n = min(max(pc.tokens - s * p.slot_tokens, 0), p.slot_tokens);
    if (n == 0) return make_int3(0, 0, 0);
    const int2 t = tiles_of(seen(p, pc.pos0, a, a + n));
    const int x = max(t.x, pc.t0), y = min(t.y, pc.t1);
    return y > x ? make_int3(x, y, n) : make_int3(0, 0, n);
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

// This CTA's stretch, and the cut at its beginning. scratch: 32 + 3 NT ints of shared memory.
template <int NQ>
__device__ __forceinline__ void find_stretch(const ChunkAttnParams &p, Stretch *out, int *scratch) {
    using C = Cfg<NQ>;
    constexpr int NT = C::kThreads, V = C::kUnitCost;
    const int tid = threadIdx.x, size = NQ * p.slot_tokens;
    // first: units before sequence b0 + j; tokens, pos: its new tokens and the first one's position
    int *sums = scratch, *first = scratch + 32, *tokens = first + NT, *pos = tokens + NT;
    if (tid == 0) {
        *out = {0, 0, 0, 0, 0, 0, 0, 0};
        p.cuts[blockIdx.x].valid = 0;
    }
    long long W = 0, start = 0, end = 0;
    int n_ctas = 1, line = 0, head = 0, target = 0, head_end = 0, target_end = 0;  // kv heads and places of the borders
    int cost = 0, at = 0, j = 0, i = 0;  // this thread's unit: unit i of sequence b0 + j
    // The CTA whose stretch has the tile before x: the largest c with c W / n <= x - 1.
    auto last_cta = [&](long long x) {
        return W < (1 << 23) ? (int)(((unsigned)x * (unsigned)n_ctas - 1u) / (unsigned)W) : (int)((x * n_ctas - 1) / W);
    };
    // The unit that a border of the stretch lies in, for the thread that has it: a short unit goes whole to the CTA behind.
    auto offset = [&](int place_in_line) {
        const int off = place_in_line - at;
        return off < 0 || off >= cost ? -1 : (cost <= V + C::kWhole ? 0 : off);
    };
    auto place = [&](int b0) {
        const int off = offset(target);
        if (off >= 0) {
            const int2 seq = chunk_rows(p.q_start, b0 + j, p.T);
            const long long unit = start - (target - at);  // where the unit begins
            out->g = head;
            out->b = b0 + j;
            out->i = i;
            out->off = off;
            out->n = seq.y;
            out->pos0 = pos[j];
            out->row0 = seq.x;
            atomicSub(&out->left, (int)(unit + off - start));
            if (off > V && share(W, blockIdx.x - 1, n_ctas) <= unit + V)
                // the first cut of this unit: its parts end in the CTA that holds its last tile
                p.cuts[blockIdx.x] = {1, last_cta(unit + cost), min(seq.y - i * size, size), seq.x + i * size, head};
        }
        const int off_end = end < W ? offset(target_end) : -1;
        if (off_end >= 0) atomicAdd(&out->left, off_end - (target_end - at));
    };
    for (int pass = 0; pass < 2; ++pass) {  // the first measures the line, the second finds the place in it
        int run = 0, trips = 0, all_units = 0;
        for (int b0 = 0; b0 < p.B; b0 += NT) {
            int n = 0, first_pos = 0, total_units;
            if (b0 + tid < p.B) {
                n = chunk_rows(p.q_start, b0 + tid, p.T).y;
                first_pos = max(p.ctx_len[b0 + tid], 0) - n;
            }
            const int before = scan_block<NT>(units_of<NQ>(p, n), total_units, sums);
            all_units += total_units;
            // a q_start that decreases has sequences share rows: not as many as would make the line longer than its ints hold
            if (all_units > units_of<NQ>(p, p.T) + p.B) {
                run = 0;
                break;
            }
            first[tid] = before;
            tokens[tid] = n;
            pos[tid] = first_pos;
            __syncthreads();
            for (int u0 = 0; u0 < total_units; u0 += NT, ++trips) {
                const int u = u0 + tid;
                cost = j = 0;
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
                    const int2 t = tiles_of(seen(p, pos[j], i * size, min(tokens[j], i * size + size)));
                    cost = t.y - t.x + V;
                }
                int sum;
                at = run + scan_block<NT>(cost, sum, sums);
                if (pass == 1) place(b0);
                run += sum;
            }
            __syncthreads();  // the scratch is read no more
        }
        if (pass == 0) {
            line = run;
            W = (long long)line * p.Hkv;
            n_ctas = (int)min((long long)gridDim.x, max((W + C::kMinCost - 1) / C::kMinCost, 1ll));
            start = share(W, blockIdx.x, n_ctas);
            end = share(W, blockIdx.x + 1, n_ctas);
            if ((int)blockIdx.x >= n_ctas || start >= end) break;
            head = (int)share(start, 1, line);
            target = (int)(start - (long long)head * line);
            head_end = (int)share(end, 1, line);
            target_end = (int)(end - (long long)head_end * line);
            if (tid == 0) out->left = (int)(end - start);
            __syncthreads();
            if (trips == 1 && p.B <= NT) {  // every unit is still in its thread's hands
                place(0);
                break;
            }
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

__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// A value that is the same in every lane of the warp, in a form that the compiler knows to be.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ uint64_t uniform(uint64_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// A wait that ends: on the barrier, when another role of the CTA gave up, or after ~8 s: a warp that sums its 32 rows of 2^20
// positions again (plain_row) holds the other roles up for 3.4e9 cycles, 4.6e9 where both slots do.
constexpr long long kWait = 4 * kWaitCycles;
__device__ __forceinline__ bool wait_or_stop(uint64_t *bar, unsigned parity, volatile int *stop) {
    if (mbar_test(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_test(bar, parity)) {
        if (*stop) return false;
        if (clock64() - t0 > kWait) {
            *stop = 1;
            record_error(&g_chunk_error, 1);
            return false;
        }
    }
    return true;
}

// v[i] of lane 4a + k becomes v[k] of lane 4a + i.
__device__ __forceinline__ void transpose4(uint4 (&v)[4]) {
    const int lane = threadIdx.x & 3;
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
        const bool up = lane & d;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & d) continue;
            uint4 give = up ? v[i] : v[i + d];
            give.x = __shfl_xor_sync(0xffffffffu, give.x, d);
            give.y = __shfl_xor_sync(0xffffffffu, give.y, d);
            give.z = __shfl_xor_sync(0xffffffffu, give.z, d);
            give.w = __shfl_xor_sync(0xffffffffu, give.w, d);
            if (up)
                v[i] = give;
            else
                v[i + d] = give;
        }
    }
}

// The softmax sums of one row over the positions [lo, hi) by plain loads, for rows whose tensor-core sum met a NaN or an
// infinity: P = 0 times such a value of a position that other rows see is NaN, and must not count. Returns O, and (m, l) in
// `ml`: its scores are sums in another order than the tensor cores', so it has a maximum of its own. Four lanes have the
// score of a position, eight positions at a time and 32 a trip; then a lane has four dims of the sum over the 32. Bound by the
// latency of the loads of a warp that has little beside it: some 100 cycles a position with 16 loads of K and 8 of V in flight
// (137 with two slots a CTA), 285 with one.
struct PlainRow {
    float4 o;
    float2 ml;
};
__device__ __noinline__ PlainRow plain_row(const ChunkAttnParams &p, int b, int g, const uint16_t *q, int lo, int hi, float qs) {
    const int lane = threadIdx.x & 31;
    uint4 x[4];  // 16-byte chunks lane % 4, + 4, + 8, + 12 of q
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const uint4 *>(q + 8 * (4 * i + (lane & 3)));
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = -INFINITY, l = 0.f;
    for (int u0 = lo; u0 < hi; u0 += 32) {
        const int u = u0 + lane;
        const int page = u < hi ? p.page_table[(size_t)b * p.max_pages + u / p.page_size] : -1;
        const bool there = page >= 0 && page < p.num_pages;  // else K and V are zeros; the first page's are read and dropped
        const size_t off = there ? (((size_t)page * p.Hkv + g) * p.page_size + u % p.page_size) * 128 : 0;
        float s = 0.f;
        uint4 a[4][4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint16_t *k = p.k_pool + __shfl_sync(0xffffffffu, (unsigned long long)off, 8 * c + (lane >> 2)) + 8 * (lane & 3);
#pragma unroll
            for (int i = 0; i < 4; ++i) a[c][i] = *reinterpret_cast<const uint4 *>(k + 32 * i);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                t = fma2_f16_f32(a[c][i].x, x[i].x, t);
                t = fma2_f16_f32(a[c][i].y, x[i].y, t);
                t = fma2_f16_f32(a[c][i].z, x[i].z, t);
                t = fma2_f16_f32(a[c][i].w, x[i].w, t);
            }
            t += __shfl_xor_sync(0xffffffffu, t, 1);
            t += __shfl_xor_sync(0xffffffffu, t, 2);
            t = __shfl_sync(0xffffffffu, t, 4 * (lane & 7));
            if (lane >> 3 == c) s = t;
        }
        s = u >= hi ? -INFINITY : (there ? s : 0.f);
        float mx = s;
#pragma unroll
        for (int e = 16; e > 0; e >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, e));
        if (mx > m) {
            const float alpha = ex2((m - mx) * qs);
            m = mx;
            l *= alpha;
            o = make_float4(o.x * alpha, o.y * alpha, o.z * alpha, o.w * alpha);
        }
        const float w = m == -INFINITY ? 0.f : ex2(fmaf(s - m, qs, kLift));
        l += w;
        const unsigned rows = __ballot_sync(0xffffffffu, there);
        float4 d = make_float4(0.f, 0.f, 0.f, 0.f);  // this trip's sum: a row of 2^20 positions adds 2^15 of them
#pragma unroll
        for (int k0 = 0; k0 < 32; k0 += 8) {
            uint2 v[8];  // in flight together: a warp alone with its loads waits 280 cycles for each
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = *reinterpret_cast<const uint2 *>(p.v_pool + __shfl_sync(0xffffffffu, (unsigned long long)off, k0 + k) + 4 * lane);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float wk = __shfl_sync(0xffffffffu, w, k0 + k);
                if (!((rows >> (k0 + k)) & 1)) v[k] = make_uint2(0u, 0u);
                const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&v[k].x));
                const float2 c = __half22float2(*reinterpret_cast<const __half2 *>(&v[k].y));
                d = make_float4(fmaf(wk, a.x, d.x), fmaf(wk, a.y, d.y), fmaf(wk, c.x, d.z), fmaf(wk, c.y, d.w));
            }
        }
        o = make_float4(o.x + d.x, o.y + d.y, o.z + d.z, o.w + d.w);
    }
    return {o, make_float2(m, warp_sum(l))};
}

template <int NQ>
__global__ void __launch_bounds__(Cfg<NQ>::kThreads, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ ChunkAttnParams p) {
    using C = Cfg<NQ>;
    constexpr int S = C::kStages, kMmaWarp = NQ * 4, kLoadWarp = kMmaWarp + NQ;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t kv_full[S], kv_empty[S], q_full[NQ], q_free[NQ], s_full[NQ][2], p_full[NQ][2];
    __shared__ __align__(8) uint64_t pv_done[NQ][2], o_free[NQ], all_done;
    __shared__ uint32_t tmem_base;
    __shared__ Stretch stretch;
    __shared__ int stop_flag;
    volatile int *stop = &stop_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = p.Hq / p.Hkv;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char *gbase = smem_raw + (base - smem_u32(smem_raw));
    const uint32_t ring = base + NQ * kTileBytes;

    if (tid == 0) {
        stop_flag = 0;
        for (int i = 0; i < S; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], NQ);
        }
        for (int s = 0; s < NQ; ++s) {
            mbar_init(&q_full[s], 1);
            mbar_init(&q_free[s], 1);
            for (int h = 0; h < 2; ++h) {
                mbar_init(&s_full[s][h], 1);
                mbar_init(&p_full[s][h], 4);
                mbar_init(&pv_done[s][h], 1);
            }
            mbar_init(&o_free[s], 4);
        }
        mbar_init(&all_done, NQ);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)),
                     "r"(C::kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == kLoadWarp && lane < 3)
        asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0 ? &tm_q : (lane == 1 ? &tm_k : &tm_v)) : "memory");
    grid_dep_wait();  // what the kernel before left: lengths, tables, q, the pages; and its use of the workspace has ended
    find_stretch<NQ>(p, &stretch, reinterpret_cast<int *>(gbase));
    fence_async_smem();  // its scratch lies where the first copy of Q will
    grid_dep_launch();  // the joining kernel may come up; it waits for this grid's end before it reads anything
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = uniform(tmem_base);  // S / P of slot s at column 128 s, O of slot s at 128 (NQ + s)

    Walker<NQ> walk(p, stretch);
    Piece pc;
    if (stretch.left <= 0) {
        // no work: straight to the end
    } else if (warp >= kMmaWarp) {
        // The rows of Q of one slot's piece: tokens behind the sequence's are another's, or zeros behind the last row; nothing
        // that comes of them is stored.
        auto load_q = [&](const Piece &c, int s) {
            if (lane == 0) {
                mbar_expect_tx(&q_full[s], (unsigned)(p.slot_tokens * G) * 256u);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    tma_load_4d(base + s * kTileBytes + h * kHalf, &tm_q, 64 * h, c.g * G, c.row0 + c.tok0 + s * p.slot_tokens, 0,
                                &q_full[s]);
            }
        };
        if (warp > kLoadWarp) {
            // ---------------- rows of Q (NQ = 2; with NQ = 1 the load warp's own)
            unsigned uses[NQ] = {};
            bool ok = true;
            while (ok && walk.next(pc)) {
#pragma unroll
                for (int s = 0; s < NQ; ++s) {
                    const int3 r = slot_tiles(p, pc, s);
                    if (r.y <= r.x) continue;
                    if (ok && uses[s] > 0) ok = wait_or_stop(&q_free[s], (uses[s] - 1) & 1, stop);
                    ok = __all_sync(0xffffffffu, ok);
                    if (ok) load_q(pc, s);
                    uses[s] += ok;
                }
            }
            if (!ok && lane == 0)  // let the copies in flight land
                for (int s = 0; s < NQ; ++s)
                    if (uses[s] > 0) mbar_wait(&q_full[s], (uses[s] - 1) & 1);
            __syncwarp();
        } else if (warp == kLoadWarp) {
            // ---------------- K and V tiles: K0 V0 K1 V1 ...
            const int np = kTile / p.page_size;  // pages of a tile
            const int half = lane / np, pg = lane % np;
            const bool loads = lane < 2 * np;
            unsigned it = 0, uses = 0;
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
                            tma_load_4d(ring + st * kTileBytes + half * kHalf + pg * p.page_size * 128, kv ? &tm_v : &tm_k,
                                        half * 64, 0, pc.g, page, &kv_full[st]);
                        if (NQ == 1 && t == pc.t0 && kv == 0) {  // behind the piece's first K tile
                            if (uses > 0) ok = wait_or_stop(&q_free[0], (uses - 1) & 1, stop);
                            ok = __all_sync(0xffffffffu, ok);
                            if (!ok) {
                                ++it;
                                break;
                            }
                            load_q(pc, 0);
                            ++uses;
                        }
                    }
                }
            }
            if (!ok && lane == 0) {  // let the copies in flight land before the CTA's memory goes
                for (unsigned k = it > S ? it - S : 0; k < it; ++k) mbar_wait(&kv_full[k % S], (k / S) & 1);
                if (NQ == 1 && uses > 0) mbar_wait(&q_full[0], (uses - 1) & 1);
            }
            __syncwarp();
        } else if (warp < kMmaWarp + NQ) {
            // ---------------- S = Q K^T and O += P V of slot s. One warp per slot: both slots' products issued by one warp took
            // longer than the tensor cores' own work
            constexpr uint32_t idesc_qk = idesc_f16(kRows, kStep), idesc_pv = idesc_f16(kRows, 128) | kIdescBMajorMN;
            const int s = (int)uniform((uint32_t)(warp - kMmaWarp));
            const uint32_t tS = tmem + 128 * s, tO = tmem + 128 * (NQ + s);
            const uint64_t qd = desc_sw128(base + s * kTileBytes), kd0 = desc_sw128(ring), vd0 = desc_sw128_mn(ring, kHalf);
            unsigned it = 0, uses = 0, steps = 0;  // ring entries, pieces and tiles so far
            bool ok = true;
            while (ok && walk.next(pc)) {
                const int3 r = slot_tiles(p, pc, s);
                if (pc.t1 <= pc.t0) continue;
#pragma unroll 1
                for (int j = pc.t0 - 1; j < pc.t1; ++j, it += 2) {
                    // entries it - 1: V of tile j, it: K of tile j + 1
                    const unsigned sv = (it - 1) % S, sk = it % S;
                    const bool has_v = j >= pc.t0, has_k = j + 1 < pc.t1;
                    const bool pv = j >= r.x && j < r.y, qk = j + 1 >= r.x && j + 1 < r.y;
                    if (has_v) {
                        ok = wait_or_stop(&kv_full[sv], ((it - 1) / S) & 1, stop);
                        const int t = j * kTile;
                        if (ok && (t < pc.see.x || t + kTile > pc.see.y)) {
                            // rows of V that the unit does not see may hold anything, NaN included: zero them (both slots' warps
                            // write the same zeros)
                            for (int e = lane; e < 2 * kTile * 8; e += 32) {
                                const int u = (e >> 3) & (kTile - 1);
                                if (t + u < pc.see.x || t + u >= pc.see.y)
                                    *reinterpret_cast<uint4 *>(gbase + (NQ + sv) * kTileBytes + e * 16) = make_uint4(0, 0, 0, 0);
                            }
                            fence_async_smem();
                        }
                        __syncwarp();
                    }
                    if (ok && has_k) ok = wait_or_stop(&kv_full[sk], (it / S) & 1, stop);
                    if (ok && qk && j + 1 == r.x) ok = wait_or_stop(&q_full[s], uses & 1, stop);
                    if (ok && pv && j == r.x) {
                        if (uses > 0) ok = wait_or_stop(&o_free[s], (uses - 1) & 1, stop);
                        ++uses;
                    }
                    const uint64_t vd = vd0 + uniform(sv) * (kTileBytes >> 4), kd = kd0 + uniform(sk) * (kTileBytes >> 4);
                    const int more = j > r.x;
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {  // the halves of the tile: P V of one, then the next tile's S over it
                        if (ok && pv) ok = wait_or_stop(&p_full[s][h], steps & 1, stop);
                        if (!__all_sync(0xffffffffu, ok)) break;
                        fence_after_sync();
                        if (elect_one()) {
                            if (pv) {
#pragma unroll
                                for (int kk = 0; kk < kStep / 16; ++kk)
                                    umma_f16_ta(tO, tS + kStep * h + 8 * kk, vd + (h * (kStep / 16) + kk) * (2048 >> 4), idesc_pv,
                                                kk > 0 ? 1 : (more | h));
                                umma_commit(&pv_done[s][h]);
                            }
                            if (qk) {
#pragma unroll
                                for (int kk = 0; kk < 8; ++kk) {
                                    const uint32_t o = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                                    umma_f16(tS + kStep * h, qd + o, kd + o + h * (kStep * 128 >> 4), idesc_qk, kk > 0 ? 1 : 0);
                                }
                                umma_commit(&s_full[s][h]);
                            }
                            if (h == 1) {
                                if (has_v) umma_commit(&kv_empty[sv]);
                                if (has_k) umma_commit(&kv_empty[sk]);
                                if (qk && j + 2 == r.y) umma_commit(&q_free[s]);
                            }
                        }
                        __syncwarp();
                    }
                    steps += pv;
                    if (!__all_sync(0xffffffffu, ok)) break;
                }
                ok = __all_sync(0xffffffffu, ok);
                it -= 2;
            }
            // nothing of this slot is in flight on the tensor cores when the CTA leaves
            if (elect_one()) umma_commit(&all_done);
            if (!mbar_wait(&all_done, 0)) record_error(&g_chunk_error, 1);
            __syncwarp();
        }
    } else {
        // ---------------- softmax of slot s: thread = row
        const int s = warp >> 2, wq = warp & 3, row = tid & 127;
        const uint32_t lanes = (uint32_t)(32 * wq) << 16;
        const uint32_t tS = tmem + 128 * s + lanes, tO = tmem + 128 * (NQ + s) + lanes;
        const int my_tok = row / G, my_head = row - my_tok * G;  // within the slot and the kv head
        const float qs = p.scale * kLog2e, grow = fminf(kGrow / qs, 1e30f);
        unsigned tiles = 0;  // so far; each was two halves of P
        bool ok = true;

        float m = -INFINITY, l = 0.f;
        float ref = 0.f;  // m and the scores count from here: 0, or a score of this row once those are far from 0
        auto limits = [&](const Piece &c, int &lo, int &hi) {  // positions that this thread's row sees
            const int pos = c.pos0 + c.tok0 + s * p.slot_tokens + my_tok;
            hi = min(pos + 1, p.max_pages * p.page_size);
            lo = first_seen(p, pos);
        };
        auto finish = [&](const Piece &last, const int3 &last_r) {
            if (last_r.z == 0) return;  // the slot has no rows
            const bool mine = my_tok < last_r.z, any = last_r.y > last_r.x;
            const int tok = last.tok0 + s * p.slot_tokens + my_tok, head = last.g * G + my_head;
            const float l_inv = l == 0.f ? 0.f : 1.f / l;
            const int slot_row = last.slot * C::kUnitRows + s * kRows + row;
            float *part = p.part_o + (size_t)(slot_row & ~3) * 128 + 4 * (lane & 3);  // the first row of this group of four lanes
            const int my_rows = min(max(last_r.z * G - (row & ~3), 0), 4);
            if (!last.whole && mine)  // an all-NaN row has l = NaN and no maximum: keep it from reading as empty
                p.part_ml[slot_row] = make_float2(l != l ? 0.f : m + ref, l);
            if (any) {
                ok = wait_or_stop(&pv_done[s][0], (tiles - 1) & 1, stop) && wait_or_stop(&pv_done[s][1], (tiles - 1) & 1, stop);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
                fence_after_sync();
            }
            const bool few = last_r.z * G <= 32;
            const long long own = mine ? ((long long)(last.row0 + tok) * p.Hq + head) * 128 : -1;
            long long to[4];  // output rows of this group of four lanes, or -1
#pragma unroll
            for (int k = 0; k < 4; ++k) to[k] = __shfl_sync(0xffffffffu, own, (lane & ~3) + k);
            float bad[4] = {0.f, 0.f, 0.f, 0.f};  // stay 0 while every value of O is finite
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                if (few && wq > 0) break;  // no rows in this warp
                uint32_t o[32];
                if (any) {
                    tmem_ld32(tO + 32 * c, o);
                    tmem_wait_ld32(o);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0u;
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) bad[i & 3] = fmaf(__uint_as_float(o[i]), 0.f, bad[i & 3]);
                // Lanes that store their own rows touch 32 lines with every store; turned four by four, 8. Rows of one warp
                // alone are stored as they are: turning costs that warp more (2.3 us against 1.2).
                if (last.whole) {
                    uint4 v[4];  // 16-byte chunks 4c .. 4c + 3 of this lane's row
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t h[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            h[k] = h2_bits(__floats2half2_rn(__uint_as_float(o[8 * i + 2 * k]) * l_inv,
                                                             __uint_as_float(o[8 * i + 2 * k + 1]) * l_inv));
                        v[i] = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                    if (few) {
                        if (mine) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4 *>(p.out + own + 32 * c + 8 * k) = v[k];
                        }
                    } else {
                        transpose4(v);  // now chunk 4c + (lane & 3) of the rows of this group of four lanes
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (to[k] >= 0) *reinterpret_cast<uint4 *>(p.out + to[k] + 32 * c + 8 * (lane & 3)) = v[k];
                    }
                } else if (any && few) {
                    if (mine) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<uint4 *>(p.part_o + (size_t)slot_row * 128 + 32 * c + 4 * i) =
                                make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                } else if (any) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint4 v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            v[k] = make_uint4(o[16 * i + 4 * k], o[16 * i + 4 * k + 1], o[16 * i + 4 * k + 2],
                                              o[16 * i + 4 * k + 3]);
                        transpose4(v);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (k < my_rows) *reinterpret_cast<uint4 *>(part + k * 128 + 32 * c + 16 * i) = v[k];
                    }
                }
            }
            if (any) {
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&o_free[s]);
            }
            // rows that met a NaN or an infinity, and whose own scores are fine, are summed again over what they see
            const bool fine = bad[0] + bad[1] + (bad[2] + bad[3]) == 0.f;
            unsigned again = __ballot_sync(0xffffffffu, mine && any && !fine && fabsf(l) < INFINITY);
            while (again) {
                const int k = __ffs(again) - 1;
                again &= again - 1;
                int lo, hi;
                limits(last, lo, hi);
                lo = max(__shfl_sync(0xffffffffu, lo, k), last_r.x * kTile);
                hi = min(__shfl_sync(0xffffffffu, hi, k), last_r.y * kTile);
                const int tk = __shfl_sync(0xffffffffu, tok, k), hk = __shfl_sync(0xffffffffu, head, k);
                const PlainRow pr =
                    plain_row(p, last.b, last.g, p.q + (size_t)(last.row0 + tk) * p.q_stride + (size_t)hk * 128, lo, hi, qs);
                const float4 v = pr.o;
                const float2 ml = pr.ml;
                if (last.whole) {
                    const float inv = ml.y == 0.f ? 0.f : 1.f / ml.y;
                    uint16_t *d = p.out + ((size_t)(last.row0 + tk) * p.Hq + hk) * 128 + 4 * lane;
                    d[0] = float_to_half_bits(v.x * inv);
                    d[1] = float_to_half_bits(v.y * inv);
                    d[2] = float_to_half_bits(v.z * inv);
                    d[3] = float_to_half_bits(v.w * inv);
                } else {
                    const int at = last.slot * C::kUnitRows + s * kRows + 32 * wq + k;
                    reinterpret_cast<float4 *>(p.part_o)[(size_t)at * 32 + lane] = v;
                    if (lane == k) p.part_ml[at] = ml;  // the lane that wrote it before
                }
            }
        };

        while (ok && walk.next(pc)) {
            const int3 r = slot_tiles(p, pc, s);
            m = -INFINITY;
            l = 0.f;
            ref = 0.f;
            int lo, hi;
            limits(pc, lo, hi);
            if (my_tok >= r.z) {  // no row: anything goes, nothing is stored
                lo = 0;
                hi = 0x7fffffff;
            }
#pragma unroll 1
            for (int u = 2 * r.x; u < 2 * r.y; ++u) {  // halves of tiles
                const int h = u & 1;
                ok = __all_sync(0xffffffffu, wait_or_stop(&s_full[s][h], tiles & 1, stop));
                if (!ok) break;
                fence_after_sync();
                uint32_t x[kStep];
                tmem_ld32(tS + kStep * h, x);
                tmem_ld32(tS + kStep * h + 32, x + 32);
                tmem_wait_ld32(x);
                tmem_wait_ld32(x + 32);
                const int a = lo - u * kStep, e = hi - u * kStep;  // the row sees [a, e) of these positions
                if (__any_sync(0xffffffffu, a > 0 || e < kStep || ref != 0.f)) {
#pragma unroll
                    for (int i = 0; i < kStep; ++i)
                        x[i] = i < a || i >= e ? 0xff800000u /* -inf */ : __float_as_uint(__uint_as_float(x[i]) - ref);
                }
                float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
                for (int i = 0; i < kStep; i += 8) {
                    mx0 = max3(mx0, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
                    mx1 = max3(mx1, __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]));
                    mx2 = max3(mx2, __uint_as_float(x[i + 4]), __uint_as_float(x[i + 5]));
                    mx3 = max3(mx3, __uint_as_float(x[i + 6]), __uint_as_float(x[i + 7]));
                }
                const float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3));
                const bool up = mx - m > grow;  // m + grow would be rounded by more than grow where m is large
                if (__any_sync(0xffffffffu, up)) {
                    const bool far = up && fabsf(mx * qs) >= kFar;
                    if (__any_sync(0xffffffffu, far)) {
                        // count from the maximum (what rounding leaves of it is a step of it at most, and nothing the next time)
                        // and take the half again
                        if (far) {
                            const float to = ref + mx;
                            m += ref - to;
                            ref = to;
                        }
                        --u;
                        continue;
                    }
                    const float alpha = up ? ex2((m - mx) * qs) : 1.f;  // 0 for a row that had seen nothing
                    if (up) m = mx;
                    l *= alpha;
                    if (u > 2 * r.x) {  // O holds still once P V of the half before has ended
                        ok = __all_sync(0xffffffffu, wait_or_stop(&pv_done[s][h ^ 1], (tiles - (h ^ 1)) & 1, stop));
                        if (!ok) break;
                        fence_after_sync();
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
                }
                const float mm = m == -INFINITY ? 0.f : fmaf(-m, qs, kLift);
                const float2 mm2 = make_float2(mm, mm), qs2 = make_float2(qs, qs);
                float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 sc = make_float2(__uint_as_float(x[32 * c + 2 * i]), __uint_as_float(x[32 * c + 2 * i + 1]));
                        float2 v = ffma2(sc, qs2, mm2);
                        v = make_float2(ex2(v.x), ex2(v.y));
                        if (i & 1)
                            sum1 = fadd2(sum1, v);
                        else
                            sum0 = fadd2(sum0, v);
                        w[i] = h2_bits(__floats2half2_rn(v.x, v.y));
                    }
                    tmem_st16(tS + kStep * h + 16 * c, w);
                }
                tmem_wait_st();
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[s][h]);
                l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
                tiles += h;
            }
            if (ok) finish(pc, r);
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        fence_after_sync();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols) : "memory");
    }
}

// The parts of the units that the stretches cut: out = sum_k w_k O_k / sum_k w_k l_k, w_k = 2^((m_k - M) scale log2(e)), in the
// order of k.
// A warp has R rows at once, lane = four columns. The weights of 32 parts are in the lanes at once and eight loads are in
// flight.
template <int R>
__device__ __forceinline__ void join_rows(const ChunkAttnParams &p, const Cut &c, int G, int unit_rows) {
    const int lane = threadIdx.x & 31, first = blockIdx.x;
    const float qs = p.scale * kLog2e;
    const int parts = c.last - first + 2;
    const auto slot = [&](int k) { return k == 0 ? 2 * first - 1 : 2 * (first + k - 1); };  // the k-th part's
    constexpr int U = 8 / R;  // parts of each of a warp's R rows that are in flight together
#pragma unroll 1
    for (int row0 = blockIdx.y * 32 + R * (threadIdx.x >> 5); row0 < (int)blockIdx.y * 32 + 32; row0 += 8 * R) {
        bool in[R];
        float M[R], L[R];
        float4 o[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int in_slot = (row0 + i) % kRows / G;
            in[i] = in_slot < p.slot_tokens && (row0 + i) / kRows * p.slot_tokens + in_slot < c.tokens;
            M[i] = -INFINITY;
            L[i] = 0.f;
            o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (!in[0]) return;  // rows of a slot without tokens are its last
        float2 ml[R];  // of part `lane`; the parts behind 32 are read again below
        auto load_ml = [&](int k0) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                ml[i] = make_float2(-INFINITY, 0.f);
                if (in[i] && k0 + lane < parts) ml[i] = p.part_ml[(size_t)slot(k0 + lane) * unit_rows + row0 + i];
            }
        };
        for (int k0 = (parts - 1) & ~31; k0 >= 0; k0 -= 32) {
            load_ml(k0);
#pragma unroll
            for (int i = 0; i < R; ++i) M[i] = fmaxf(M[i], ml[i].x);
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) M[i] = fmaxf(M[i], __shfl_xor_sync(0xffffffffu, M[i], x));
        for (int k0 = 0; k0 < parts; k0 += 32) {
            if (k0 > 0) load_ml(k0);
            float w[R];
            unsigned there[R];  // parts that saw something: the others have no O
#pragma unroll
            for (int i = 0; i < R; ++i) {
                w[i] = ml[i].x > -INFINITY ? exp2f((ml[i].x - M[i]) * qs) : 0.f;
                L[i] += warp_sum(w[i] * ml[i].y);
                there[i] = __ballot_sync(0xffffffffu, ml[i].x > -INFINITY);
            }
            const int n = min(32, parts - k0);
#pragma unroll 1
            for (int k1 = 0; k1 < n; k1 += U) {
                float4 v[U][R];
#pragma unroll
                for (int k = 0; k < U; ++k)
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        v[k][i] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if ((there[i] >> (k1 + k)) & 1)
                            v[k][i] = reinterpret_cast<const float4 *>(
                                p.part_o)[((size_t)slot(k0 + k1 + k) * unit_rows + row0 + i) * 32 + lane];
                    }
#pragma unroll
                for (int k = 0; k < U; ++k)
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        const float wk = __shfl_sync(0xffffffffu, w[i], k1 + k);
                        o[i] = make_float4(fmaf(wk, v[k][i].x, o[i].x), fmaf(wk, v[k][i].y, o[i].y), fmaf(wk, v[k][i].z, o[i].z),
                                           fmaf(wk, v[k][i].w, o[i].w));
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (!in[i]) continue;
            const float inv = L[i] == 0.f ? 0.f : 1.f / L[i];
            const int row = row0 + i, in_slot = row % kRows / G, tok = row / kRows * p.slot_tokens + in_slot;
            uint2 h;
            h.x = h2_bits(__floats2half2_rn(o[i].x * inv, o[i].y * inv));
            h.y = h2_bits(__floats2half2_rn(o[i].z * inv, o[i].w * inv));
            const int hq = c.g * G + row % kRows - in_slot * G;
            *reinterpret_cast<uint2 *>(p.out + ((size_t)(c.row + tok) * p.Hq + hq) * 128 + 4 * lane) = h;
        }
    }
}

// Grid (CTAs of the main kernel, blocks of 32 rows). The kernel costs a few latencies and is bound by nothing else, so a unit
// of at most eight rows has one a warp, with eight parts in flight (four single tokens: 14.2 us against 14.7 with two
// rows, one at 32768 positions 24.1 against 26.3).
template <int R>
__global__ void __launch_bounds__(256, 3) chunk_join_kernel(const __grid_constant__ ChunkAttnParams p, int unit_rows) {
    grid_dep_launch();
    grid_dep_wait();
    const Cut c = p.cuts[blockIdx.x];
    const int G = p.Hq / p.Hkv;
    if (!c.valid) return;
    if (c.tokens * G <= 8)
        join_rows<1>(p, c, G, unit_rows);
    else
        join_rows<R>(p, c, G, unit_rows);
}

// ------------------------------------------------------------------ host side

// A tensor map of fp16 rows of 128 dims in boxes of 64: rows x y x z with the given strides in bytes and box sizes.
static int row_map(CUtensorMap *m, const uint16_t *base, const cuuint64_t (&dims)[4], const cuuint64_t (&strides)[3],
                   const cuuint32_t (&box)[4]) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return fail(I4_ECUDA, "i4_paged_gqa_chunk: cuTensorMapEncodeTiled is not available");
    const cuuint32_t step[4] = {1, 1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<uint16_t *>(base), dims, strides, box, step,
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
static int launch_chunk(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, ChunkAttnParams p, int sms,
                        cudaStream_t stream) {
    const unsigned unit = NQ * p.slot_tokens;
    p.unit_inv = (unsigned)((0x100000000ull + unit - 1) / unit);
    const int st = cuda_check(launch(chunk_attn_kernel<NQ>, dim3(sms), dim3(Cfg<NQ>::kThreads), Cfg<NQ>::kSmem, stream, g_pdl, tq, tk,
                                     tv, p),
                              "i4_paged_gqa_chunk");
    if (st) return st;
    return cuda_check(launch(chunk_join_kernel<Cfg<NQ>::kJoinRows>, dim3(sms, Cfg<NQ>::kUnitRows / 32), dim3(256), 0, stream, g_pdl, p,
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

// Workspace: cuts | part_ml | part_o; two parts for every CTA, of the larger unit's rows.
constexpr size_t kWsRows = (size_t)2 * kNumSMs * Cfg<2>::kUnitRows;
constexpr size_t kWsMl = (kNumSMs * sizeof(Cut) + 255) / 256 * 256;
constexpr size_t kWsO = kWsMl + kWsRows * sizeof(float2);
constexpr size_t kWsBytes = kWsO + kWsRows * 128 * sizeof(float);
static_assert(kWsO % 256 == 0, "parts are read 16 bytes at a time");

}  // namespace i4

using namespace i4;

extern "C" size_t i4_paged_gqa_chunk_ws_bytes(void) { return kWsBytes; }

extern "C" int i4_paged_gqa_chunk(const i4_chunk_attn_args *args, void *stream) {
    if (!args) return fail(I4_EINVAL, "i4_paged_gqa_chunk: null args");
    const auto [q, q_stride, k_pool, v_pool, page_table, q_start, ctx_len, out, ws, ws_bytes, T, B, Hq, Hkv, D, page_size,
                max_pages_per_seq, num_pages, window, max_q, scale] = *args;
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
    // a CTA's share of the line of tiles is counted in 31 bits
    if ((double)Hkv * (T / (kRows / (Hq / Hkv)) + (double)B) * ((double)max_pages_per_seq * page_size / kTile + 3) > 1e11)
        return fail(I4_EUNSUPPORTED, "i4_paged_gqa_chunk: T, B, Hkv and the page-table row are too large together");
    // |q . k| is at most 128 * 65504^2 = 5.5e11: a scaled score stays a finite float
    if (!(scale > 0.f) || scale > 1e20f) return fail(I4_EINVAL, "i4_paged_gqa_chunk: scale %g must be positive, at most 1e20", scale);
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
    const int G = Hq / Hkv;
    CUtensorMap tq, tk, tv;
    // q as [T][Hq][128] in boxes of one kv head's rows of a slot's tokens; the pools as [pages][Hkv][P][128] in boxes of a page
    const cuuint64_t page = 256ull * page_size, tok = 2ull * (cuuint64_t)q_stride;
    const cuuint64_t qd[4] = {128, (cuuint64_t)Hq, (cuuint64_t)T, 1}, qs[3] = {256, tok, tok};
    const cuuint64_t pd[4] = {128, (cuuint64_t)page_size, (cuuint64_t)Hkv, (cuuint64_t)num_pages}, ps[3] = {256, page, page * Hkv};
    const cuuint32_t qb[4] = {64, (cuuint32_t)G, (cuuint32_t)(kRows / G), 1}, pb[4] = {64, (cuuint32_t)page_size, 1, 1};
    if ((st = row_map(&tq, q, qd, qs, qb))) return st;
    if ((st = row_map(&tk, k_pool, pd, ps, pb))) return st;
    if ((st = row_map(&tv, v_pool, pd, ps, pb))) return st;
    ChunkAttnParams p = {q,   k_pool, v_pool, q_stride,  page_table,        q_start,   ctx_len, out,  T,
                         B,   Hq,     Hkv,    page_size, max_pages_per_seq, num_pages, window,  scale};
    char *w = reinterpret_cast<char *>(ws);
    p.cuts = reinterpret_cast<Cut *>(w);
    p.part_ml = reinterpret_cast<float2 *>(w + kWsMl);
    p.part_o = reinterpret_cast<float *>(w + kWsO);
    p.slot_tokens = kRows / G;
    // One slot of 128 rows when every chunk fits it: the other warpgroup would idle. Also when units of one slot find an SM each
    // and have a few tiles only, as far as the host can tell from the width of the page table and the number of its rows (a cache
    // of wide rows or many slots does not get there: the prompt of 512 below then takes 19.5 us): a slot alone takes a tile in 1.3 us, two in 1.9, and the kernel begins and ends sooner. (28
    // heads on 4, 512 tokens at 512 positions: 17.0 us against 19.6, at 1024: 26.5 and 26.0, at 2048: 38.4 against 32.5; 256
    // tokens: 13.4 against 16.0, 21.4 against 23.0, 27.7 against 25.7.)
    const int longest = max_q > 0 && max_q < T ? max_q : T;
    const long long units = ((long long)(T + p.slot_tokens - 1) / p.slot_tokens + B) * Hkv;  // at most
    const bool few = units <= sms && (long long)max_pages_per_seq * page_size <= 1024;
    if (longest <= p.slot_tokens || few) return launch_chunk<1>(tq, tk, tv, p, sms, (cudaStream_t)stream);
    return launch_chunk<2>(tq, tk, tv, p, sms, (cudaStream_t)stream);
}
