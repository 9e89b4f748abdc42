// The pages of a cache: copying, reserving, forking, freeing and compacting.
//
// State, all on the device:  page_table [S][max_pages], ctx_len [S] (tokens of
// each sequence) and refs [num_pages] (sequences that hold the page; 0 = free).
// Sequence s holds the pages page_table[s][0 .. ceil(ctx_len[s] / P)). A page
// that is not full has one holder, since a fork copies it.
//
// Every operation is deterministic: pages are handed out lowest id first, in the
// order of the requests. Reserving, forking and compacting decide in one CTA (a
// few thousand integers, bound by the latency of a handful of dependent passes
// over them: several CTAs would need grid-wide barriers that cost as much) and
// leave a list of copies in the workspace; a second kernel over the whole GPU,
// brought up while the first runs, moves the data of all pools at once and is
// bound by HBM. Three forks of a short sequence in 4 pools take 7.4 us, 63 of
// one of 4015 tokens in 56 pools 21.5 us (12 to decide; 54 MB written, the one
// source page read once from HBM), compacting 9 pages of 4 pools 7 us, 300 pages
// of 56 pools 95 us (12 to decide). Reserving 17 tokens for each of 64 sequences
// and freeing them again takes 9.9 us, for 512 sequences in 65536 pages 23.
#include <mutex>

#include "chunk.cuh"
#include "common.cuh"

namespace i4 {

constexpr int kPlanThreads = 1024;
constexpr int kMaxSeqs = 16384;      // a 64 KB table of owners in shared memory
constexpr int kMaxPages = 1 << 20;   // a sum over 1024 requests of at most this many pages fits 31 bits
constexpr int kPoolsPerLaunch = 256;  // pool addresses in the kernel's parameters
constexpr int kLanePages = 8;         // page ids that a lane has in flight: a row of 256 pages costs one latency, not eight

struct PoolPtrs {
    unsigned char *p[kPoolsPerLaunch];
};

// ------------------------------------------------------------------ block-wide scans

struct ScanSmem {
    int warp[kPlanThreads / 32];
    int total;
};

// Exclusive prefix sum of v over the CTA's threads, and the sum over all of them.
__device__ __forceinline__ int block_scan(int v, int &total, ScanSmem &sm) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) sm.warp[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        const int w = sm.warp[lane];
        int iw = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, iw, o);
            if (lane >= o) iw += u;
        }
        sm.warp[lane] = iw - w;
        if (lane == 31) sm.total = iw;
    }
    __syncthreads();
    const int r = sm.warp[warp] + inc - v;
    total = sm.total;
    __syncthreads();  // the scratch is free for the next scan
    return r;
}

// The `want` lowest free pages in ascending order to list[]; returns how many there are (at most want).
__device__ __forceinline__ int find_free(const int32_t *refs, int num_pages, int want, int32_t *list, ScanSmem &sm) {
    int found = 0;
    for (int p0 = 0; p0 < num_pages && found < want; p0 += 4 * kPlanThreads) {  // block-uniform trips
        const int p = p0 + 4 * threadIdx.x;
        int r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = p + i < num_pages ? *(volatile const int32_t *)(refs + p + i) : 1;  // written by atomics
        int total;
        int at = found + block_scan((r[0] == 0) + (r[1] == 0) + (r[2] == 0) + (r[3] == 0), total, sm);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (r[i] == 0) {
                if (at < want) list[at] = p + i;
                ++at;
            }
        found += total;
    }
    __syncthreads();
    return found < want ? found : want;
}

__device__ __forceinline__ int pages_of(int ctx, int P, int max_pages) {
    const int n = ctx <= 0 ? 0 : (ctx - 1) / P + 1;
    return n < max_pages ? n : max_pages;
}

struct CacheArgs {
    int32_t *table, *ctx_len, *refs;
    int S, max_pages, P, num_pages;
};

// ------------------------------------------------------------------ plans (one CTA)

// Workspace of every operation: count | a | b | c, arrays of `cap` int32 each.
struct Lists {
    int32_t *count, *a, *b, *c;
};
__host__ __device__ inline Lists ws_lists(void *ws, size_t cap) {
    int32_t *p = reinterpret_cast<int32_t *>(ws);
    return {p, p + 64, p + 64 + cap, p + 64 + 2 * cap};
}

__global__ void __launch_bounds__(kPlanThreads) kv_reserve_kernel(const CacheArgs c, const int32_t *seqs, const int32_t *add,
                                                                  int n, int32_t *status, Lists ws) {
    grid_dep_launch();
    grid_dep_wait();
    extern __shared__ int owner[];
    __shared__ ScanSmem sm;
    const int tid = threadIdx.x;
    for (int s = tid; s < c.S; s += kPlanThreads) owner[s] = n;
    __syncthreads();
    for (int i = tid; i < n; i += kPlanThreads)
        if (seqs[i] >= 0 && seqs[i] < c.S) atomicMin(&owner[seqs[i]], i);
    __syncthreads();
    // pages that each request needs, and where its pages begin in the list of free ones
    int want = 0;
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int i = i0 + tid;
        int need = -1;
        if (i < n) {
            const int s = seqs[i];
            if (s >= 0 && s < c.S && owner[s] == i && add[i] >= 0 && c.ctx_len[s] >= 0 &&
                (long long)c.ctx_len[s] + add[i] <= (long long)c.max_pages * c.P)
                need = min(pages_of(c.ctx_len[s] + add[i], c.P, c.max_pages) - pages_of(c.ctx_len[s], c.P, c.max_pages),
                           c.num_pages + 1);
        }
        int total;
        const int at = want + block_scan(need > 0 ? need : 0, total, sm);
        if (i < n) {
            ws.b[i] = need;
            ws.c[i] = at;
        }
        want = want > c.num_pages - total ? c.num_pages + 1 : want + total;  // more than exist is never granted
    }
    const int have = find_free(c.refs, c.num_pages, want < c.num_pages ? want : c.num_pages, ws.a, sm);
    for (int i = tid >> 5; i < n; i += kPlanThreads / 32) {  // one warp per request
        const int need = ws.b[i], at = ws.c[i], lane = tid & 31;
        int st = 0;
        if (need < 0)
            st = 2;
        else if (need > 0 && at + need > have)
            st = 1;
        if (st == 0) {
            const int s = seqs[i], old = pages_of(c.ctx_len[s], c.P, c.max_pages);
            for (int j = lane; j < need; j += 32) {
                const int page = ws.a[at + j];
                c.table[(size_t)s * c.max_pages + old + j] = page;
                c.refs[page] = 1;
            }
            __syncwarp();
            if (lane == 0) c.ctx_len[s] += add[i];
        }
        if (lane == 0 && status) status[i] = st;
    }
}

__global__ void __launch_bounds__(kPlanThreads) kv_fork_kernel(const CacheArgs c, const int32_t *src, const int32_t *dst, int n,
                                                               int32_t *status, Lists ws, int smem_refs) {
    grid_dep_launch();  // the copy may come up; it waits for this kernel's end before it reads anything
    grid_dep_wait();
    extern __shared__ int owner[];  // [S], then the counts of the pages where they fit
    __shared__ ScanSmem sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t kNone = n;
    int32_t *refs = smem_refs ? owner + c.S : c.refs;
    for (int s = tid; s < c.S; s += kPlanThreads) owner[s] = kNone;
    if (smem_refs)
        for (int p = tid; p < c.num_pages; p += kPlanThreads) refs[p] = c.refs[p];
    __syncthreads();
    for (int i = tid; i < n; i += kPlanThreads)
        if (dst[i] >= 0 && dst[i] < c.S) atomicMin(&owner[dst[i]], i);
    __syncthreads();
    auto valid = [&](int i) {
        const int s = src[i], d = dst[i];
        return s >= 0 && s < c.S && d >= 0 && d < c.S && owner[d] == i && owner[s] == kNone;
    };
    // give back what the targets hold, and hold the full pages of the sources
    for (int i = warp; i < n; i += kPlanThreads / 32) {
        if (!valid(i)) continue;
        const int32_t *old = c.table + (size_t)dst[i] * c.max_pages, *row = c.table + (size_t)src[i] * c.max_pages;
        const int held = pages_of(c.ctx_len[dst[i]], c.P, c.max_pages);
        const int full = min(max(c.ctx_len[src[i]], 0) / c.P, c.max_pages);
        for (int j0 = lane; j0 < max(held, full); j0 += 32 * kLanePages) {
            int a[kLanePages], b[kLanePages];
#pragma unroll
            for (int k = 0; k < kLanePages; ++k) {
                const int j = j0 + 32 * k;
                a[k] = j < held ? old[j] : -1;
                b[k] = j < full ? row[j] : -1;
            }
#pragma unroll
            for (int k = 0; k < kLanePages; ++k) {
                if (a[k] >= 0 && a[k] < c.num_pages) atomicSub(&refs[a[k]], 1);
                if (b[k] >= 0 && b[k] < c.num_pages) atomicAdd(&refs[b[k]], 1);
            }
        }
    }
    __syncthreads();
    // one free page for every source whose last page is not full
    int want = 0;
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int i = i0 + tid;
        int need = 0;
        if (i < n && valid(i)) {
            const int ctx = max(c.ctx_len[src[i]], 0);
            need = ctx % c.P != 0 && ctx / c.P < c.max_pages;
        }
        int total;
        const int at = want + block_scan(need, total, sm);
        if (i < n) ws.b[i] = need ? at : -1;
        want += total;
    }
    const int have = find_free(refs, c.num_pages, want, ws.a, sm);
    for (int i = warp; i < n; i += kPlanThreads / 32) {
        const bool ok = valid(i);
        const int at = ws.b[i];
        __syncwarp();  // every lane has read ws.b[i], which the copy list below shares
        int from = 0, to = 0, fill = 0;
        const bool room = at < 0 || at < have;
        if (ok) {
            const int32_t *row = c.table + (size_t)src[i] * c.max_pages;
            int32_t *out = c.table + (size_t)dst[i] * c.max_pages;
            const int ctx = min(max(c.ctx_len[src[i]], 0), c.max_pages * c.P), full = ctx / c.P;
            if (room) {
                for (int j0 = lane; j0 < c.max_pages; j0 += 32 * kLanePages) {
                    int a[kLanePages];
#pragma unroll
                    for (int k = 0; k < kLanePages; ++k) a[k] = j0 + 32 * k < full ? row[j0 + 32 * k] : -1;
#pragma unroll
                    for (int k = 0; k < kLanePages; ++k)
                        if (j0 + 32 * k < c.max_pages) out[j0 + 32 * k] = a[k];
                }
            } else {  // no page left: the target stays empty and holds nothing
                for (int j = lane; j < full; j += 32)
                    if (row[j] >= 0 && row[j] < c.num_pages) atomicSub(&refs[row[j]], 1);
                for (int j = lane; j < c.max_pages; j += 32) out[j] = -1;
            }
            if (at >= 0 && room) {
                from = row[full];
                to = ws.a[at];
                fill = from >= 0 && from < c.num_pages ? ctx % c.P : 0;
            }
            __syncwarp();
            if (lane == 0) {
                if (at >= 0 && room) {
                    out[full] = to;
                    refs[to] = 1;
                }
                c.ctx_len[dst[i]] = room ? ctx : 0;
            }
        }
        if (lane == 0) {
            ws.b[i] = from;
            ws.c[i] = to;
            ws.c[n + i] = fill;
            if (status) status[i] = !ok ? 2 : (room ? 0 : 1);
        }
    }
    if (smem_refs) {
        __syncthreads();
        for (int p = tid; p < c.num_pages; p += kPlanThreads) c.refs[p] = refs[p];
    }
}

// One warp per sequence. The exchange makes a sequence that is named twice release its pages once.
__global__ void kv_free_kernel(const CacheArgs c, const int32_t *seqs, int n) {
    grid_dep_launch();
    grid_dep_wait();
    const int i = (int)((blockIdx.x * blockDim.x + threadIdx.x) >> 5), lane = threadIdx.x & 31;
    if (i >= n) return;
    const int s = seqs[i];
    if (s < 0 || s >= c.S) return;
    int ctx = 0;
    if (lane == 0) ctx = atomicExch(&c.ctx_len[s], 0);
    ctx = __shfl_sync(0xffffffffu, ctx, 0);
    if (ctx <= 0) return;
    const int held = pages_of(ctx, c.P, c.max_pages);
    int32_t *row = c.table + (size_t)s * c.max_pages;
    for (int j = lane; j < c.max_pages; j += 32) {
        const int p = row[j];
        if (j < held && p >= 0 && p < c.num_pages) atomicSub(&c.refs[p], 1);
        row[j] = -1;
    }
}

// a: target, b: source of each move; c[p]: the new id of a page p >= n_live.
__global__ void __launch_bounds__(kPlanThreads) kv_compact_plan_kernel(int32_t *refs, int num_pages, int32_t *n_live_out,
                                                                      Lists ws) {
    grid_dep_launch();
    grid_dep_wait();
    __shared__ ScanSmem sm;
    const int tid = threadIdx.x;
    int mine = 0, n_live;
    for (int p = tid; p < num_pages; p += kPlanThreads) mine += refs[p] > 0;
    block_scan(mine, n_live, sm);
    int gaps = 0, movers = 0;
    for (int p0 = 0; p0 < num_pages; p0 += 4 * kPlanThreads) {
        const int p = p0 + 4 * tid;
        int gap[4], move[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = p + i < num_pages, live = in && refs[p + i] > 0;
            gap[i] = in && !live && p + i < n_live;
            move[i] = live && p + i >= n_live;
            if (in && !live && p + i >= n_live) ws.c[p + i] = p + i;  // an id that a table should not hold stays
        }
        // both counts in one scan: pages of one trip number at most 4096, so 16 bits hold each
        int total;
        const int at = block_scan((gap[0] + gap[1] + gap[2] + gap[3]) | (move[0] + move[1] + move[2] + move[3]) << 16, total, sm);
        int g = gaps + (at & 0xffff), m = movers + (at >> 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (gap[i]) ws.a[g++] = p + i;
            if (move[i]) ws.b[m++] = p + i;
        }
        gaps += total & 0xffff;
        movers += total >> 16;
    }
    __syncthreads();
    for (int i = tid; i < movers; i += kPlanThreads) {  // as many movers as gaps
        const int to = ws.a[i], from = ws.b[i];
        refs[to] = refs[from];
        refs[from] = 0;
        ws.c[from] = to;
    }
    if (tid == 0) {
        *ws.count = movers;
        ws.count[1] = n_live;
        if (n_live_out) *n_live_out = n_live;
    }
}

// ------------------------------------------------------------------ data movement (the whole GPU)

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;  // 16-byte loads in flight per thread

__device__ __forceinline__ void copy_span(unsigned char *dst, const unsigned char *src, int vecs, int part) {
    uint4 v[kCopyUnroll];
    const int v0 = part * kCopyThreads * kCopyUnroll + threadIdx.x;
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
        if (v0 + u * kCopyThreads < vecs) v[u] = __ldcs(reinterpret_cast<const uint4 *>(src) + v0 + u * kCopyThreads);
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
        if (v0 + u * kCopyThreads < vecs) __stcs(reinterpret_cast<uint4 *>(dst) + v0 + u * kCopyThreads, v[u]);
}

// Whole pages src[i] -> dst[i] of pool blockIdx.y; n_dev, when given, is the device's count. Work item: (i, part of the page). The
// first remap_blocks blocks of a row of the grid instead give table entries of held pages at or above n_live (n_dev[1])
// the page's new id. Bound by HBM: 300 pages of 56 pools in 83 us, of whose 551 MB 501 have passed HBM by then (6.0 TB/s); the
// rest is written back from L2 later.
__global__ void __launch_bounds__(kCopyThreads) kv_copy_kernel(const __grid_constant__ PoolPtrs pools, const int32_t *src,
                                                               const int32_t *dst, int n, const int32_t *n_dev, int num_pages,
                                                               int page_vecs, int parts, const CacheArgs c, const int32_t *new_id,
                                                               int remap_blocks) {
    grid_dep_launch();
    grid_dep_wait();
    if ((int)blockIdx.x < remap_blocks) {
        const int n_live = n_dev[1];
        const long long entries = (long long)c.S * c.max_pages, step = (long long)remap_blocks * gridDim.y * kCopyThreads;
        for (long long x = (blockIdx.x * (long long)gridDim.y + blockIdx.y) * kCopyThreads + threadIdx.x; x < entries; x += step) {
            const int s = (int)(x / c.max_pages), j = (int)(x % c.max_pages), p = c.table[x];
            if (j < pages_of(c.ctx_len[s], c.P, c.max_pages) && p >= n_live && p < c.num_pages) c.table[x] = new_id[p];
        }
        return;
    }
    if (n_dev) n = min(n, *n_dev);
    unsigned char *pool = pools.p[blockIdx.y];
    const unsigned items = (unsigned)n * (unsigned)parts;
    for (unsigned it = blockIdx.x - remap_blocks; it < items; it += gridDim.x - remap_blocks) {
        const unsigned i = it / (unsigned)parts;
        const int from = src[i], to = dst[i];
        if (from < 0 || from >= num_pages || to < 0 || to >= num_pages || from == to) continue;
        copy_span(pool + (size_t)to * page_vecs * 16, pool + (size_t)from * page_vecs * 16, page_vecs, (int)(it - i * parts));
    }
}

// The first `fill` rows of every head of page from[i] -> page to[i] in pool blockIdx.y. Work item: (i, part of the page); the
// filled rows of the heads of a page are numbered one after the other, and a thread has kCopyUnroll of them in flight.
__global__ void __launch_bounds__(kCopyThreads) kv_copy_rows_kernel(const __grid_constant__ PoolPtrs pools, const int32_t *from,
                                                                    const int32_t *to, const int32_t *fill, int n, int Hkv, int P,
                                                                    int row_vecs, int parts) {
    grid_dep_launch();
    grid_dep_wait();
    const unsigned items = (unsigned)n * (unsigned)parts;
    for (unsigned it = blockIdx.x; it < items; it += gridDim.x) {
        const unsigned i = it / (unsigned)parts;
        const int span = fill[i] * row_vecs, vecs = span * Hkv;  // 16-byte vectors of one head, of all
        int x = (int)(it - i * parts) * kCopyThreads * kCopyUnroll + threadIdx.x;
        if (x - (int)threadIdx.x >= vecs) continue;
        const uint4 *s = reinterpret_cast<const uint4 *>(pools.p[blockIdx.y]) + (size_t)from[i] * Hkv * P * row_vecs;
        uint4 *d = reinterpret_cast<uint4 *>(pools.p[blockIdx.y]) + (size_t)to[i] * Hkv * P * row_vecs;
        int head = x / span, in_head = x - head * span;
        uint4 v[kCopyUnroll];
        int at[kCopyUnroll];
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u) {
            at[u] = head * P * row_vecs + in_head;
            if (x + u * kCopyThreads < vecs) v[u] = __ldcg(s + at[u]);
            in_head += kCopyThreads;
            while (in_head >= span) {  // once at most where a head has 256 filled vectors
                in_head -= span;
                ++head;
            }
        }
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u)
            if (x + u * kCopyThreads < vecs) d[at[u]] = v[u];
    }
}

// ------------------------------------------------------------------ host side

static int check_pools(const char *what, void *const *pools, int n_pools, int num_pages, int Hkv, int P, int D) {
    if (!pools) return fail(I4_EINVAL, "%s: null pointer", what);
    if (n_pools < 1 || num_pages < 1 || num_pages > kMaxPages || Hkv < 1 || P < 1 || D < 8 || D % 8 ||
        (long long)Hkv * P * D > (1 << 22))
        return fail(I4_EINVAL, "%s: bad sizes (pools %d, pages %d, Hkv %d, page_size %d, D %d)", what, n_pools, num_pages, Hkv, P,
                    D);
    for (int i = 0; i < n_pools; ++i) {
        if (!pools[i]) return fail(I4_EINVAL, "%s: pool %d is null", what, i);
        if (!aligned(pools[i], 16)) return fail(I4_EALIGN, "%s: pool %d must be 16-byte aligned", what, i);
    }
    return I4_OK;
}

static int check_cache(const char *what, const i4_kv_cache *c) {
    if (!c || !c->page_table || !c->ctx_len || !c->refs) return fail(I4_EINVAL, "%s: null pointer", what);
    if (c->n_seqs < 1 || c->max_pages_per_seq < 1 || c->page_size < 1 || c->num_pages < 1 || c->num_pages > kMaxPages ||
        (long long)c->max_pages_per_seq * c->page_size > 0x7fffffffll)
        return fail(I4_EINVAL, "%s: bad sizes (sequences %d, pages per sequence %d, page_size %d, pages %d)", what, c->n_seqs,
                    c->max_pages_per_seq, c->page_size, c->num_pages);
    if (c->n_seqs > kMaxSeqs) return fail(I4_EUNSUPPORTED, "%s: %d sequences (at most %d)", what, c->n_seqs, kMaxSeqs);
    if (!aligned(c->page_table, 4) || !aligned(c->ctx_len, 4) || !aligned(c->refs, 4))
        return fail(I4_EALIGN, "%s: page_table, ctx_len and refs must be 4-byte aligned", what);
    return I4_OK;
}

static int check_list(const char *what, int n, const void *a, const void *b) {
    if (n < 0 || n > kMaxSeqs) return fail(I4_EINVAL, "%s: %d entries (0 to %d)", what, n, kMaxSeqs);
    if (n && (!a || !b)) return fail(I4_EINVAL, "%s: null pointer", what);
    if (!aligned(a, 4) || !aligned(b, 4)) return fail(I4_EALIGN, "%s: lists must be 4-byte aligned", what);
    return I4_OK;
}

static size_t ws_cap(int num_pages, int n_seqs) { return (size_t)num_pages + 2 * (size_t)n_seqs; }

static int check_ws(const char *what, void *ws, size_t bytes, int num_pages, int n_seqs) {
    const size_t need = i4_kv_pages_ws_bytes(num_pages, n_seqs);
    if (!ws || bytes < need) return fail(I4_EINVAL, "%s: workspace of %zu bytes needed (got %zu)", what, need, bytes);
    if (!aligned(ws, 16)) return fail(I4_EALIGN, "%s: workspace must be 16-byte aligned", what);
    return I4_OK;
}

static CacheArgs cache_args(const i4_kv_cache *c) {
    return {c->page_table, c->ctx_len, c->refs, c->n_seqs, c->max_pages_per_seq, c->page_size, c->num_pages};
}

// The plan kernels keep an int per sequence, and the fork one per page too where they fit, in dynamic shared memory: many
// targets of one source count the same pages up and down, and 63 of them over 251 pages took 17 us on global atomics. The
// attribute that allows more than 48 KB belongs to the kernel on the device, whoever calls it: it is set once, to the most
// that any call takes.
constexpr size_t kPlanSmem = 200 * 1024;
static_assert(kMaxSeqs * sizeof(int) <= kPlanSmem, "the table of owners always fits");

constexpr int kMaxDevices = 64;
struct PlanState {
    std::once_flag once;
    cudaError_t err = cudaSuccess;
};

static int plan_smem(size_t bytes, const char *what) {
    if (bytes <= 47 * 1024) return I4_OK;
    static PlanState state[kMaxDevices];
    int dev = 0;
    const int st = cuda_check(cudaGetDevice(&dev), what);
    if (st) return st;
    if (dev < 0 || dev >= kMaxDevices) return fail(I4_EUNSUPPORTED, "%s: device %d", what, dev);
    PlanState &d = state[dev];
    std::call_once(d.once, [&] {
        d.err = cudaFuncSetAttribute(kv_reserve_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPlanSmem);
        if (d.err == cudaSuccess)
            d.err = cudaFuncSetAttribute(kv_fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPlanSmem);
    });
    return d.err == cudaSuccess ? I4_OK : cuda_check(d.err, what);
}

// Blocks along x for `items` work items in each of m pools: enough for the whole GPU, and no more than there are items.
static unsigned copy_grid(long long items, int m) {
    const long long most = (32ll * kNumSMs + m - 1) / m;
    return (unsigned)(items < most ? (items > 0 ? items : 1) : most);
}

static int launch_copy(void *const *pools, int n_pools, const int32_t *src, const int32_t *dst, int n, const int32_t *n_dev,
                       int num_pages, long long page_bytes, const CacheArgs *remap, const int32_t *new_id, cudaStream_t stream,
                       const char *what) {
    const int vecs = (int)(page_bytes / 16), parts = (vecs + kCopyThreads * kCopyUnroll - 1) / (kCopyThreads * kCopyUnroll);
    for (int p0 = 0; p0 < n_pools; p0 += kPoolsPerLaunch) {
        PoolPtrs pp;
        const int m = n_pools - p0 < kPoolsPerLaunch ? n_pools - p0 : kPoolsPerLaunch;
        for (int i = 0; i < m; ++i) pp.p[i] = reinterpret_cast<unsigned char *>(pools[p0 + i]);
        int blocks = 0;
        if (remap && p0 == 0) {
            const long long b = ((long long)remap->S * remap->max_pages + kCopyThreads - 1) / kCopyThreads, rows = (b + m - 1) / m;
            blocks = (int)(rows < 8 ? rows : 8);
        }
        const dim3 grid(blocks + copy_grid((long long)n * parts, m), m);
        const int st = cuda_check(launch(kv_copy_kernel, grid, dim3(kCopyThreads), 0, stream,
                                         g_pdl, pp, src, dst, n, n_dev, num_pages, vecs, parts,
                                         remap ? *remap : CacheArgs{}, new_id, blocks),
                                  what);
        if (st) return st;
    }
    return I4_OK;
}

}  // namespace i4

using namespace i4;

extern "C" size_t i4_kv_pages_ws_bytes(int num_pages, int n_seqs) {
    if (num_pages < 1 || num_pages > kMaxPages || n_seqs < 1 || n_seqs > kMaxSeqs) return 0;
    return (64 + 3 * ws_cap(num_pages, n_seqs)) * sizeof(int32_t);
}

extern "C" int i4_kv_pages_copy(void *const *pools, int n_pools, int num_pages, int Hkv, int page_size, int D, const int32_t *src,
                                const int32_t *dst, int n, void *stream) {
    int st = check_pools("i4_kv_pages_copy", pools, n_pools, num_pages, Hkv, page_size, D);
    if (st) return st;
    if (n < 0 || n > kMaxPages) return fail(I4_EINVAL, "i4_kv_pages_copy: %d pages", n);
    if (n == 0) return I4_OK;
    if (!src || !dst) return fail(I4_EINVAL, "i4_kv_pages_copy: null pointer");
    if (!aligned(src, 4) || !aligned(dst, 4)) return fail(I4_EALIGN, "i4_kv_pages_copy: lists must be 4-byte aligned");
    return launch_copy(pools, n_pools, src, dst, n, nullptr, num_pages, (long long)Hkv * page_size * D * 2, nullptr,
                       nullptr, (cudaStream_t)stream, "i4_kv_pages_copy");
}

extern "C" int i4_kv_pages_reserve(const i4_kv_cache *cache, const int32_t *seqs, const int32_t *add, int n, int32_t *status, void *ws,
                                   size_t ws_bytes, void *stream) {
    int st = check_cache("i4_kv_pages_reserve", cache);
    if (!st) st = check_list("i4_kv_pages_reserve", n, seqs, add);
    if (!st) st = check_ws("i4_kv_pages_reserve", ws, ws_bytes, cache->num_pages, cache->n_seqs);
    if (st || n == 0) return st;
    if (n > cache->n_seqs) return fail(I4_EINVAL, "i4_kv_pages_reserve: %d requests for %d sequences", n, cache->n_seqs);
    const size_t smem = (size_t)cache->n_seqs * sizeof(int);
    if ((st = plan_smem(smem, "i4_kv_pages_reserve"))) return st;
    return cuda_check(launch(kv_reserve_kernel, dim3(1), dim3(kPlanThreads), smem, (cudaStream_t)stream, g_pdl, cache_args(cache), seqs,
                             add, n, status, ws_lists(ws, ws_cap(cache->num_pages, cache->n_seqs))),
                      "i4_kv_pages_reserve");
}

extern "C" int i4_kv_pages_fork(const i4_kv_cache *cache, void *const *pools, int n_pools, int Hkv, int D, const int32_t *src,
                                const int32_t *dst, int n, int32_t *status, void *ws, size_t ws_bytes, void *stream) {
    int st = check_cache("i4_kv_pages_fork", cache);
    if (!st) st = check_pools("i4_kv_pages_fork", pools, n_pools, cache->num_pages, Hkv, cache->page_size, D);
    if (!st) st = check_list("i4_kv_pages_fork", n, src, dst);
    if (!st) st = check_ws("i4_kv_pages_fork", ws, ws_bytes, cache->num_pages, cache->n_seqs);
    if (st || n == 0) return st;
    if (n > cache->n_seqs) return fail(I4_EINVAL, "i4_kv_pages_fork: %d forks for %d sequences", n, cache->n_seqs);
    size_t smem = ((size_t)cache->n_seqs + cache->num_pages) * sizeof(int);
    const int smem_refs = smem <= kPlanSmem;
    if (!smem_refs) smem = (size_t)cache->n_seqs * sizeof(int);
    if ((st = plan_smem(smem, "i4_kv_pages_fork"))) return st;
    const Lists L = ws_lists(ws, ws_cap(cache->num_pages, cache->n_seqs));
    st = cuda_check(launch(kv_fork_kernel, dim3(1), dim3(kPlanThreads), smem, (cudaStream_t)stream, g_pdl, cache_args(cache), src, dst,
                           n, status, L, smem_refs),
                    "i4_kv_pages_fork");
    if (st) return st;
    const int row_vecs = D / 8, vecs = Hkv * cache->page_size * row_vecs;
    const int parts = (vecs + kCopyThreads * kCopyUnroll - 1) / (kCopyThreads * kCopyUnroll);
    for (int p0 = 0; p0 < n_pools; p0 += kPoolsPerLaunch) {
        PoolPtrs pp;
        const int m = n_pools - p0 < kPoolsPerLaunch ? n_pools - p0 : kPoolsPerLaunch;
        for (int i = 0; i < m; ++i) pp.p[i] = reinterpret_cast<unsigned char *>(pools[p0 + i]);
        const dim3 grid(copy_grid((long long)n * parts, m), m);
        st = cuda_check(launch(kv_copy_rows_kernel, grid, dim3(kCopyThreads), 0, (cudaStream_t)stream,
                               g_pdl, pp, (const int32_t *)L.b, (const int32_t *)L.c, (const int32_t *)L.c + n, n, Hkv,
                               cache->page_size, row_vecs, parts),
                        "i4_kv_pages_fork copy");
        if (st) return st;
    }
    return I4_OK;
}

extern "C" int i4_kv_pages_free(const i4_kv_cache *cache, const int32_t *seqs, int n, void *stream) {
    int st = check_cache("i4_kv_pages_free", cache);
    if (!st) st = check_list("i4_kv_pages_free", n, seqs, seqs);
    if (st || n == 0) return st;
    return cuda_check(launch(kv_free_kernel, dim3((n + 3) / 4), dim3(128), 0, (cudaStream_t)stream, g_pdl, cache_args(cache), seqs, n),
                      "i4_kv_pages_free");
}

extern "C" int i4_kv_pages_compact(const i4_kv_cache *cache, void *const *pools, int n_pools, int Hkv, int D, int32_t *n_live, void *ws,
                                   size_t ws_bytes, void *stream) {
    int st = check_cache("i4_kv_pages_compact", cache);
    if (!st) st = check_pools("i4_kv_pages_compact", pools, n_pools, cache->num_pages, Hkv, cache->page_size, D);
    if (!st) st = check_ws("i4_kv_pages_compact", ws, ws_bytes, cache->num_pages, cache->n_seqs);
    if (st) return st;
    const Lists L = ws_lists(ws, ws_cap(cache->num_pages, cache->n_seqs));
    st = cuda_check(launch(kv_compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, (cudaStream_t)stream, g_pdl, cache->refs,
                           cache->num_pages, n_live, L),
                    "i4_kv_pages_compact plan");
    if (st) return st;
    const CacheArgs args = cache_args(cache);
    return launch_copy(pools, n_pools, L.b, L.a, cache->num_pages, L.count, cache->num_pages,
                       (long long)Hkv * cache->page_size * D * 2, &args, L.c, (cudaStream_t)stream, "i4_kv_pages_compact");
}
