// Metadata of a ragged batch (chunked prefill, prompts, single tokens, in any mix), built on the
// device from the requests' lengths in one launch: the page table and int32 lengths that
// init_forward_metadata of the SGLang FlashMLA backend page (flashmla_backend.py) prepares, the
// offsets of the requests' rows (cu_seqlens), each new token's position and pool slot (the
// cache_loc of set_kv_buffer), with whole new pages taken from a free list when there is one, and
// the split plan of the ragged attention (chunk.cuh).
//
// With p_b cached tokens, n_b new ones and L_b = p_b + n_b:
//   cu[b] = sum_{j < b} n_j,  have_b = cdiv(p_b, 64),  need_b = cdiv(L_b, 64) - have_b,
//   off_b = sum_{j < b} need_j;
//   page(b, p) = req_to_token[row_b, 64 p] / 64 for p < have_b (and for every page without a free
//   list), free_pages[off_b + p - have_b] for have_b <= p < cdiv(L_b, 64);
//   token cu[b] + i: position p_b + i, slot 64 page(b, pos / 64) + pos % 64.
//
// Latency bounds it (a few KB to a few MB; 6.3 us for 64 single tokens, 8.3 us for 96 long chunks
// with 2 MB of maps, replayed in a graph).  Both prefix sums run over requests only, so every CTA
// computes them for itself in shared memory, instead of one CTA handing them to the others through
// a second launch or a grid-wide wait; then CTA 0 plans, and the others fill 1024 entries each of
// the table and of the token maps (a token finds its request by bisection in shared memory).
#pragma once
#include "ptx.cuh"

namespace mla {
namespace chunk {

constexpr int kMetaThreads = 256;
constexpr int kMetaMaxRequests = 4096;   // prefix sums of the whole batch in shared memory
constexpr int kMetaPerThread = 4;        // table or token entries per thread
constexpr int kMetaPerCta = kMetaThreads * kMetaPerThread;
constexpr int kTileRows = 128;           // query rows of an attention unit
constexpr int kTileKeys = 128;           // keys of an attention tile
// Cost model of the plan, in key tiles: a unit's (query tile's) fixed cost and the shortest piece
// (24 prompts of 16 heads / 64 single tokens / 2 short requests, us: 194.9 / 70.1 / 14.5 with a cost of 3;
// 210.6 / 69.4 / 18.6 with 1.5, 195.4 / 69.4 / 18.6 with 2, 204.9 / 72.7 / 14.5 with 4; long chunks within
// 2 %.  Pieces of 1 tile or more instead of 2: within 0.5 %; of 4: 192.7 / 73.4 / 14.5).
constexpr double kUnitCost = 3.0;
constexpr int kMinPiece = 2;

struct MetaParams {
    int32_t* req_to_token;
    int64_t r2t_rows, r2t_stride, r2t_cols;   // a row's pitch, and the columns of it that are the map's
    const void* rpi;
    const void* prefix_lens;
    const void* chunk_lens;
    int32_t bs, num_tokens, max_pages, num_heads;
    const void* free_pages;            // null: every slot is in req_to_token already
    int64_t num_free;
    int32_t causal, pad_slot, fill_tail, parts;
    int32_t* block_table;
    int64_t bt_stride;
    int32_t *cache_seqlens, *cu_seqlens, *positions, *cache_loc, *plan, *pages_taken;
    int32_t table_ctas;
};

// Last query row of row tile m of a request of `rows` rows (h per token): its token's causal limit
// bounds the tile's keys.  Shared by the plan and the attention kernel, which must agree.
__host__ __device__ __forceinline__ int unit_keys(int L, int n, int h, int m, int causal) {
    if (!causal) return L > 0 ? L : 0;
    // (n * h < 2^31: the callers' row counts are bounded so)
    const unsigned rows = (unsigned)n * (unsigned)h, end = ((unsigned)m + 1u) * kTileRows;
    const unsigned last = (end < rows ? end : rows) - 1u;
    const int64_t lim = (int64_t)L - n + (int)(last / (unsigned)h) + 1;
    return lim < L ? (lim > 0 ? (int)lim : 0) : (L > 0 ? L : 0);
}

// The plan's cost of the first m row tiles of a request: every tile costs kUnitCost plus its keys
// (the mean over the tile's rounding: the causal limit of row tile j is about p + 128 (j + 1) / h).
__device__ __forceinline__ double units_cost(double m, double p, double L, double inv_h, int causal) {
    return causal ? m * (kUnitCost + p * (1.0 / kTileKeys)) + 0.5 * m * (m + 1.0) * inv_h
                  : m * (kUnitCost + L * (1.0 / kTileKeys));
}

template <typename T>
__device__ __forceinline__ int64_t load_index(const void* p, int64_t i) {
    return static_cast<int64_t>(static_cast<const T*>(p)[i]);
}

struct MetaSmem {
    int32_t cu[kMetaMaxRequests + 1];    // rows before request b
    int32_t off[kMetaMaxRequests + 1];   // new pages before request b
    int32_t warp_n[kMetaThreads / 32], warp_p[kMetaThreads / 32];
    int64_t warp_c[kMetaThreads / 32];
    int64_t cost[kMetaThreads];          // plan: cost before each thread's requests
};

__device__ __forceinline__ int32_t sat_add(int32_t a, int32_t b, int32_t cap) {
    const int64_t s = (int64_t)a + b;
    return s > cap ? cap : (int32_t)s;
}

// A length, made safe: not negative, in 32 bits.
__device__ __forceinline__ int64_t safe_len(int64_t x) { return x < 0 ? 0 : (x > INT32_MAX ? INT32_MAX : x); }

// Lengths of a request that brings n tokens, made safe: no negative ones, positions past the table or
// past the columns of req_to_token have no page.
struct Req {
    int64_t row, p, L;
    int32_t have, total;   // pages holding cached tokens, pages holding all tokens
    int32_t n;
    bool row_ok, too_long;
};

template <typename IdxT, typename LenT>
__device__ __forceinline__ Req make_req(const MetaParams& a, int b, int32_t n) {
    Req r;
    r.row = load_index<IdxT>(a.rpi, b);
    const int64_t p = safe_len(load_index<LenT>(a.prefix_lens, b));
    r.p = p;
    r.n = n;
    r.L = p + n;
    int64_t cap = (int64_t)a.max_pages * 64;
    if (cap > a.r2t_cols) cap = a.r2t_cols;
    r.too_long = r.L > cap;
    const int64_t pc = p < cap ? p : cap, lc = r.L < cap ? r.L : cap;
    r.have = (int32_t)((pc + 63) / 64);
    r.total = (int32_t)((lc + 63) / 64);
    r.row_ok = r.row >= 0 && r.row < a.r2t_rows;
    return r;
}

// A request as it is after the sums: with the new tokens that have a row (all of them, where num_tokens
// holds the batch).
template <typename IdxT, typename LenT>
__device__ __forceinline__ Req load_req(const MetaParams& a, const MetaSmem& s, int b) {
    return make_req<IdxT, LenT>(a, b, s.cu[b + 1] - s.cu[b]);
}

template <typename IdxT, typename LenT>
__device__ __forceinline__ int32_t new_pages(const MetaParams& a, int b, int32_t n) {
    const Req r = make_req<IdxT, LenT>(a, b, n);
    return r.row_ok ? r.total - r.have : 0;
}

// Turn cu[b + 1] and off[b + 1] (of request b alone) into sums, saturating at `rows` rows and INT32_MAX
// pages, by the whole CTA.
__device__ __forceinline__ void sum_requests(int bs, int32_t rows, MetaSmem& s) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (bs + kMetaThreads - 1) / kMetaThreads;
    __syncthreads();
    const int lo = min(tid * per, bs), hi = min(lo + per, bs);
    int32_t n = 0, q = 0;
    for (int b = lo; b < hi; ++b) {
        n = sat_add(n, s.cu[b + 1], rows);
        q = sat_add(q, s.off[b + 1], INT32_MAX);
    }
    int32_t ni = n, qi = q;
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t tn = __shfl_up_sync(0xffffffffu, ni, d), tq = __shfl_up_sync(0xffffffffu, qi, d);
        if (lane >= d) {
            ni = sat_add(ni, tn, rows);
            qi = sat_add(qi, tq, INT32_MAX);
        }
    }
    if (lane == 31) {
        s.warp_n[warp] = ni;
        s.warp_p[warp] = qi;
    }
    __syncthreads();
    int32_t bn = 0, bq = 0;   // of the warps and lanes before this thread
    for (int w = 0; w < warp; ++w) {
        bn = sat_add(bn, s.warp_n[w], rows);
        bq = sat_add(bq, s.warp_p[w], INT32_MAX);
    }
    const int32_t en = __shfl_up_sync(0xffffffffu, ni, 1), eq = __shfl_up_sync(0xffffffffu, qi, 1);
    if (lane > 0) {
        bn = sat_add(bn, en, rows);
        bq = sat_add(bq, eq, INT32_MAX);
    }
    for (int b = lo; b < hi; ++b) {
        bn = sat_add(bn, s.cu[b + 1], rows);
        bq = sat_add(bq, s.off[b + 1], INT32_MAX);
        s.cu[b + 1] = bn;
        s.off[b + 1] = bq;
    }
    __syncthreads();
}

// Both prefix sums, by the whole CTA.  Where the batch has more new tokens than rows, what goes beyond
// counts nowhere: the lengths, the pages and the plan are those of the tokens that have a row.
template <typename IdxT, typename LenT>
__device__ __forceinline__ void scan_requests(const MetaParams& a, MetaSmem& s) {
    const int tid = threadIdx.x;
    if (tid == 0) s.cu[0] = s.off[0] = 0;
    // (a loop of one pass, or of two: a second copy of the sums would make every launch's code longer)
    for (bool cut = false;; cut = true) {
        for (int b = tid; b < a.bs; b += kMetaThreads) {
            const int32_t n = cut ? s.off[b + 1] : (int32_t)safe_len(load_index<LenT>(a.chunk_lens, b));
            s.cu[b + 1] = n;
            s.off[b + 1] = new_pages<IdxT, LenT>(a, b, n);
        }
        sum_requests(a.bs, cut ? a.num_tokens : a.num_tokens + 1, s);   // (num_tokens < 2^31 - 256)
        if (s.cu[a.bs] <= a.num_tokens) return;
        for (int b = tid; b < a.bs; b += kMetaThreads)
            s.off[b + 1] = min(s.cu[b + 1], a.num_tokens) - min(s.cu[b], a.num_tokens);
        __syncthreads();
    }
}

// Page of entry (b, p), p < total: from the free list or from req_to_token; -1 where there is none.
template <typename IdxT>
__device__ __forceinline__ int32_t page_of(const MetaParams& a, const Req& r, int32_t off, int32_t p, int& err) {
    if (a.free_pages && p >= r.have) {
        const int64_t i = (int64_t)off + (p - r.have);
        if (i >= a.num_free) {
            err |= 512 /* MLA_DEVERR_NO_FREE_PAGE */;
            return -1;
        }
        const int64_t page = load_index<IdxT>(a.free_pages, i);
        if (page < 0 || page > INT32_MAX / 64 - 1) {
            err |= 64 /* MLA_DEVERR_SLOT_INVALID */;
            return -1;
        }
        return (int32_t)page;
    }
    const int32_t slot = a.req_to_token[r.row * a.r2t_stride + (int64_t)p * 64];
    if (slot < 0 || (slot & 63) != 0) err |= 64;
    return slot >= 0 ? slot / 64 : -1;
}

// The split plan: the units (query row tiles of 128 rows, in order) laid end to end by cost, cut
// into `parts` ranges of equal cost; a range may begin or end inside a unit, at a key tile.  Row i
// of the plan = [begin request, row tile, key tile, end request, row tile, key tile, 0, 0], the
// end exclusive.  A thread a cut; the work does not grow with the tokens.
template <typename IdxT, typename LenT>
__device__ __forceinline__ void plan_chunks(const MetaParams& a, MetaSmem& s) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = a.num_heads;
    const double inv_h = 1.0 / h;
    auto len_of = [&](int b, int& n, int& L) {
        const Req r = load_req<IdxT, LenT>(a, s, b);
        n = r.n;
        const int64_t cap = (int64_t)a.max_pages * 64;
        L = (int)(r.L > INT32_MAX ? INT32_MAX : r.L);
        return cap;
    };
    // a request's cost in 1/256 key tiles: whole numbers, so that every thread agrees on the sums
    // and each cut falls into exactly one request
    auto request_cost = [&](int b) -> int64_t {
        int n, L;
        len_of(b, n, L);
        const int64_t mt = ((int64_t)n * h + kTileRows - 1) / kTileRows;
        return (int64_t)ceil(256.0 * units_cost((double)mt, L > n ? (double)(L - n) : 0.0, (double)L, inv_h, a.causal));
    };
    const int per = (a.bs + kMetaThreads - 1) / kMetaThreads;
    const int lo = min(tid * per, a.bs), hi = min(lo + per, a.bs);
    int64_t c = 0;
    for (int b = lo; b < hi; ++b) c += request_cost(b);
    int64_t ci = c;
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, ci, d);
        if (lane >= d) ci += t;
    }
    if (lane == 31) s.warp_c[warp] = ci;
    __syncthreads();
    int64_t total = 0, at = ci - c;   // at: the cost before this thread's requests
    for (int w = 0; w < kMetaThreads / 32; ++w) {
        if (w == warp) at += total;
        total += s.warp_c[w];
    }
    // no part shorter than its fixed cost and four tiles: few keys stay with few parts
    const int64_t share = (total + a.parts - 1) / a.parts, least = (int64_t)(256.0 * (kUnitCost + 4.0));
    const int64_t budget = share > least ? share : least;
    auto put = [&](int64_t i, int b, int m, int t) {   // cut i: the end of part i - 1 and the begin of part i
        if (i > 0) {
            int32_t* e = a.plan + 8 * (i - 1);
            e[3] = b;
            e[4] = m;
            e[5] = t;
            e[6] = 0;
            e[7] = 0;
        }
        if (i < a.parts) {
            int32_t* e = a.plan + 8 * i;
            e[0] = b;
            e[1] = m;
            e[2] = t;
        }
    };
    s.cost[tid] = at;
    __syncthreads();
    // A thread places one cut: bisection over the threads' costs, the requests of that thread, then
    // the row tiles by the closed form.
    for (int64_t i = tid; i < a.parts && i * budget < total; i += kMetaThreads) {
        const int64_t x64 = i * budget;
        int t0 = 0, t1 = kMetaThreads;   // the last thread whose cost is <= x64
        while (t1 - t0 > 1) {
            const int mid = (t0 + t1) >> 1;
            if (s.cost[mid] <= x64) t0 = mid; else t1 = mid;
        }
        int64_t c0 = s.cost[t0];
        int b = t0 * per;
        for (int64_t mine = request_cost(b); c0 + mine <= x64; mine = request_cost(b)) {   // x64 < total: it ends
            c0 += mine;
            ++b;
        }
        int n, L;
        const int64_t cap = len_of(b, n, L);
        const double p = L > n ? (double)(L - n) : 0.0;
        const int64_t mt = ((int64_t)n * h + kTileRows - 1) / kTileRows;
        const double x = (double)(x64 - c0) * (1.0 / 256.0);
        int64_t m0 = 0, m1 = mt;   // largest m with cost(m) <= x
        while (m1 - m0 > 1) {
            const int64_t mid = (m0 + m1) / 2;
            if (units_cost((double)mid, p, (double)L, inv_h, a.causal) <= x) m0 = mid; else m1 = mid;
        }
        int64_t keys = unit_keys(L, n, h, (int)m0, a.causal);
        if (keys > cap) keys = cap;
        const int64_t tiles = (keys + kTileKeys - 1) / kTileKeys;
        int64_t t = (int64_t)floor(x - units_cost((double)m0, p, (double)L, inv_h, a.causal) - kUnitCost);
        if (t < kMinPiece) t = 0;
        if (t > 0 && t + kMinPiece > tiles) {
            t = 0;
            ++m0;
        }
        if (m0 >= mt)
            put(i, b + 1, 0, 0);
        else
            put(i, b, (int)m0, (int)t);
    }
    // the cuts at and past the total cost
    for (int64_t i = (total + budget - 1) / budget + tid; i <= a.parts; i += kMetaThreads) put(i, a.bs, 0, 0);
}

template <typename IdxT, typename LenT>
__global__ void __launch_bounds__(kMetaThreads)
chunk_metadata_kernel(const __grid_constant__ MetaParams a) {
    // The attention grid, launched as a programmatic dependent, sets itself up meanwhile and waits
    // for this grid's completion before it reads anything.
    pdl_launch_dependents();
    __shared__ MetaSmem s;
    int err = 0;
    scan_requests<IdxT, LenT>(a, s);
    if (blockIdx.x == 0) {
        for (int b = threadIdx.x; b <= a.bs; b += kMetaThreads) {
            a.cu_seqlens[b] = s.cu[b];
            if (b == a.bs) break;
            const Req r = load_req<IdxT, LenT>(a, s, b);
            a.cache_seqlens[b] = (int32_t)(r.L > INT32_MAX ? INT32_MAX : r.L);
            if (!r.row_ok) err |= 2 /* MLA_DEVERR_ROW_OUT_OF_RANGE */;
            if (r.too_long) err |= 4 /* MLA_DEVERR_LEN_OUT_OF_RANGE */;
            if (safe_len(load_index<LenT>(a.chunk_lens, b)) > r.n) err |= 4;   // more rows than num_tokens
        }
        if (threadIdx.x == 0 && a.pages_taken) {
            const int64_t taken = s.off[a.bs];
            *a.pages_taken = (int32_t)(taken > a.num_free ? a.num_free : taken);
        }
        plan_chunks<IdxT, LenT>(a, s);
        if (err) raise_error(err);
        return;
    }
    const int cta = blockIdx.x - 1;
    if (cta < a.table_ctas) {
        const int64_t entries = (int64_t)a.bs * a.max_pages;
        const int64_t base = (int64_t)cta * kMetaPerCta + threadIdx.x;
#pragma unroll
        for (int k = 0; k < kMetaPerThread; ++k) {
            const int64_t idx = base + (int64_t)k * kMetaThreads;
            if (idx >= entries) break;
            const int b = (int)(idx / a.max_pages);
            const int32_t p = (int32_t)(idx - (int64_t)b * a.max_pages);
            const Req r = load_req<IdxT, LenT>(a, s, b);
            int32_t* dst = a.block_table + b * a.bt_stride + p;
            if (r.row_ok && p < r.total)
                *dst = page_of<IdxT>(a, r, s.off[b], p, err);
            else if (a.fill_tail)
                *dst = -1;
        }
    } else {
        const int64_t base = (int64_t)(cta - a.table_ctas) * kMetaPerCta + threadIdx.x;
        const int32_t rows = s.cu[a.bs];
#pragma unroll
        for (int k = 0; k < kMetaPerThread; ++k) {
            const int64_t t = base + (int64_t)k * kMetaThreads;
            if (t >= a.num_tokens) break;
            if (t >= rows) {
                if (a.fill_tail) {
                    a.positions[t] = 0;
                    a.cache_loc[t] = a.pad_slot;
                }
                continue;
            }
            int lo = 0, hi = a.bs;   // cu[lo] <= t < cu[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s.cu[mid] <= t) lo = mid; else hi = mid;
            }
            const int b = lo;
            const Req r = load_req<IdxT, LenT>(a, s, b);
            const int64_t pos = r.p + (t - s.cu[b]);
            int32_t slot = -1;
            if (r.row_ok && pos < (int64_t)r.total * 64 && pos < a.r2t_cols) {
                int32_t* where = a.req_to_token + r.row * a.r2t_stride + pos;
                if (a.free_pages) {
                    const int32_t page = page_of<IdxT>(a, r, s.off[b], (int32_t)(pos / 64), err);
                    if (page >= 0) {
                        slot = page * 64 + (int32_t)(pos % 64);
                        *where = slot;
                    }
                } else {
                    slot = *where;
                    if (slot < 0) {
                        err |= 64;
                        slot = -1;
                    }
                }
            }
            a.positions[t] = (int32_t)(pos > INT32_MAX ? INT32_MAX : pos);
            a.cache_loc[t] = slot;
        }
    }
    if (err) raise_error(err);
}

}  // namespace chunk
}  // namespace mla
