// Attention of ragged chunks of new tokens over the paged MLA cache for sm_100a: the queries of
// request b are rows [cu_seqlens[b], cu_seqlens[b + 1]) of q, any number of them (none, one, a
// prefill chunk, a whole prompt), and token i of n sees the keys j < L - n + i + 1 of the request's
// L cached rows (causal, its own row last), in the role of flash_mla_with_kvcache in the SGLang
// FlashMLA backend page (flashmla_backend.py, forward_extend) for new-token counts that differ.
//
// A unit is a tile of 128 query rows of one request (row = token * h + head, so one token of 128
// heads, or eight of 16): the rows share their keys, S = Q K^T and O = P V are dense contractions.
// One 2-CTA cluster per plan part walks the part's units (chunk_plan.cuh), computing with pair
// MMAs in the decode kernel's layout (decode.cuh: S split by tokens, O by output columns, the
// partner's V loaded into the chunks that S no longer needs).
//
//   * 16 warps a CTA, so that every stage has its own: two warps issue S and PV (neither waits
//     behind the other's barriers), eight run the softmax (32 keys of a row a thread), four bring Q
//     and write the result.  (Four softmax warps of 64 keys a thread and one issuer: 2,000 tokens at
//     32,768 keys took 16.7 ms instead of 16.0.)
//   * From one unit to the next nothing stands still that need not: the next unit's Q is half in
//     registers and half in shared memory when the last S MMA releases it (traced: 775 cycles from there to
//     Q in place; 3,500 as row-per-thread loads), its first S and softmax run while the Q warps write the
//     unit before, from row sums handed over in shared memory.
//   * A unit that lies whole in its part writes bf16 o and lse.  A part's first unit may continue
//     one that the part before began, its last may go on in the next: such pieces store fp32
//     partials in slot 2 part (continued) or 2 part + 1 (begun here), and chunk_merge_kernel joins
//     them.  At most two pieces per part, so the workspace does not grow with the batch, and no
//     piece waits for another.
//   * Rows of a page at or past L (never written) are cleared in shared memory before P V reads
//     them: P is 0 there, but 0 x NaN is not.
//
// What bounds it.  A tile of 128 keys is ~2,170 cycles of MMAs, and 328 KB through each CTA's shared memory
// (operands 208, pages in 104, P 16), 2,560 cycles; a two-slot page ring turns round in load 900 + S +
// softmax 2,000 + PV + signals, which leaves ~3,240 cycles a tile (bf16).  At that rate
// a long chunk runs into the power limit (1.44-1.72 GHz): 2,000 tokens of 128 heads at 32,768 keys take
// 15.8 ms (calls in a row), 1.19 PFLOP/s, 84 % of a sustained library GEMM.  An 8-bit cache adds the
// widening to every tile (~3,800 cycles, 0.83 PFLOP/s).  One token a request reads the cache once: 64
// requests of ~2,500 keys take 70 us replayed in a graph, 2.9 TB/s.  Separate rings for K groups and V
// pieces (V read twice) were slower: 136 KB into the SM per tile instead of 104, at ~57 bytes a cycle.
#pragma once
#include "chunk_plan.cuh"
#include "decode.cuh"

namespace mla {
namespace chunk {

using decode::kBox;
using decode::kChunk8;
using decode::kChunks;
using decode::kCtaRows;
using decode::kDqk;
using decode::kDv;
using decode::kIdescPV;
using decode::kIdescPV16;
using decode::kIdescQK;
using decode::kIdescQK16;
using decode::kKSlotBytes;
using decode::kKSlots;
using decode::kPage;
using decode::kPage8Bytes;
using decode::kPBytes;
using decode::kQHiBytes;
using decode::kQHiChunks;
using decode::kQLoChunks;
using decode::kQWarp0;
using decode::kRaw8Off;
using decode::kRescaleThreshold;
using decode::kTmemCols;
using decode::kTmemO;
using decode::kTmemQ;
using decode::kTmemS;
using decode::PageWindow;

constexpr int kThreads = 512;          // 16 warps: 0 K loads, 1 S issuer, 2 PV issuer (leader), 3 partner V
                                       // (8-bit cache: K of odd tiles), 4..7 and 12..15 softmax, 8..11 Q
                                       // and o (8-bit cache: and partner V)
constexpr int kSoftmaxWarps = 8;
constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
constexpr int kLoBoxes = kQLoChunks;   // a page's chunks 0..3 and 4..8 load, and free their slot, apart
constexpr int kHiBoxes = kChunks - kLoBoxes;

// Shared-memory map (offsets from the 1024-aligned base).
constexpr int kOffQ = 0;                            // Q chunks 4..8
constexpr int kOffK = kOffQ + kQHiBytes;
constexpr int kOffP = kOffK + kKSlots * kKSlotBytes;
constexpr int kOffX = kOffP + kPBytes + 2 * kBox;   // row-max exchange 2 x 256 floats; of two finished
                                                    // units each: row sums 256, row maxima 64
constexpr int kOffStage = kOffP + kPBytes;           // 16 KB: half of Q columns [0, 256) on its way to tensor
                                                    // memory, or o on its way out (4 warps x 4 KB)
constexpr int kUnitSums = 2 * kSoftmaxThreads, kUnitSumsStride = kSoftmaxThreads + kCtaRows;   // floats
constexpr int kOffPSig = kOffX + 5120;              // leader: landing words of the peer's signals
constexpr int kOffBar = kOffPSig + 256;             // words: P 0..7, V 8..11, K 12, 13, Q 14..17, S 18..25, O 26..29, Q high 30..33

enum : int {
    kBarKFull = 0,                      // leader (slot, half): both CTAs' chunks 0..3 / 4..8 landed
    kBarKEmpty = kBarKFull + 2 * kKSlots,    // both (slot, half): the PV MMAs finished with chunks 0..3 / all
    kBarQKDone = kBarKEmpty + 2 * kKSlots,   // both (slot): the tile's S MMAs finished reading the slot
    kBarVFull = kBarQKDone + kKSlots,   // leader (slot, half): the pair's partner V of output block 0 / 1 landed
    kBarQFull = kBarVFull + 2 * kKSlots,     // leader: Q columns [0, 256) in tensor memory
    kBarQHiFull,                        // leader: Q columns [256, 576) in shared memory
    kBarQLo,                            // local: a half of Q columns [0, 256) landed in the staging area
    kBarQHi,                            // local, 8-bit cache: Q columns [256, 576) landed as bf16
    kBarStage,                          // local: the 4 Q warps are done with the staging area's content
    kBarQEmpty,                         // both: the unit's last S MMA finished (Q reusable)
    kBarSFull,                          // both (x2): S tile in tensor memory
    kBarSFree = kBarSFull + 2,          // leader (x2): 16 softmax warps have read S
    kBarPFull = kBarSFree + 2,          // leader: 16 softmax warps wrote P
    kBarPvDone,                         // both: the PV MMAs of a tile finished (P reusable)
    kBarOFull,                          // both: the unit's last PV finished
    kBarOEmpty,                         // leader: 8 Q warps read O out
    kBarXchg,                           // local (x2): the 8 softmax warps posted row maxima
    kBarLx = kBarXchg + 2,              // local (x2): the 8 softmax warps posted a unit's row sums and maxima
    kBarVTail = kBarLx + 2,             // local: the partner V of a tile with a cut page landed
    kBarKRaw,                           // local (x2), 8-bit cache: this CTA's page landed
    kNumBars = kBarKRaw + kKSlots
};
constexpr int kOffMisc = kOffBar + kNumBars * 8;    // tensor-memory base, abort flag
constexpr int kSmemBytes = kOffMisc + 64 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");
static_assert(kOffK % 1024 == 0 && kOffP % 1024 == 0,
              "128-byte swizzle atoms need 1 KB alignment");
static_assert(kOffBar % 8 == 0, "mbarriers are 8 bytes");

// Partial results, two slots per part: fp32 rows [2 parts, 128, 512] and their lse [2 parts, 128].
__host__ __device__ constexpr size_t part_o_floats(int parts) { return (size_t)parts * 2 * kTileRows * kDv; }

struct Params {
    const uint8_t* kv;             // [num_pages * 64, 576]
    const int32_t* block_table;    // [bs, bt_stride]
    int64_t bt_stride;
    int32_t max_keys;              // positions the table has columns for (64 per column)
    const int32_t* cache_seqlens;  // [bs]
    const int32_t* cu;             // [bs + 1]
    const int32_t* plan;           // [parts, 8]
    int32_t bs, h, num_tokens;
    int64_t num_pages;
    float scale_log2;              // softmax_scale * log2(e)
    const float* descale_q;        // nullable
    const float* descale_k;        // nullable
    int32_t causal;
    __nv_bfloat16* out;            // [num_tokens * h, 512]
    float* lse;                    // [num_tokens * h]
    float* part_o;                 // [2 parts, 128, 512]
    float* part_lse;               // [2 parts, 128]
    uint64_t wait_budget_ns;       // budget of one pipeline wait
    int32_t withhold_tile;         // test hook: the leader's K load of this tile is not issued (-1: none)
};

// A unit, or the piece of it that lies in this part: request b, query rows row0 + [0, nrows) of q,
// key tiles [t0, t1), pages [2 t0, kb1); slot: where the piece's partial goes (-1: the whole unit).
struct Unit {
    int b, row_in_req, nrows, n, L, t0, t1, kb1, slot;
    int row0;   // first row in q / out
    __device__ int tiles() const { return t1 - t0; }
};

// Rows [c0, c1) of request b, whatever the caller's offsets hold.
__device__ __forceinline__ void request_rows(const int32_t* cu, int b, int num_tokens, int& c0, int& n) {
    c0 = cu[b];
    int c1 = cu[b + 1];
    c0 = c0 < 0 ? 0 : (c0 > num_tokens ? num_tokens : c0);
    c1 = c1 < c0 ? c0 : (c1 > num_tokens ? num_tokens : c1);
    n = c1 - c0;
}

// Keys of row tile m of a request that the table has columns for.  The merge kernel goes by it too: what
// is a piece, and what holds keys, follows from the call's lengths, which need not be the plan's.
__device__ __forceinline__ int table_keys(int L, int n, int h, int m, int causal, int max_keys) {
    return min(unit_keys(L, n, h, m, causal), max_keys);
}

// The units of a part, identical in every role.
struct UnitIter {
    int b, m, t, b1, m1, t1;
    int part;
    int cb, c0, n, L;   // rows and length of request cb, kept while its units follow one another
    __device__ bool next(const Params& p, Unit& u) {
        while (b < p.bs && (b < b1 || (b == b1 && (m < m1 || (m == m1 && t < t1))))) {
            if (cb != b) {
                request_rows(p.cu, b, p.num_tokens, c0, n);
                L = p.cache_seqlens[b];
                cb = b;
            }
            const int rows = n * p.h;
            if (m >= (rows + kTileRows - 1) / kTileRows) {
                ++b;
                m = t = 0;
                continue;
            }
            const int keys = table_keys(L, n, p.h, m, p.causal, p.max_keys);
            const int tiles = (keys + kTileKeys - 1) / kTileKeys;
            const int hi = (b == b1 && m == m1) ? min(t1, tiles) : tiles;
            const int lo = t;
            u.b = b;
            u.n = n;
            u.L = L;
            u.row_in_req = m * kTileRows;
            u.nrows = min(kTileRows, rows - m * kTileRows);
            u.row0 = c0 * p.h + m * kTileRows;
            u.t0 = lo;
            u.t1 = hi;
            u.kb1 = min(2 * hi, (keys + kPage - 1) / kPage);
            u.slot = lo > 0 ? 2 * part : (hi < tiles ? 2 * part + 1 : -1);
            ++m;
            t = 0;
            if (lo >= hi && lo > 0) continue;   // nothing left of a unit whose keys end before the cut
            return true;
        }
        return false;
    }
    // The next unit that has keys (the roles that only feed the MMAs skip the others).
    __device__ bool next_tiles(const Params& p, Unit& u) {
        while (next(p, u))
            if (u.tiles() > 0) return true;
        return false;
    }
};

__device__ __forceinline__ UnitIter make_iter(const Params& p, int part, bool& ok) {
    const int4 r0 = *reinterpret_cast<const int4*>(p.plan + 8 * (int64_t)part);
    const int2 r1 = *reinterpret_cast<const int2*>(p.plan + 8 * (int64_t)part + 4);
    UnitIter it;
    it.b = r0.x;
    it.m = r0.y;
    it.t = r0.z;
    it.b1 = r0.w;
    it.m1 = r1.x;
    it.t1 = r1.y;
    it.part = part;
    it.cb = -1;
    it.c0 = it.n = it.L = 0;
    ok = it.b >= 0 && it.b <= it.b1 && it.b1 <= p.bs && it.m >= 0 && it.t >= 0 && it.m1 >= 0 && it.t1 >= 0;
    if (!ok) it.b = p.bs;   // no units
    return it;
}

// Widen one 8-bit chunk as decode::widen_chunk_fp8 does, rows at or past `valid` as zeros.
template <bool kE5M2>
__device__ __forceinline__ void widen_chunk_rows(uint32_t src, uint32_t dst, int lane, int valid) {
    uint4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v[j] = ld_shared_v4u(src + 16u * (uint32_t)(lane + 32 * j));
        if (((lane + 32 * j) >> 2) >= valid) v[j] = make_uint4(0, 0, 0, 0);
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int x = lane + 32 * j;        // row x / 4, 16-value quarter x % 4
        const uint32_t t = (uint32_t)(x >> 2), q = (uint32_t)(x & 3);
        const uint32_t row = dst + 128u * t;
        st_shared_v4u(row + 16u * ((2u * q) ^ (t & 7u)), fp8x2_to_f16x2<kE5M2>(v[j].x), fp8x2_to_f16x2<kE5M2>(v[j].x >> 16),
                      fp8x2_to_f16x2<kE5M2>(v[j].y), fp8x2_to_f16x2<kE5M2>(v[j].y >> 16));
        st_shared_v4u(row + 16u * ((2u * q + 1u) ^ (t & 7u)), fp8x2_to_f16x2<kE5M2>(v[j].z),
                      fp8x2_to_f16x2<kE5M2>(v[j].z >> 16), fp8x2_to_f16x2<kE5M2>(v[j].w), fp8x2_to_f16x2<kE5M2>(v[j].w >> 16));
    }
    __syncwarp();
}

// Clear rows [valid, 64) of the four V chunks at slot positions 4n + c, + 1 (n = 0, 1): a lane a 16-byte
// unit of every row.
__device__ __forceinline__ void clear_v_rows(uint32_t slot, int c, int valid, int lane) {
    const int pos = 4 * (lane >> 4) + c + ((lane >> 3) & 1);
    const uint32_t unit = slot + (uint32_t)(pos * kBox + 16 * (lane & 7));
    for (int row = max(valid, 0); row < kPage; ++row) st_shared_v4u(unit + 128u * (uint32_t)row, 0u, 0u, 0u, 0u);
}

// kKv: the cache's element type, 0 bf16, 1 e4m3, 2 e5m2 (8-bit caches are widened to f16).
template <int kKv>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
mla_chunk_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap klo_map,
                 const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap q_map,
                 const __grid_constant__ CUtensorMap qlo_map, const __grid_constant__ Params p) {
    constexpr bool kFp8 = kKv != 0;
    constexpr bool kE5M2 = kKv == 2;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) -> uint32_t { return sbase + kOffBar + 8u * i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);   // warp-uniform to the compiler
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int part = blockIdx.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kKSlots; ++s) {
            for (int j = 0; j < 2; ++j) {
                mbar_init(bar(kBarKFull + 2 * s + j), 1);
                mbar_init(bar(kBarKEmpty + 2 * s + j), 1);
                mbar_init(bar(kBarVFull + 2 * s + j), kFp8 ? 4 : 1);
            }
            mbar_init(bar(kBarQKDone + s), 1);
            mbar_init(bar(kBarKRaw + s), 1);
        }
        mbar_init(bar(kBarQFull), 4);
        mbar_init(bar(kBarQHiFull), kFp8 ? 4 : 1);
        mbar_init(bar(kBarQLo), 1);
        mbar_init(bar(kBarQHi), 1);
        mbar_init(bar(kBarStage), 4);
        mbar_init(bar(kBarQEmpty), 1);
        for (int j = 0; j < 2; ++j) {
            mbar_init(bar(kBarSFull + j), 1);
            mbar_init(bar(kBarSFree + j), kSoftmaxWarps);
            mbar_init(bar(kBarXchg + j), kSoftmaxWarps);
            mbar_init(bar(kBarLx + j), kSoftmaxWarps);
        }
        mbar_init(bar(kBarPFull), kSoftmaxWarps);
        mbar_init(bar(kBarPvDone), 1);
        mbar_init(bar(kBarOFull), 1);
        mbar_init(bar(kBarOEmpty), 4);
        mbar_init(bar(kBarVTail), 1);
        *abort_flag = 0;
        fence_mbarrier_init_cluster();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish_pair();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&k_map);
        prefetch_tensormap(&klo_map);
        prefetch_tensormap(&v_map);
        prefetch_tensormap(&q_map);
        prefetch_tensormap(&qlo_map);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    // Set up without reading anything another grid writes; from here on everything may be read, and
    // the merge kernel, which reads the plan before its own wait, may be let in.
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    bool plan_ok = true;
    UnitIter iter = make_iter(p, part, plan_ok);
    const uint32_t tmem = *tmem_slot;
    const AbortCtl actl{abort_flag, map_to_cta(smem_u32(tmem_slot + 1), rank ^ 1u), p.wait_budget_ns};
    if (!plan_ok && threadIdx.x == 0) raise_error(8 /* MLA_DEVERR_BAD_METADATA */);

    // A warp reporting to the leader's MMA issuer: the leader's warp arrives with expect_tx of 4
    // bytes, the peer's warp sends a 4-byte st.async whose complete_tx lands on the leader's barrier.
    auto signal_leader = [&](int b_idx, int word) {
        __syncwarp();
        if (lane == 0) {
            if (leader)
                mbar_arrive_expect_tx(bar(b_idx), 4);
            else
                st_async_b32(map_to_cta(sbase + kOffPSig + 4u * (uint32_t)word, 0), 0u,
                             map_to_cta(bar(b_idx), 0));
        }
    };
    // let copies already issued land before shared memory can go away
    auto drain_on_abort = [&]() {
        if (lane == 0 && *abort_flag) {
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 200000ull) {
            }
        }
    };

    if (warp == 0 || (kFp8 && warp == 3)) {
        // ------------------------------------------------------------ K loads
        // (8-bit cache: two warps take alternate tiles, and widen them)
        const uint32_t mine = warp == 3 ? 1u : 0u;
        uint32_t g = 0;
        bool alive = true;
        Unit u;
        while (alive && iter.next_tiles(p, u)) {
            const int n = u.tiles();
            PageWindow pw;
            pw.init(p.block_table + (int64_t)u.b * p.bt_stride, 2 * u.t0, u.kb1, lane, p.num_pages, warp == 0);
            for (int i = 0; i < n; ++i, ++g) {
                const int blk = 2 * (u.t0 + i) + (int)rank;
                const int32_t row = pw.row(blk);
                if (kFp8 && (g & 1u) != mine) continue;
                int ok = 1;
                const int s = (int)(g & 1u);
                const uint32_t slot = sbase + kOffK + s * kKSlotBytes;
                const bool withhold = leader && (int)g == p.withhold_tile;
                if (lane == 0) {
                    const uint32_t free = ((g >> 1) & 1u) ^ 1u;
                    if constexpr (kFp8) {
                        // the raw page lies in the slot's back half
                        ok = mbar_wait_bounded(bar(kBarKEmpty + 2 * s + 1), free, actl);
                        if (ok && !withhold) {
                            mbar_arrive_expect_tx(bar(kBarKRaw + s), kPage8Bytes);
                            tma_load_3d(slot + kRaw8Off, &k_map, bar(kBarKRaw + s), 0, row, 0);
                        }
                    } else {
                        ok = mbar_wait_bounded(bar(kBarKEmpty + 2 * s), free, actl);
                        if (ok && !withhold) {
                            const uint32_t kf = bar(kBarKFull + 2 * s);
                            if (leader) mbar_arrive_expect_tx(kf, 2 * kLoBoxes * kBox);
                            tma_load_3d_pair(slot, &klo_map, map_to_cta(kf, 0), 0, row, 0);
                        }
                        ok = ok && mbar_wait_bounded(bar(kBarKEmpty + 2 * s + 1), free, actl);
                        if (ok && !withhold) {
                            const uint32_t kf = bar(kBarKFull + 2 * s + 1);
                            if (leader) mbar_arrive_expect_tx(kf, 2 * kHiBoxes * kBox);
                            tma_load_3d_pair(slot + kLoBoxes * kBox, &k_map, map_to_cta(kf, 0), 0, row, kLoBoxes);
                        }
                    }
                }
                if (!__shfl_sync(0xffffffffu, ok, 0)) {
                    alive = false;
                    break;
                }
                if constexpr (kFp8) {
                    const bool landed = mbar_wait_bounded(bar(kBarKRaw + s), (g >> 1) & 1u, actl);
                    if (!__all_sync(0xffffffffu, landed)) {
                        alive = false;
                        break;
                    }
                    const int valid = u.L - blk * kPage;
#pragma unroll 1
                    for (int c = 0; c < kChunks; ++c) {
                        widen_chunk_rows<kE5M2>(slot + kRaw8Off + c * kChunk8, slot + c * kBox, lane, valid);
                        if (c == kLoBoxes - 1 || c == kChunks - 1) {
                            fence_proxy_async_smem();
                            signal_leader(kBarKFull + 2 * s + (c == kChunks - 1), 12 + (c == kChunks - 1));
                        }
                    }
                }
            }
        }
        drain_on_abort();
    } else if (!kFp8 && warp == 3) {
        // ------------------------------------------------------------ partner V (bf16 cache)
        // Two 16 KB loads of the partner's page once the tile's S MMAs are done.  A tile whose pages
        // reach past L: the rows there are cleared, in this CTA's own V chunks and in the partner's
        // once they landed, before the leader is told.
        uint32_t g = 0, ntail = 0;
        bool alive = true;
        Unit u;
        while (alive && iter.next_tiles(p, u)) {
            const int n = u.tiles();
            PageWindow pw;
            pw.init(p.block_table + (int64_t)u.b * p.bt_stride, 2 * u.t0, u.kb1, lane, p.num_pages, false);
            for (int i = 0; i < n; ++i, ++g) {
                const int blk = 2 * (u.t0 + i) + 1 - (int)rank;
                const int32_t row = pw.row(blk);
                const int s = (int)(g & 1u);
                const uint32_t slot = sbase + kOffK + s * kKSlotBytes;
                const int own_valid = u.L - (blk ^ 1) * kPage, valid = u.L - blk * kPage;
                const bool cut = (own_valid < kPage && (blk ^ 1) < u.kb1) || (valid < kPage && blk < u.kb1);
                int ok = 1;
                if (lane == 0) {
                    ok = mbar_wait_bounded(bar(kBarQKDone + s), (g >> 1) & 1u, actl);
                    if (ok) {
                        if (cut) mbar_arrive_expect_tx(bar(kBarVTail), 2 * 2 * kBox);
#pragma unroll
                        for (int nn = 0; nn < 2; ++nn) {
                            const uint32_t vf = bar(kBarVFull + 2 * s + nn);
                            if (!cut && leader) mbar_arrive_expect_tx(vf, 2 * 2 * kBox);
                            const uint32_t dst = slot + (4 * nn + 2 * (1 - (int)rank)) * kBox;
                            if (cut)
                                tma_load_3d(dst, &v_map, bar(kBarVTail), 0, row, 4 * nn + 2 * (int)rank);
                            else
                                tma_load_3d_pair(dst, &v_map, map_to_cta(vf, 0), 0, row, 4 * nn + 2 * (int)rank);
                        }
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (ok && cut) {
                    if (own_valid < kPage) clear_v_rows(slot, 2 * (int)rank, own_valid, lane);
                    const bool landed = mbar_wait_bounded(bar(kBarVTail), ntail & 1u, actl);
                    ok = __all_sync(0xffffffffu, landed);
                    if (valid < kPage) clear_v_rows(slot, 2 * (1 - (int)rank), valid, lane);
                    fence_proxy_async_smem();
                    signal_leader(kBarVFull + 2 * s, 8);
                    signal_leader(kBarVFull + 2 * s + 1, 9);
                    ++ntail;
                }
                if (!ok) {
                    alive = false;
                    break;
                }
            }
        }
        drain_on_abort();
    } else if (warp >= kQWarp0 && warp < kQWarp0 + 4) {
        // ------------------------------------------------------------ Q, o (8-bit cache: and partner V)
        // These warps bring a unit's Q, then write the result of the unit before while the softmax
        // warps are at the new unit's first tile already.  Q columns [0, 256) pass through the staging
        // area in two halves (a TMA load each, then shared -> registers -> tensor memory): by the time
        // the unit before is done with Q, the first half is in registers and the second has landed.
        const int quarter = warp & 3;
        const int qt = threadIdx.x - kQWarp0 * 32;          // 0..127
        const int rloc = (32 * quarter + lane) & 63;
        const int rtile = kCtaRows * (int)rank + rloc;      // row of the unit's tile
        const uint32_t lane_off = (uint32_t)(32 * quarter) << 16;
        const int half = quarter >> 1;                      // lanes of O's columns [0, 128) / [128, 256) of a block
        const float dk = p.descale_k ? *p.descale_k : 1.0f;
        const float* xmax = reinterpret_cast<const float*>(smem + kOffX);
        const uint32_t stage = sbase + kOffStage;
        const bool issuer = quarter == 3 && lane == 0;
        uint32_t uq = 0, g = 0, ue = 0, nstage = 0;   // nstage: phases of kBarStage, three a unit
        bool alive = true;
        uint32_t q_top = 0;   // 8-bit cache: largest magnitudes of q (bf16 pairs)
        Unit u, done;
        done.slot = done.row0 = done.nrows = 0;
        auto all = [](bool ok) -> bool { return __all_sync(0xffffffffu, ok); };
        // this warp is done with the staging area's content (1 of 4); the issuer goes on once all are.
        // The fence holds back the arrival until the warp's loads have their data: the next TMA load
        // would overwrite it (without the fence single units of Q came out as the next half's).
        auto stage_read = [&]() -> bool {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarStage));
            bool ok = true;
            if (issuer) ok = mbar_wait_bounded(bar(kBarStage), nstage & 1u, actl);
            ++nstage;
            return all(ok);
        };
        auto q_load = [&](const Unit& v, int hb) {   // (issuer)
            mbar_arrive_expect_tx(bar(kBarQLo), 2 * kBox);
            tma_load_3d(stage, &qlo_map, bar(kBarQLo), 0, v.row0 + kCtaRows * (int)rank, 2 * hb);
        };
        // bf16 -> f16, keeping the largest magnitude of the unit's rows (past 65504 f16 has no value;
        // below it only magnitudes under 2^-17 round, by 2^-25 at most)
        auto q_to_f16 = [&](uint4& x, bool row) {
            uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (row) q_top = __vmaxu2(q_top, w[k] & 0x7FFF7FFFu);
                w[k] = pack_f16x2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
            }
            x = make_uint4(w[0], w[1], w[2], w[3]);
        };
        // the row's 128 columns in the staging area (rows past the unit's last are other rows, or
        // zeros past q: computed, never stored)
        auto q_read = [&](uint4 (&v)[16]) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                v[k] = ld_shared_v4u(stage + (uint32_t)((k >> 3) * kBox + rloc * 128) + 16u * (((uint32_t)k & 7u) ^ ((uint32_t)rloc & 7u)));
                if constexpr (kFp8) {
                    q_to_f16(v[k], rtile < u.nrows);
                }
            }
        };
        auto q_write = [&](const uint4 (&v)[16], int hb) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t w[16];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    w[4 * k] = v[4 * c + k].x;
                    w[4 * k + 1] = v[4 * c + k].y;
                    w[4 * k + 2] = v[4 * c + k].z;
                    w[4 * k + 3] = v[4 * c + k].w;
                }
                tmem_st16(tmem + lane_off + kTmemQ + 64u * hb + 16u * c, w);
            }
        };
        // o (or the piece's fp32 partial, normalised) and lse of unit `done`: 64 tensor-memory columns
        // a step, 128 bytes of each of the warp's 32 rows a pass (bf16: one pass, fp32: two), turned in
        // 4 KB of the staging area (16-byte unit k of row r at k ^ (r & 7)) so that 8 lanes write a
        // whole line.  (A unit's 64 KB in 32-column steps: ~4,400 cycles as 32-byte stores straight
        // from the registers, one line each; ~5,200 as TMA boxes of 2 KB, two in flight a warp.)
        auto epilogue = [&]() -> bool {
            const bool full = mbar_wait_bounded(bar(kBarOFull), ue & 1u, actl);
            const bool sums = mbar_wait_bounded(bar(kBarLx + (ue & 1u)), (ue >> 1) & 1u, actl);
            if (!all(full && sums)) return false;
            tc_fence_after();
            const float* x = xmax + kUnitSums + (ue & 1u) * kUnitSumsStride + rloc;
            const float l_run = (x[0] + x[64]) + (x[128] + x[192]);
            const float m_run = x[kSoftmaxThreads];
            // (0: no key; a NaN goes on into o and lse)
            const float inv = l_run != 0.f ? dk / l_run : 0.f;
            const float lse_val = l_run != 0.f ? (m_run + __log2f(l_run)) * 0.69314718055994531f : -INFINITY;
            const bool direct = done.slot < 0;
            const int r0 = kCtaRows * (int)rank + 32 * (quarter & 1);   // the warp's first row
            const int rows = direct ? min(32, done.nrows - r0) : 32;    // rows to write (<= 0: none)
            const uint32_t buf = stage + 4096u * (uint32_t)quarter;
            const int rsub = lane >> 3, unit = lane & 7;                // store: row 4 j + rsub, 16-byte unit
            uint8_t* const dst = direct ? reinterpret_cast<uint8_t*>(p.out + ((int64_t)done.row0 + r0) * kDv)
                                        : reinterpret_cast<uint8_t*>(p.part_o + ((int64_t)done.slot * kTileRows + r0) * kDv);
            const int esize = direct ? 2 : 4;
            const int nst = direct ? 4 : 8;   // passes of 128 bytes a row: 64 bf16 columns, or 32 fp32
#pragma unroll 1
            for (int st = 0; st < nst; ++st) {
                const int c0 = direct ? 64 * st : 32 * st;   // tensor-memory column
                __syncwarp();   // the pass before has been read
#pragma unroll
                for (int hp = 0; hp < 2; ++hp) {
                    if (!direct && hp == 1) break;
                    uint32_t raw[32];
                    tmem_ld16(tmem + lane_off + kTmemO + (uint32_t)(c0 + 32 * hp), *reinterpret_cast<uint32_t(*)[16]>(raw));
                    tmem_ld16(tmem + lane_off + kTmemO + (uint32_t)(c0 + 32 * hp) + 16u, *reinterpret_cast<uint32_t(*)[16]>(raw + 16));
                    tc_wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; ++k) raw[k] = __float_as_uint(__uint_as_float(raw[k]) * inv);
                    if (direct) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) raw[k] = pack_bf16x2(__uint_as_float(raw[2 * k]), __uint_as_float(raw[2 * k + 1]));
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (direct && k >= 4) break;
                        const uint32_t unit_at = (uint32_t)(k + 4 * hp) ^ ((uint32_t)lane & 7u);
                        st_shared_v4u(buf + 128u * (uint32_t)lane + 16u * unit_at, raw[4 * k], raw[4 * k + 1], raw[4 * k + 2], raw[4 * k + 3]);
                    }
                }
                if (st == nst - 1) {
                    tc_fence_before();
                    signal_leader(kBarOEmpty, 26 + quarter);   // O is free for the next unit
                }
                __syncwarp();
                const int col = 256 * (c0 >> 7) + 128 * half + (c0 & 127);
                // (rows behind the unit's last belong to another request or to nobody)
#pragma unroll
                for (int j4 = 0; j4 < 8; j4 += 4) {
                    uint4 v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[j] = ld_shared_v4u(buf + 128u * (uint32_t)(4 * (j4 + j) + rsub) +
                                             16u * ((uint32_t)unit ^ ((uint32_t)(4 * (j4 + j) + rsub) & 7u)));
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (4 * (j4 + j) + rsub < rows)
                            *reinterpret_cast<uint4*>(dst + ((int64_t)(4 * (j4 + j) + rsub) * kDv + col) * esize + 16 * unit) = v[j];
                }
            }
            if (half == 0) {
                if (!direct)
                    p.part_lse[(int64_t)done.slot * kTileRows + rtile] = lse_val;
                else if (rtile < done.nrows)
                    p.lse[(int64_t)done.row0 + rtile] = lse_val;
            }
            ++ue;
            return true;
        };
        bool more = iter.next_tiles(p, u);
        if (more && issuer) q_load(u, 0);
        while (more) {
            // ---- Q of the unit
            uint4 v[16];
            if (!all(mbar_wait_bounded(bar(kBarQLo), 0u, actl))) break;
            q_read(v);
            if (!stage_read()) break;
            if (issuer) q_load(u, 1);
            if (!all(uq == 0 || mbar_wait_bounded(bar(kBarQEmpty), (uq - 1) & 1u, actl))) break;
            tc_fence_after();
            if (issuer) {   // columns [256, 576): where S reads them (8-bit cache: converted in place first)
                if constexpr (kFp8) {
                    mbar_arrive_expect_tx(bar(kBarQHi), kQHiBytes);
                    tma_load_3d(sbase + kOffQ, &q_map, bar(kBarQHi), 0, u.row0 + kCtaRows * (int)rank, kQLoChunks);
                } else {
                    if (leader) mbar_arrive_expect_tx(bar(kBarQHiFull), 2 * kQHiBytes);
                    tma_load_3d_pair(sbase + kOffQ, &q_map, map_to_cta(bar(kBarQHiFull), 0), 0,
                                     u.row0 + kCtaRows * (int)rank, kQLoChunks);
                }
            }
            __syncwarp();
            q_write(v, 0);
            if (!all(mbar_wait_bounded(bar(kBarQLo), 1u, actl))) break;
            q_read(v);
            if (!stage_read()) break;
            q_write(v, 1);
            tc_wait_st();
            tc_fence_before();
            signal_leader(kBarQFull, 14 + quarter);
            if constexpr (kFp8) {
                if (!all(mbar_wait_bounded(bar(kBarQHi), uq & 1u, actl))) break;
                // bf16 -> f16 in place: 16-byte unit qt + 128 j of the 64 rows x 5 chunks x 8 units
#pragma unroll 4
                for (int j = 0; j < 20; ++j) {
                    const uint32_t at = sbase + kOffQ + 16u * (uint32_t)(qt + 128 * j);
                    uint4 x = ld_shared_v4u(at);
                    q_to_f16(x, kCtaRows * (int)rank + (((qt + 128 * j) >> 3) & 63) < u.nrows);
                    st_shared_v4u(at, x.x, x.y, x.z, x.w);
                }
                fence_proxy_async_smem();
                signal_leader(kBarQHiFull, 30 + quarter);
                // (0x477F: the largest bf16 below 65504; infinities and NaN lie above, too)
                const bool range = (q_top & 0xFFFFu) > 0x477Fu || (q_top >> 16) > 0x477Fu;
                if (__any_sync(0xffffffffu, range) && lane == 0) raise_error(32 /* MLA_DEVERR_Q_RANGE */);
                __syncwarp();
            }
            // ---- the unit before: its result
            if (!all(mbar_wait_bounded(bar(kBarStage), (nstage - 1) & 1u, actl))) break;   // every warp has read its Q
            if (uq > 0 && !epilogue()) break;
            done = u;
            ++uq;
            const Unit cur = u;
            more = iter.next_tiles(p, u);
            if (!stage_read()) break;
            if (more && issuer) q_load(u, 0);
            if constexpr (kFp8) {
                // ---- partner V of each tile: 4 chunks x 64 rows x 4 sixteen-byte units of 8-bit
                // values, 8 per thread, widened to f16 on the way into the slot once the tile's S
                // MMAs are done, rows at or past L as zeros
                const int32_t* bt_row = p.block_table + (int64_t)cur.b * p.bt_stride;
                for (int i = 0; i < cur.tiles(); ++i, ++g) {
                    const int blk = 2 * (cur.t0 + i) + 1 - (int)rank;
                    int pg = blk < cur.kb1 ? __ldg(bt_row + blk) : -1;
                    if (pg < 0 || (int64_t)pg >= p.num_pages) pg = -1;   // reported by the K loads
                    const int s = (int)(g & 1u);
                    const uint32_t slot = sbase + kOffK + s * kKSlotBytes;
                    const int valid = cur.L - blk * kPage;
                    uint4 w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int x = qt + 128 * j, hh = x >> 8, row = (x >> 2) & 63, q4 = x & 3;
                        const int chunk = 4 * (hh >> 1) + 2 * (int)rank + (hh & 1);
                        w[j] = pg >= 0 && row < valid ? __ldg(reinterpret_cast<const uint4*>(
                                             p.kv + ((int64_t)pg * kPage + row) * kDqk + chunk * 64 + q4 * 16))
                                       : make_uint4(0, 0, 0, 0);
                    }
                    const bool s_done = mbar_wait_bounded(bar(kBarQKDone + s), (g >> 1) & 1u, actl);
                    if (!__all_sync(0xffffffffu, s_done)) {
                        alive = more = false;
                        break;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int x = qt + 128 * j, hh = x >> 8, row = (x >> 2) & 63, q4 = x & 3;
                        const int pos = 4 * (hh >> 1) + 2 * (1 - (int)rank) + (hh & 1);
                        const uint32_t r = slot + pos * kBox + row * 128;
                        const uint32_t sw = (uint32_t)row & 7u;
                        st_shared_v4u(r + 16u * ((2u * q4) ^ sw), fp8x2_to_f16x2<kE5M2>(w[j].x),
                                      fp8x2_to_f16x2<kE5M2>(w[j].x >> 16), fp8x2_to_f16x2<kE5M2>(w[j].y),
                                      fp8x2_to_f16x2<kE5M2>(w[j].y >> 16));
                        st_shared_v4u(r + 16u * ((2u * q4 + 1u) ^ sw), fp8x2_to_f16x2<kE5M2>(w[j].z),
                                      fp8x2_to_f16x2<kE5M2>(w[j].z >> 16), fp8x2_to_f16x2<kE5M2>(w[j].w),
                                      fp8x2_to_f16x2<kE5M2>(w[j].w >> 16));
                        if (j == 3 || j == 7) {   // an output block's two chunks are in place
                            fence_proxy_async_smem();
                            signal_leader(kBarVFull + 2 * s + (j >> 2), 8 + quarter);
                        }
                    }
                }
            }
        }
        if (alive && ue < uq) epilogue();
        drain_on_abort();
    } else if (warp == 1) {
        // ------------------------------------------------------------ S issuer (leader)
        // A warp each for S and PV, so that neither waits behind the other's barriers; the whole
        // warp walks the tiles, an elected lane issues each MMA.
        if (leader) {
            uint32_t g = 0, uq = 0;
            bool alive = true;
            auto wait = [&](int b, uint32_t parity) -> bool {
                return __all_sync(0xffffffffu, mbar_wait_bounded(bar(b), parity, actl));
            };
            Unit u;
            while (alive && iter.next_tiles(p, u)) {
                const int n = u.tiles();
                if (!wait(kBarQFull, uq & 1u)) break;
                for (int i = 0; i < n; ++i, ++g) {
                    const int s = (int)(g & 1u);
                    const uint32_t slot = sbase + kOffK + s * kKSlotBytes;
                    const uint32_t d = tmem + kTmemS + 64u * (g & 1u);
                    if ((g >= 2 && !wait(kBarSFree + s, ((g >> 1) & 1u) ^ 1u)) || !wait(kBarKFull + 2 * s, (g >> 1) & 1u)) {
                        alive = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < kQLoChunks; ++c)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_pair_ts(d, tmem + kTmemQ + 32u * c + 8u * kk, smem_desc_sw128(slot + c * kBox + 32u * kk, 16, 1024),
                                        kFp8 ? kIdescQK16 : kIdescQK, (c | kk) ? 1u : 0u);
                    if ((i == 0 && !wait(kBarQHiFull, uq & 1u)) || !wait(kBarKFull + 2 * s + 1, (g >> 1) & 1u)) {
                        alive = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int c = kQLoChunks; c < kChunks; ++c)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_pair_ss(d, smem_desc_sw128(sbase + kOffQ + (c - kQLoChunks) * kBox + 32u * kk, 16, 1024),
                                        smem_desc_sw128(slot + c * kBox + 32u * kk, 16, 1024), kFp8 ? kIdescQK16 : kIdescQK, 1u);
                    tc_commit_pair(bar(kBarQKDone + s));
                    tc_commit_pair(bar(kBarSFull + s));
                    if (i == n - 1) tc_commit_pair(bar(kBarQEmpty));
                }
                ++uq;
            }
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ PV issuer (leader)
        // Output block 0 (slot chunks 0..3) before block 1 (4..7): each half of the slot goes back to
        // the K loads as soon as its block is done.
        if (leader) {
            uint32_t g = 0, uq = 0;
            bool alive = true;
            auto wait = [&](int b, uint32_t parity) -> bool {
                return __all_sync(0xffffffffu, mbar_wait_bounded(bar(b), parity, actl));
            };
            Unit u;
            while (alive && iter.next_tiles(p, u)) {
                const int n = u.tiles();
                if (uq > 0 && !wait(kBarOEmpty, (uq - 1) & 1u)) break;
                for (int i = 0; i < n; ++i, ++g) {
                    const int s = (int)(g & 1u);
                    const uint32_t slot = sbase + kOffK + s * kKSlotBytes;
                    if (!wait(kBarPFull, g & 1u)) {
                        alive = false;
                        break;
                    }
#pragma unroll
                    for (int nn = 0; nn < 2; ++nn) {
                        if (!wait(kBarVFull + 2 * s + nn, (g >> 1) & 1u)) {
                            alive = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll
                        for (int pp = 0; pp < 2; ++pp)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_pair_ss(tmem + kTmemO + 128u * nn,
                                            smem_desc_sw128(sbase + kOffP + pp * kBox + 32u * kk, 16, 1024),
                                            smem_desc_sw128(slot + (4 * nn + 2 * pp) * kBox + 2048u * kk, kBox, 1024),
                                            kFp8 ? kIdescPV16 : kIdescPV, (i == 0 && pp == 0 && kk == 0) ? 0u : 1u);
                        tc_commit_pair(bar(kBarKEmpty + 2 * s + nn));
                    }
                    if (!alive) break;
                    tc_commit_pair(bar(kBarPvDone));
                    if (i == n - 1) tc_commit_pair(bar(kBarOFull));
                }
                ++uq;
            }
        }
    } else {
        // ------------------------------------------------------------ softmax / epilogue
        // Two warps per tensor-memory lane quarter (4..7 and 12..15): a thread has 32 of a row's 128
        // keys, and 128 of its CTA row's 256 tensor-memory columns of O.
        const int quarter = warp & 3, sub = warp >> 3;
        const int t = 32 * quarter + lane;                    // TMEM lane
        const int rloc = t & 63;                              // row within this CTA's 64
        const int half = t >> 6;                              // key half (page) of each tile
        const int sw8 = quarter + 4 * sub;                    // softmax warp 0..7
        const uint32_t lane_off = (uint32_t)(32 * quarter) << 16;
        const int rtile = kCtaRows * (int)rank + rloc;        // row of the unit's tile
        const float sl2 = p.scale_log2 * (p.descale_q ? *p.descale_q : 1.0f) * (p.descale_k ? *p.descale_k : 1.0f);
        float* xmax = reinterpret_cast<float*>(smem + kOffX);  // the exchange area
        const uint32_t swz = (uint32_t)(rloc & 7);
        auto post = [&](int b) {   // this warp's shared-memory posts are done
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(b));
        };

        uint32_t g = 0, uq = 0;
        bool alive = true;
        Unit u;
        while (alive && iter.next(p, u)) {
            const int n = u.tiles();
            const bool row_valid = rtile < u.nrows;
            if (n <= 0) {
                // no key at all: o = 0, lse = -inf
                if (row_valid) {
                    __nv_bfloat16* row_out = p.out + ((int64_t)u.row0 + rtile) * kDv + 256 * half + 128 * sub;
                    for (int c = 0; c < 16; ++c) reinterpret_cast<uint4*>(row_out)[c] = make_uint4(0, 0, 0, 0);
                    if (half == 0 && sub == 0) p.lse[(int64_t)u.row0 + rtile] = -INFINITY;
                }
                continue;
            }
            int lim = u.L;
            if (p.causal) {
                const int64_t l = (int64_t)u.L - u.n + (int)((unsigned)(u.row_in_req + rtile) / (unsigned)p.h) + 1;
                lim = l < u.L ? (int)l : u.L;
            }
            if (lim > u.kb1 * kPage) lim = u.kb1 * kPage;   // keys of this piece (and of the table) only
            float m_run = -INFINITY, l_part = 0.f;
            for (int i = 0; i < n; ++i, ++g) {
                const uint32_t sb = g & 1u;
                if (!mbar_wait_bounded(bar(kBarSFull + sb), (g >> 1) & 1u, actl)) {
                    alive = false;
                    break;
                }
                tc_fence_after();
                float s[32];
                {
                    uint32_t raw[2][16];
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        tmem_ld16(tmem + lane_off + kTmemS + 64u * sb + 32u * sub + 16u * c, raw[c]);
                    tc_wait_ld();
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int k = 0; k < 16; ++k) s[16 * c + k] = __uint_as_float(raw[c][k]);
                }
                tc_fence_before();
                signal_leader(kBarSFree + sb, 18 + sw8);
                // scale to log2 units, mask the keys at or past the limit, these keys' maximum (a NaN among
                // the others, from q, wins it: with the plain maximum the row would look as if it had no key)
                const int kbase = (u.t0 + i) * kTileKeys + kPage * half + 32 * sub;
#pragma unroll
                for (int j = 0; j < 32; j += 2) mul2(s[j], s[j + 1], sl2);
                if (kbase + 32 > lim) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (kbase + j >= lim) s[j] = -INFINITY;
                }
                float hmax;
                {
                    float m0 = max_nan(s[0], s[1]), m1 = max_nan(s[2], s[3]);
#pragma unroll
                    for (int j = 4; j < 32; j += 4) {
                        m0 = max3_nan(m0, s[j], s[j + 1]);
                        m1 = max3_nan(m1, s[j + 2], s[j + 3]);
                    }
                    hmax = max_nan(m0, m1);
                }
                // three other threads hold the row's other keys
                xmax[sb * kSoftmaxThreads + 128 * sub + t] = hmax;
                post(kBarXchg + sb);
                if (!mbar_wait_bounded(bar(kBarXchg + sb), (g >> 1) & 1u, actl)) {
                    alive = false;
                    break;
                }
                float tmax;
                {
                    const float* x = xmax + sb * kSoftmaxThreads + rloc;
                    tmax = max_nan(max_nan(x[0], x[64]), max_nan(x[128], x[192]));
                }
                const float m_new = max_nan(m_run, tmax);
                const bool rescale = m_new > m_run + kRescaleThreshold || m_new != m_new;   // (a NaN, too)
                float factor = 1.f;
                if (rescale) {
                    factor = fast_exp2(m_run - m_new);  // 0 when m_run = -inf
                    l_part *= factor;
                    m_run = m_new;
                }
                // P packed in pairs into s[0..15]; zeros while every key so far is masked
                if (m_run != -INFINITY) {
                    float ps0 = 0.f, ps1 = 0.f;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float p0 = s[2 * j], p1 = s[2 * j + 1];
                        sub2(p0, p1, m_run);
                        p0 = fast_exp2(p0);
                        p1 = fast_exp2(p1);
                        add2(ps0, ps1, p0, p1);
                        s[j] = __uint_as_float(kFp8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1));
                    }
                    l_part += ps0 + ps1;
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) s[j] = 0.f;
                }
                // the P buffer is free, and O holds every PV up to tile g - 1, once PV(g - 1) is done
                if (g >= 1 && !mbar_wait_bounded(bar(kBarPvDone), (g - 1) & 1u, actl)) {
                    alive = false;
                    break;
                }
                if (i > 0 && __any_sync(0xffffffffu, rescale)) {
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 8; ++c) {
                        uint32_t raw[16];
                        tmem_ld16(tmem + lane_off + kTmemO + 128u * sub + 16u * c, raw);
                        tc_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            raw[k] = __float_as_uint(__uint_as_float(raw[k]) * factor);
                        tmem_st16(tmem + lane_off + kTmemO + 128u * sub + 16u * c, raw);
                    }
                    tc_wait_st();
                    tc_fence_before();
                }
                // P -> shared memory, K-major with 128-byte swizzle
                {
                    const uint32_t prow = sbase + kOffP + half * kBox + rloc * 128u;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        st_shared_v4u(prow + (((4u * sub + c) ^ swz) << 4), __float_as_uint(s[4 * c]),
                                      __float_as_uint(s[4 * c + 1]), __float_as_uint(s[4 * c + 2]),
                                      __float_as_uint(s[4 * c + 3]));
                }
                fence_proxy_async_smem();
                signal_leader(kBarPFull, sw8);
            }
            if (!alive) break;
            // The unit's row sums and maxima, for the warps that write its result: two places and two
            // barriers in turn, since a unit of one tile can end here before the unit before has been
            // written (the one before that has: this unit's P waited for the PV that followed it).
            {
                float* x = xmax + kUnitSums + (uq & 1u) * kUnitSumsStride;
                x[128 * sub + t] = l_part;
                if (sub == 0 && half == 0) x[kSoftmaxThreads + rloc] = m_run;
                post(kBarLx + (uq & 1u));
            }
            ++uq;
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

// Join the pieces of the units that the plan cut: lse = ln sum_i exp(lse_i), o = sum_i
// exp(lse_i - lse) o_i, in part order.  Part i begins a cut unit when its end lies inside a unit
// that it does not itself continue; its piece is slot 2 i + 1, and the parts after it that begin
// inside the same unit hold the others in slot 2 j.  A unit whose keys end before its first cut is
// whole, and a piece behind the last key was never written (lengths below the plan's).  Every CTA lists
// the cut units from the plan and the lengths (before it waits for the attention grid: they are older
// than that grid), then its warps take
// whole rows in turn, 16 columns a lane, two pieces' loads in flight -- or, when the cut units'
// rows are fewer than the warps (few units of many pieces), quarters of rows, 4 columns a lane and
// eight pieces in flight.
constexpr int kMergeThreads = 256;
constexpr int kMergeCtasPerPart = 6;   // three CTAs an SM, all resident at once
constexpr int kMergeMaxParts = 1024;

template <int kCols, int kAhead>
__device__ __forceinline__ void merge_unit_row(const int32_t* __restrict__ plan, int2 tk, int row, int col0, int64_t orow,
                                               const float* __restrict__ part_o, const float* __restrict__ part_lse,
                                               __nv_bfloat16* __restrict__ out, float* __restrict__ lse, int lane) {
    const int pieces = tk.y + 1;
    auto slot_row = [&](int k) { return (int64_t)(k == 0 ? 2 * tk.x + 1 : 2 * (tk.x + k)) * kTileRows + row; };
    auto lse_of = [&](int k) -> float {
        if (k >= pieces) return -INFINITY;
        if (k > 0) {   // a part that begins inside the unit but holds none of it
            const int32_t* e = plan + 8 * (int64_t)(tk.x + k);
            if (e[0] == e[3] && e[1] == e[4] && e[2] >= e[5]) return -INFINITY;
        }
        return part_lse[slot_row(k)];
    };
    const float l0 = lse_of(lane);   // of the first 32 pieces, a lane each
    float mx = l0;           // (a NaN piece makes the row NaN)
    for (int k = lane + 32; k < pieces; k += 32) mx = max_nan(mx, lse_of(k));
    for (int d = 16; d > 0; d >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    float sum = 0.f;
    if (mx != -INFINITY) {
        sum = expf(l0 - mx);
        for (int k = lane + 32; k < pieces; k += 32) sum += expf(lse_of(k) - mx);
    }
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    const float total = mx != -INFINITY ? mx + logf(sum) : -INFINITY;
    float acc[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c) acc[c] = 0.f;
    if (mx != -INFINITY) {
        float wl = expf(l0 - total);
        for (int k0 = 0; k0 < pieces; k0 += kAhead) {
            if (k0 > 0 && (k0 & 31) == 0) wl = expf(lse_of(k0 + lane) - total);   // the next 32 pieces' weights
            float4 v[kAhead][kCols / 4];
            float wt[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                wt[j] = __shfl_sync(0xffffffffu, wl, (k0 + j) & 31);
                if (k0 + j >= pieces) wt[j] = 0.f;
#pragma unroll
                for (int c = 0; c < kCols / 4; ++c)
                    v[j][c] = wt[j] != 0.f ? *reinterpret_cast<const float4*>(part_o + slot_row(k0 + j) * kDv + col0 + 128 * c + 4 * lane)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
#pragma unroll
                for (int c = 0; c < kCols / 4; ++c) {
                    acc[4 * c] += wt[j] * v[j][c].x;
                    acc[4 * c + 1] += wt[j] * v[j][c].y;
                    acc[4 * c + 2] += wt[j] * v[j][c].z;
                    acc[4 * c + 3] += wt[j] * v[j][c].w;
                }
        }
    }
#pragma unroll
    for (int c = 0; c < kCols / 4; ++c)
        *reinterpret_cast<uint2*>(out + orow * kDv + col0 + 128 * c + 4 * lane) =
            make_uint2(pack_bf16x2(acc[4 * c], acc[4 * c + 1]), pack_bf16x2(acc[4 * c + 2], acc[4 * c + 3]));
    if (col0 == 0 && lane == 0) lse[orow] = total;
}

__global__ void __launch_bounds__(kMergeThreads, kMergeCtasPerPart / 2)
chunk_merge_kernel(const int32_t* __restrict__ plan, const int32_t* __restrict__ cu,
                   const int32_t* __restrict__ cache_seqlens, int32_t parts, int32_t bs, int32_t h, int32_t num_tokens,
                   int32_t max_keys, int32_t causal, const float* __restrict__ part_o, const float* __restrict__ part_lse,
                   __nv_bfloat16* __restrict__ out, float* __restrict__ lse) {
    __shared__ int2 task[kMergeMaxParts];   // part that begins the unit, parts that continue it
    __shared__ int ntask;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x < 32) {   // in part order: every CTA must number the units alike
        int count = 0;
        for (int i0 = 0; i0 < parts; i0 += 32) {
            const int i = i0 + lane;
            int n = 0;
            if (i < parts) {
                const int32_t* r = plan + 8 * (int64_t)i;
                const int b = r[3], m = r[4], t = r[5];
                const bool continues = r[0] == b && r[1] == m && (r[2] > 0 || r[2] >= t);
                if (t > 0 && b >= 0 && b < bs && m >= 0 && !continues) {
                    int c0, rows, tiles = 0;
                    request_rows(cu, b, num_tokens, c0, rows);
                    if ((int64_t)m * kTileRows < (int64_t)rows * h)
                        tiles = (table_keys(cache_seqlens[b], rows, h, m, causal, max_keys) + kTileKeys - 1) / kTileKeys;
                    // (t >= tiles: whole, or no unit at all; a part that begins there holds none of it)
                    if (t < tiles)
                        for (const int32_t* e = r + 8; i + 1 + n < parts && e[0] == b && e[1] == m && e[2] > 0 && e[2] < tiles; e += 8) ++n;
                }
            }
            const unsigned found = __ballot_sync(0xffffffffu, n > 0);
            if (n > 0) task[count + __popc(found & ((1u << lane) - 1u))] = make_int2(i, n);
            count += __popc(found);
        }
        if (lane == 0) ntask = count;
    }
    __syncthreads();
    pdl_wait_prerequisites();
    const int64_t warp = (int64_t)blockIdx.x * (kMergeThreads / 32) + (threadIdx.x >> 5);
    const int64_t nwarps = (int64_t)gridDim.x * (kMergeThreads / 32);
    const bool quarters = (int64_t)ntask * kTileRows < nwarps;
    const int64_t total = (int64_t)ntask * kTileRows * (quarters ? 4 : 1);
    for (int64_t w = warp; w < total; w += nwarps) {
        const int64_t unit_row = quarters ? w >> 2 : w;
        const int row = (int)(unit_row % kTileRows);
        const int2 tk = task[unit_row / kTileRows];
        const int32_t* r = plan + 8 * (int64_t)tk.x;
        int c0, n;
        request_rows(cu, r[3], num_tokens, c0, n);
        const int64_t in_req = (int64_t)r[4] * kTileRows + row;
        if (in_req >= (int64_t)n * h) continue;
        const int64_t orow = (int64_t)c0 * h + in_req;
        if (quarters)
            merge_unit_row<4, 8>(plan, tk, row, 128 * (int)(w & 3), orow, part_o, part_lse, out, lse, lane);
        else
            merge_unit_row<16, 2>(plan, tk, row, 0, orow, part_o, part_lse, out, lse, lane);
    }
}

}  // namespace chunk
}  // namespace mla
