// Attention of a verify block over the paged key/value cache (moe_mxfp4_cache_attend).
//
// Mathematics.  A query row (stream s, position b, head) with scores x_j = scale q.k_j over the
// keys it sees: out = sum_j 2^(t_j - m) v_j / sum_j 2^(t_j - m), t = x log2 e, for any m near the
// largest t; partial results over parts of the keys are merged by their logarithms of sums.
//
// Work.  The G = q_heads / kv_heads rows that read one kv head are packed (b, g) and, over the
// shared prefix, (s, b, g): a unit is up to 256 such rows, a job a unit with its run of keys (the
// shared prefix once for the rows of all streams; every stream's own keys), cut into tiles of 128
// keys.  The tiles of all jobs in order are dealt out evenly to one CTA per SM, so that a long
// context is split over many CTAs and short ones are packed; a CTA's part of a job is a segment.
// A segment that is all its rows need is written straight to the output; the others leave
// normalised partial rows and the logarithm of their sum, which a second kernel merges in a fixed
// order.  The lengths are read on the device, so a captured graph follows the cache.
//
// A segment.  Two row slots of 128 rows, each with a softmax warpgroup (a thread per row), share
// a producer warp (TMA boxes of one head's page into a ring of K and V tiles) and an MMA warp
// (tcgen05: S = Q K^T from shared memory into tensor memory; O += P V with P, in 16 bits, from
// tensor memory over the columns of S).  While one slot's softmax runs, the tensor core works for
// the other.  Units of more than 128 rows use the slots for rows (each tile is used twice);
// smaller ones use both for the same rows, with every other tile, and merge the two accumulators
// at the end, so that a few rows over long keys, which wait for memory, keep two tiles going.
// The reference of the exponentials follows the running maximum only when that passes it by 2^8
// (P stays below 2^8 in any type, sums are fp32), so the accumulator is rescaled rarely, by the
// softmax warps themselves.
#include <cuda_fp16.h>

#include "cache.cuh"
#include "mma_f16.cuh"

namespace moe {

constexpr int kKeyTile = 128;
constexpr int kUnitRows = 256;                 // rows of a unit: two slots
constexpr int kAttThreads = 384;               // softmax warps 0-3 (slot 0), 4-7 (slot 1), producer, MMA, 2 idle
constexpr int kAttProducer = 8, kAttMma = 9;
constexpr uint32_t kTmemS = 0, kTmemO = 256;   // columns: S of slot x at 128 x, O at 256 + 128 x
constexpr float kRescale = 8.0f;               // exponents that the maximum may pass the reference by

struct AttendParams {
    moe_mxfp4_attend_args a;
    const uint16_t* v_pool;
    int G;                     // query heads per kv head
    int U;                     // units of a stream's own rows
    int U_sh;                  // units of all streams' rows
    int R_own;                 // rows of a slot for a stream's unit, a multiple of 4
    float c;                   // |scale| log2 e
    uint32_t q_flip;           // sign flips of a pair of query elements (a negative scale)
    unsigned long long timeout_ns;
    long long* head;           // workspace: schedule for the merge
    long long* cum;            // first own tile of each unit (of a head)
    float* split;              // partial rows of split jobs: 2 per CTA, kUnitRows rows each
    float* whole_sh;           // partial rows of whole jobs: shared, ...
    float* whole_own;          // ... and own
};
enum : int { kHeadShared = 0, kHeadTilesSh, kHeadTilesOwn, kHeadWords = 8 };

template <int D>
struct AttSmem {
    static constexpr int kPanel = 128 * 128;                 // 128 rows x 64 elements
    static constexpr int kTileBytes = kPanel * (D / 64);     // a K, V or Q tile
    static constexpr int kStages = D == 128 ? 5 : 10;
    uint8_t q[2][kTileBytes];
    uint8_t kv[kStages][kTileBytes];
    uint64_t full[kStages], empty[kStages], qfull, sfull[2], pfull[2], ofull[2], pair, drain;
    long long scan[3][12];
    long long first_y;
    float ml[2][128][2];                                     // the slots' references and sums
    uint32_t tmem;
    int first_unit, first_off;
    int bad_value;                                           // last segment (+ 1) with a non-finite block value
    int abort;
};

// ---- bounded waits ---------------------------------------------------------------------

__device__ __forceinline__ bool att_wait(uint64_t* bar, uint32_t parity, int* abort, unsigned long long timeout_ns) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long until = globaltimer_ns() + timeout_ns;
    while (!mbar_try_wait_sleep(bar, parity, 20000)) {
        if (*reinterpret_cast<volatile int*>(abort)) return false;
        if (globaltimer_ns() > until) {
            *reinterpret_cast<volatile int*>(abort) = 1;
            return false;
        }
    }
    return true;
}
// The same for a whole warp, which leaves together.
__device__ __forceinline__ bool att_warp_wait(uint64_t* bar, uint32_t parity, int* abort, unsigned long long timeout_ns) {
    return __all_sync(0xFFFFFFFFu, att_wait(bar, parity, abort, timeout_ns));
}

// ---- the schedule ------------------------------------------------------------------------

__device__ __forceinline__ int att_ctx(const CacheView& c, int s) {
    return min(max(c.length()[s], 0), c.L.M << c.page_shift);
}
__device__ __forceinline__ int att_used(const AttendParams& p, int s) {
    return p.a.lengths_dev ? min(max(p.a.lengths_dev[s], 0), p.a.block) : p.a.block;
}
// Whether stream s holds the pages of the shared prefix (their last one decides, as the tables
// of streams that hold a page at one index agree before it).
__device__ __forceinline__ bool att_shares(const CacheView& c, const AttendParams& p, int s, int shared) {
    if (shared <= 0) return false;
    const int i = (shared >> c.page_shift) - 1;
    return c.length()[s] >= shared && c.held()[s] > i && c.table(s)[i] == c.table(p.a.shared_stream)[i];
}
__device__ __forceinline__ int att_shared(const CacheView& c, const AttendParams& p) {
    const int n = p.a.shared_tokens;
    if (n <= 0) return 0;
    return c.length()[p.a.shared_stream] >= n && c.held()[p.a.shared_stream] >= (n >> c.page_shift) ? n : 0;
}

// A unit of a stream's own rows: its keys [begin, end) and rows.
struct OwnUnit {
    int r0, nrows, ctx, begin, end;
    __device__ int tiles() const { return (end - begin + kKeyTile - 1) / kKeyTile; }
};
__device__ __forceinline__ OwnUnit att_unit(const CacheView& c, const AttendParams& p, int unit, int shared) {
    OwnUnit w{0, 0, 0, 0, 0};
    const int s = unit / p.U;
    if (s >= p.a.streams) return w;
    w.r0 = (unit - s * p.U) * kUnitRows;
    const int used = att_used(p, s), rows = used * p.G;
    if (w.r0 >= rows) return w;
    w.nrows = min(kUnitRows, rows - w.r0);
    w.ctx = att_ctx(c, s);
    w.end = w.ctx + (p.a.mask_dev ? used : (w.r0 + w.nrows - 1) / p.G + 1);
    w.begin = att_shares(c, p, s, shared) ? shared : 0;
    return w;
}

// Sums over the CTA of a value per thread, and the thread's exclusive prefix.
template <int D>
__device__ __forceinline__ long long att_scan(AttSmem<D>& sm, int k, long long v, long long* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sm.scan[k][warp] = x;
    __syncthreads();
    long long before = 0, all = 0;
    for (int w = 0; w < kAttThreads / 32; ++w) {
        if (w < warp) before += sm.scan[k][w];
        all += sm.scan[k][w];
    }
    *total = all;
    __syncthreads();
    return before + x - v;
}

// What every warp knows of the schedule.
struct Schedule {
    int shared, tiles_sh;             // shared prefix in use, its tiles
    long long W_sh, W1;               // tiles of the shared jobs, of one head's own jobs
    long long g0, g1;                 // this CTA's tiles
};

template <int D>
__device__ Schedule att_schedule(const CacheView& c, const AttendParams& p, AttSmem<D>& sm) {
    Schedule sc;
    const int units = p.a.streams * p.U, tid = threadIdx.x;
    const int shared = att_shared(c, p);
    long long with = 0, without = 0, sharers = 0, t;
    for (int i = tid; i < units; i += kAttThreads) {
        const OwnUnit w = att_unit(c, p, i, shared);
        if (w.nrows == 0) continue;
        with += w.tiles();
        without += (w.end + kKeyTile - 1) / kKeyTile;
        sharers += w.r0 == 0 && w.begin > 0;
    }
    att_scan(sm, 0, sharers, &t);
    sharers = t;
    att_scan(sm, 1, with, &t);
    with = t;
    att_scan(sm, 2, without, &t);
    without = t;
    sc.shared = sharers > 1 ? shared : 0;      // one stream alone reads all through its own table
    sc.tiles_sh = (sc.shared + kKeyTile - 1) / kKeyTile;
    sc.W_sh = (long long)c.Hkv * p.U_sh * sc.tiles_sh;
    sc.W1 = sc.shared ? with : without;
    const long long W = sc.W_sh + (long long)c.Hkv * sc.W1;
    // as many CTAs as there are tiles, so that none of them is without one
    const long long n_cta = min((long long)gridDim.x, W), cta = blockIdx.x;
    sc.g0 = cta < n_cta ? W * cta / n_cta : W;
    sc.g1 = cta < n_cta ? W * (cta + 1) / n_cta : W;
    // the unit and the tile of it where this CTA's own jobs begin
    const long long y = sc.g0 > sc.W_sh ? (sc.g0 - sc.W_sh) % sc.W1 : 0;
    if (tid == 0) {
        sm.first_unit = 0;
        sm.first_off = 0;
    }
    __syncthreads();
    if (blockIdx.x == 0 || y > 0) {
        long long at = 0;
        for (int i0 = 0; i0 < units; i0 += kAttThreads) {
            const int i = i0 + tid;
            const int n = i < units ? att_unit(c, p, i, sc.shared).tiles() : 0;
            long long sum;
            const long long x = at + att_scan(sm, 0, n, &sum);
            if (n > 0 && x <= y && y < x + n) {
                sm.first_unit = i;
                sm.first_off = (int)(y - x);
            }
            if (blockIdx.x == 0 && i < units) p.cum[i] = x;
            at += sum;
        }
    }
    if (blockIdx.x == 0 && tid == 0) {
        p.head[kHeadShared] = sc.shared;
        p.head[kHeadTilesSh] = sc.W_sh;
        p.head[kHeadTilesOwn] = sc.W1;
    }
    __syncthreads();
    return sc;
}

// Where the partial rows of a segment go: first float4 of row 0 (rows run fastest, then the
// columns in fours), and the logarithms behind them.
struct Slot {
    float* base;
    int R;                     // rows of the slot
};
template <int D>
__device__ __forceinline__ int64_t slot_floats(int R) { return (int64_t)R * (D + 1); }
template <int D>
__device__ __forceinline__ Slot att_slot(const AttendParams& p, bool own, long long job, int cta, bool whole, bool first) {
    if (!whole) return {p.split + (2 * (int64_t)cta + (first ? 1 : 0)) * slot_floats<D>(kUnitRows), kUnitRows};
    if (own) return {p.whole_own + job * slot_floats<D>(p.R_own), p.R_own};
    return {p.whole_sh + job * slot_floats<D>(kUnitRows), kUnitRows};
}

struct Segment {
    bool own;
    bool by_keys;              // both slots hold the same rows and take every other tile
    bool direct;               // the rows need nothing else
    int h, s;
    int r0, nrows;
    int key0, T, key_end, ctx; // first key, tiles, end of the unit's keys, first block position
    long long job;
    bool whole, first;         // all tiles of the job; its first tile is here
};

// A warp's walk over its CTA's segments; all lanes hold the same values but `n`.
struct Walk {
    long long g;
    int h, unit, off;
    int base, n;               // tiles of the units base + lane
};
template <int D>
__device__ __forceinline__ Walk att_walk(const Schedule& sc, const AttSmem<D>& sm) {
    Walk w;
    w.g = sc.g0;
    w.h = sc.g0 > sc.W_sh ? (int)((sc.g0 - sc.W_sh) / sc.W1) : 0;
    w.unit = sm.first_unit;
    w.off = sm.first_off;
    w.base = -1;
    w.n = 0;
    return w;
}
__device__ bool att_next(const CacheView& c, const AttendParams& p, const Schedule& sc, Walk& w, Segment& sg) {
    if (w.g >= sc.g1) return false;
    if (w.g < sc.W_sh) {
        sg.own = false;
        sg.job = w.g / sc.tiles_sh;
        const int t0 = (int)(w.g - sg.job * sc.tiles_sh);
        sg.h = (int)(sg.job / p.U_sh);
        sg.r0 = (int)(sg.job % p.U_sh) * kUnitRows;
        sg.nrows = (int)min((long long)kUnitRows, (long long)p.a.streams * p.a.block * p.G - sg.r0);
        sg.s = p.a.shared_stream;
        sg.T = (int)min((long long)(sc.tiles_sh - t0), sc.g1 - w.g);
        sg.key0 = t0 * kKeyTile;
        sg.key_end = sg.ctx = sc.shared;
        sg.first = t0 == 0;
        sg.whole = sg.T == sc.tiles_sh;
        sg.direct = false;
    } else {
        const int units = p.a.streams * p.U, lane = threadIdx.x & 31;
        for (;;) {             // the next unit with tiles
            if (w.unit >= units) {
                w.unit = 0;
                if (++w.h >= c.Hkv) return false;
            }
            const int base = w.unit & ~31;
            if (base != w.base) {
                w.base = base;
                w.n = base + lane < units ? att_unit(c, p, base + lane, sc.shared).tiles() : 0;
            }
            const unsigned some = __ballot_sync(0xFFFFFFFFu, w.n > 0) >> (w.unit - base);
            if (some) {
                w.unit += __ffs(some) - 1;
                break;
            }
            w.unit = base + 32;
        }
        const OwnUnit u = att_unit(c, p, w.unit, sc.shared);
        const int n = u.tiles();
        sg.own = true;
        sg.h = w.h;
        sg.s = w.unit / p.U;
        sg.r0 = u.r0;
        sg.nrows = u.nrows;
        sg.job = (long long)w.h * units + w.unit;
        sg.T = (int)min((long long)(n - w.off), sc.g1 - w.g);
        sg.key0 = u.begin + w.off * kKeyTile;
        sg.key_end = u.end;
        sg.ctx = u.ctx;
        sg.first = w.off == 0;
        sg.whole = sg.T == n;
        sg.direct = sg.whole && u.begin == 0;
        w.off = 0;
        ++w.unit;
    }
    sg.by_keys = sg.nrows <= 128;
    w.g += sg.T;
    return true;
}

// Positions in the ring of a segment's tiles, in the order in which the MMA warp takes them:
// by rows K0 V0 K1 V1 ..., by keys K0 K1 V0 K2 V1 K3 ...
__device__ __forceinline__ int ring_k(const Segment& sg, int t) { return !sg.by_keys ? 2 * t : t < 2 ? t : 2 * t - 1; }
__device__ __forceinline__ int ring_v(const Segment& sg, int t) { return !sg.by_keys ? 2 * t + 1 : t + min(sg.T, t + 2); }

// ---- producer ------------------------------------------------------------------------------

template <int D>
__device__ void att_produce(const CacheView& c, const AttendParams& p, const Schedule& sc, AttSmem<D>& sm,
                            const CUtensorMap* kmap, const CUtensorMap* vmap) {
    using SM = AttSmem<D>;
    const int lane = threadIdx.x & 31, per_tile = kKeyTile >> c.page_shift;
    Walk w = att_walk<D>(sc, sm);
    Segment sg;
    uint32_t n = 0;                                    // tiles issued so far
    bool ok = true;
    while (ok && att_next(c, p, sc, w, sg)) {
        const int* table = c.table(sg.s);
        const int pages = min(min(c.held()[sg.s], c.L.M), (sg.key_end + c.page - 1) >> c.page_shift);
        // the page that this lane copies of a tile; outside the pool (zeros) where there is none
        const auto page_of = [&](int t) {
            const int i = ((sg.key0 + t * kKeyTile) >> c.page_shift) + lane;
            const int id = lane < per_tile && t < sg.T && i < pages ? table[i] : -1;
            return (unsigned)id < (unsigned)c.L.P ? id : c.L.P;
        };
        int kt = 0, vt = 0;                            // next K and V tile
        int kp = page_of(0), vp = kp;
        for (int i = 0; ok && i < 2 * sg.T; ++i, ++n) {
            const bool is_k = kt < sg.T && ring_k(sg, kt) == i;
            const int id = is_k ? kp : vp;
            const uint32_t st = n % SM::kStages;
            if (!att_warp_wait(&sm.empty[st], ((n / SM::kStages) & 1) ^ 1, &sm.abort, p.timeout_ns)) {
                ok = false;
                break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&sm.full[st], SM::kTileBytes);
            __syncwarp();
            if (lane < per_tile) {
                const uint32_t dst = smem_u32(sm.kv[st]) + lane * c.page * 128;
#pragma unroll
                for (int x = 0; x < D / 64; ++x)
                    tma_load_3d(dst + x * SM::kPanel, is_k ? kmap : vmap, 64 * x, sg.h * c.page, id, &sm.full[st]);
            }
            if (is_k) kp = page_of(++kt);
            else vp = page_of(++vt);
        }
    }
    // every copy has landed before the CTA leaves (already so but after an abort)
    const uint32_t last = n > SM::kStages ? n - SM::kStages : 0;
    if (!ok || *reinterpret_cast<volatile int*>(&sm.abort))
        for (uint32_t i = last; i < n; ++i) {
            const unsigned long long until = globaltimer_ns() + p.timeout_ns;
            while (!mbar_try_wait(&sm.full[i % SM::kStages], (i / SM::kStages) & 1))
                if (globaltimer_ns() > until) break;
        }
}

// ---- MMA -------------------------------------------------------------------------------------

// Rows of a V tile that no product may see: positions behind the unit's keys become zero, and so
// do non-finite elements at block positions, which some rows may not see (0 x NaN is NaN); the
// epilogue adds those to the rows that do see them.  Whole warp.
template <int D, bool kBf16>
__device__ __forceinline__ void att_mend_v(AttSmem<D>& sm, uint8_t* tile, const Segment& sg, int key0, int seg_no) {
    const int lane = threadIdx.x & 31;
    const int from = min(max(sg.ctx - key0, 0), kKeyTile), end = min(max(sg.key_end - key0, 0), kKeyTile);
    constexpr uint32_t kExp = kBf16 ? 0x7F80u : 0x7C00u;
    bool bad = false;
    for (int i = lane; i < (kKeyTile - from) * 8; i += 32) {
        const int row = from + (i >> 3);
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {
            uint4* at = reinterpret_cast<uint4*>(tile + x * AttSmem<D>::kPanel + row * 128 + (i & 7) * 16);
            if (row >= end) {
                *at = make_uint4(0u, 0u, 0u, 0u);
                continue;
            }
            uint4 v = *at;
            uint32_t* e = reinterpret_cast<uint32_t*>(&v);
            bool hit = false;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if ((e[k] & kExp) == kExp) { e[k] &= 0xFFFF0000u; hit = true; }
                if ((e[k] >> 16 & kExp) == kExp) { e[k] &= 0x0000FFFFu; hit = true; }
            }
            if (hit) *at = v;
            bad |= hit;
        }
    }
    if (bad) {
        *reinterpret_cast<volatile int*>(&sm.bad_value) = seg_no + 1;
        __threadfence_block();
    }
    fence_proxy_async_shared();
    __syncwarp();
}

template <int D, bool kBf16>
__device__ void att_mma(const CacheView& c, const AttendParams& p, const Schedule& sc, AttSmem<D>& sm, uint32_t tmem) {
    using SM = AttSmem<D>;
    constexpr uint32_t idesc_s = idesc_f16(128, 128, kBf16, false), idesc_o = idesc_f16(128, D, kBf16, true);
    const int lane = threadIdx.x & 31;
    Walk w = att_walk<D>(sc, sm);
    Segment sg;
    uint32_t base = 0, np[2] = {0, 0};
    int seg_no = 0;
    for (; att_next(c, p, sc, w, sg); ++seg_no) {
        const int N = sg.by_keys ? sg.T : 2 * sg.T;     // steps: slot n & 1
        const auto wait_full = [&](int pos) {
            const uint32_t i = base + pos;
            const bool ok = att_warp_wait(&sm.full[i % SM::kStages], (i / SM::kStages) & 1, &sm.abort, p.timeout_ns);
            tc_fence_after();
            return ok;
        };
        const auto scores = [&](int n) {                // S of step n
            const int t = sg.by_keys ? n : n >> 1, pos = ring_k(sg, t), x = n & 1;
            if (!wait_full(pos)) return false;
            if (lane == 0) {
                const uint32_t st = (base + pos) % SM::kStages;
                const uint32_t q = smem_u32(sm.q[sg.by_keys ? 0 : x]), k = smem_u32(sm.kv[st]);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint32_t o = (i / 4) * SM::kPanel + (i % 4) * 32;
                    tc_mma_f16_ss(tmem + kTmemS + 128 * x, smem_desc_sw128(q + o), smem_desc_sw128(k + o), idesc_s, i > 0);
                }
                tc_commit(&sm.sfull[x]);
                if (sg.by_keys || x == 1) tc_commit(&sm.empty[st]);
            }
            __syncwarp();
            return true;
        };
        if (!att_warp_wait(&sm.qfull, seg_no & 1, &sm.abort, p.timeout_ns)) return;
        tc_fence_after();
        for (int n = 0; n < min(N, 2); ++n)
            if (!scores(n)) return;
        for (int n = 0; n < N; ++n) {
            const int t = sg.by_keys ? n : n >> 1, pos = ring_v(sg, t), x = n & 1;
            if (!wait_full(pos)) return;
            const uint32_t st = (base + pos) % SM::kStages;
            const int key0 = sg.key0 + t * kKeyTile;
            if (key0 + kKeyTile > sg.ctx && (sg.by_keys || x == 0)) att_mend_v<D, kBf16>(sm, sm.kv[st], sg, key0, seg_no);
            if (!att_warp_wait(&sm.pfull[x], np[x]++ & 1, &sm.abort, p.timeout_ns)) return;
            tc_fence_after();
            if (lane == 0) {
                const uint32_t v = smem_u32(sm.kv[st]);
#pragma unroll
                for (int i = 0; i < kKeyTile / 16; ++i)
                    tc_mma_f16_ts(tmem + kTmemO + 128 * x, tmem + kTmemS + 128 * x + 8 * i,
                                  smem_desc_mn_sw128(v + i * 2048, SM::kPanel), idesc_o, n > 1 || i > 0);
                if (sg.by_keys || x == 1) tc_commit(&sm.empty[st]);
                if (n + 2 >= N) tc_commit(&sm.ofull[x]);
            }
            __syncwarp();
            if (n + 2 < N && !scores(n + 2)) return;
        }
        base += 2 * sg.T;
    }
}

// ---- softmax ---------------------------------------------------------------------------------

// A row of a segment: its token (stream * block + position) and query head.
struct Row {
    int64_t tok;
    int s, b, head;
    bool valid;
};
__device__ __forceinline__ Row att_row(const CacheView& c, const AttendParams& p, const Schedule& sc, const Segment& sg, int r) {
    Row x;
    const int i = sg.r0 + r, q = i / p.G;
    x.head = sg.h * p.G + (i - q * p.G);
    x.valid = r < sg.nrows;
    if (sg.own) {
        x.s = sg.s;
        x.b = q;
        x.tok = (int64_t)sg.s * p.a.block + q;
    } else {
        x.s = q / p.a.block;
        x.b = q - x.s * p.a.block;
        x.tok = q;
        if (x.valid) x.valid = x.b < att_used(p, x.s) && att_shares(c, p, x.s, sc.shared);
    }
    return x;
}

// Query rows r .. r + n - 1 of a segment into a Q tile (128-byte swizzle), zeros behind the unit.
// 128 threads; 16-byte chunks of a row on neighbouring lanes.
template <int D>
__device__ __forceinline__ void att_load_q(const AttendParams& p, const Segment& sg, uint8_t* tile, int from_row, int tile_row,
                                           int n) {
    constexpr int kChunks = D / 8;
    const int tid = threadIdx.x & 127;
    const uint16_t* q = static_cast<const uint16_t*>(p.a.q_dev);
#pragma unroll 8
    for (int i = tid; i < n * kChunks; i += 128) {
        const int row = i / kChunks, x = i % kChunks, r = sg.r0 + from_row + row;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (from_row + row < sg.nrows) {
            const int t = r / p.G;
            const int64_t tok = sg.own ? (int64_t)sg.s * p.a.block + t : t;
            v = *reinterpret_cast<const uint4*>(q + tok * p.a.q_stride + (int64_t)(sg.h * p.G + r - t * p.G) * D + x * 8);
            v.x ^= p.q_flip; v.y ^= p.q_flip; v.z ^= p.q_flip; v.w ^= p.q_flip;
        }
        const int tr = tile_row + row;
        *reinterpret_cast<uint4*>(tile + (x / 8) * AttSmem<D>::kPanel + tr * 128 + (((x & 7) ^ (tr & 7)) << 4)) = v;
    }
}

// Bit i: the row sees key j0 + i.
__device__ __forceinline__ void att_visible(const AttendParams& p, const Segment& sg, const Row& row, uint64_t bits, int j0,
                                            uint32_t (&vis)[4]) {
    const int lim = !sg.own ? sg.key_end : p.a.mask_dev ? sg.ctx : sg.ctx + row.b + 1;   // keys below it are seen
    const int n = min(max(lim - j0, 0), kKeyTile);
    uint64_t lo = n >= 64 ? ~0ull : (1ull << n) - 1, hi = n >= 128 ? ~0ull : n > 64 ? (1ull << (n - 64)) - 1 : 0ull;
    if (sg.own && p.a.mask_dev) {
        const int len = sg.key_end - sg.ctx;                                             // block positions, at most 64
        bits &= len >= 64 ? ~0ull : (1ull << len) - 1;
        const int at = sg.ctx - j0;                                                      // of block position 0 in the tile
        if (at <= -64 || at >= kKeyTile) bits = 0;
        else if (at < 0) lo |= bits >> -at;
        else if (at < 64) { lo |= bits << at; if (at) hi |= bits >> (64 - at); }
        else hi |= bits << (at - 64);
    }
    vis[0] = (uint32_t)lo; vis[1] = (uint32_t)(lo >> 32); vis[2] = (uint32_t)hi; vis[3] = (uint32_t)(hi >> 32);
}

// Non-finite values at block positions that this row sees, added to columns col .. col + 31 of o.
template <int D, bool kBf16>
__device__ __noinline__ void att_add_bad(const CacheView& c, const AttendParams& p, const Segment& sg, const Row& row,
                                         uint64_t bits, int col, float (&o)[32]) {
    const int from = max(sg.ctx, sg.key0), end = min(sg.key_end, sg.key0 + sg.T * kKeyTile);
    const int held = min(c.held()[sg.s], c.L.M);
    constexpr uint32_t kExp = kBf16 ? 0x7F80u : 0x7C00u;
    for (int j = from; j < end; ++j) {
        const int i = j - sg.ctx;
        if (p.a.mask_dev ? !(bits >> i & 1) : i > row.b) continue;
        const int pi = j >> c.page_shift, page = pi < held ? c.table(sg.s)[pi] : -1;
        if ((unsigned)page >= (unsigned)c.L.P) continue;
        const uint16_t* v = p.v_pool + page * c.page_stride + ((int64_t)sg.h * c.page + (j & (c.page - 1))) * D + col;
        for (int k = 0; k < 32; ++k)
            if ((v[k] & kExp) == kExp)
                o[k] += kBf16 ? __uint_as_float((uint32_t)v[k] << 16) : __half2float(__ushort_as_half(v[k]));
    }
}

template <int D, bool kBf16>
__device__ void att_softmax(const CacheView& c, const AttendParams& p, const Schedule& sc, AttSmem<D>& sm, uint32_t tmem) {
    const int slot = threadIdx.x >> 7, tid = threadIdx.x & 127, warp = tid >> 5, lane = threadIdx.x & 31;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;          // this warp's quarter of the tensor memory
    const uint32_t ts = tmem + kTmemS + 128 * slot + lanes, to = tmem + kTmemO + 128 * slot + lanes;
    Walk w = att_walk<D>(sc, sm);
    Segment sg;
    uint32_t ns = 0, no[2] = {0, 0}, np = 0;
    int seg_no = 0;
    bool ok = true;
    const auto both_here = [&] {              // a bounded barrier of the two warpgroups
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.pair);
        const bool here = att_warp_wait(&sm.pair, np++ & 1, &sm.abort, p.timeout_ns);
        tc_fence_after();
        return here;
    };
    for (; ok && att_next(c, p, sc, w, sg); ++seg_no) {
        // the query rows; the products that read the last ones have completed (ofull, below)
        if (sg.by_keys) att_load_q<D>(p, sg, sm.q[0], 64 * slot, 64 * slot, 64);
        else att_load_q<D>(p, sg, sm.q[slot], 128 * slot, 0, 128);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.qfull);
        const int r = sg.by_keys ? tid : 128 * slot + tid;
        const Row row = att_row(c, p, sc, sg, r);
        const bool busy = __any_sync(0xFFFFFFFFu, row.valid);
        const uint64_t bits = sg.own && p.a.mask_dev && row.valid ? p.a.mask_dev[row.tok] : 0;
        const int steps = sg.by_keys ? (sg.T + 1 - slot) / 2 : sg.T;
        float m = -INFINITY, l = 0.0f;
        for (int i = 0; i < steps; ++i) {
            const int t = sg.by_keys ? 2 * i + slot : i, j0 = sg.key0 + t * kKeyTile;
            if (!att_warp_wait(&sm.sfull[slot], ns++ & 1, &sm.abort, p.timeout_ns)) { ok = false; break; }
            tc_fence_after();
            if (busy) {
                uint32_t x[4][32];
#pragma unroll
                for (int k = 0; k < 4; ++k) tc_ld_x32(ts + 32 * k, x[k]);
                tc_wait_ld();
                if (j0 + kKeyTile > sg.ctx) {
                    uint32_t vis[4];
                    att_visible(p, sg, row, bits, j0, vis);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(vis[k] >> e & 1)) x[k][e] = 0xFF800000u;
                }
                float mx[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    mx[k] = __uint_as_float(x[k][0]);
#pragma unroll
                    for (int e = 1; e < 32; ++e) mx[k] = fmaxf(mx[k], __uint_as_float(x[k][e]));
                }
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.c;
                const bool passed = m != -INFINITY && top > m + kRescale;
                if (__any_sync(0xFFFFFFFFu, passed)) {
                    const float f = passed ? exp2_approx(m - top) : 1.0f;
                    l *= f;
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) {
                        uint32_t o[32];
                        tc_ld_x32(to + 32 * k, o);
                        tc_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tc_st_x32(to + 32 * k, o);
                    }
                }
                if (passed || m == -INFINITY) m = top;
                const float ref = m == -INFINITY ? 0.0f : m;
                float sum[2][2] = {};
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    uint32_t pk[32];
#pragma unroll
                    for (int e = 0; e < 64; e += 2) {
                        float a, b;
                        fma_x2(a, b, __uint_as_float(x[k + e / 32][e % 32]), __uint_as_float(x[k + e / 32][e % 32 + 1]), p.c,
                               -ref);
                        a = exp2_approx(a);
                        b = exp2_approx(b);
                        add_x2(sum[(e / 2) & 1][0], sum[(e / 2) & 1][1], a, b);
                        pk[e / 2] = pack_f16<kBf16>(a, b);
                    }
                    tc_st_x32(ts + 16 * k, pk);
                }
                l += (sum[0][0] + sum[0][1]) + (sum[1][0] + sum[1][1]);
                tc_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.pfull[slot]);
        }
        // the rows: out of tensor memory, by keys merged from both slots (half of the columns each)
        const bool both = sg.by_keys && sg.T > 1;
        if (ok && (both || !sg.by_keys || slot == 0)) {
            if (both || slot == 0) ok = att_warp_wait(&sm.ofull[0], no[0] & 1, &sm.abort, p.timeout_ns);
            if (ok && (both || (!sg.by_keys && slot == 1))) ok = att_warp_wait(&sm.ofull[1], no[1] & 1, &sm.abort, p.timeout_ns);
        } else if (ok) {       // slot 1 without a tile: the products that read the queries have completed
            ok = att_warp_wait(&sm.ofull[0], no[0] & 1, &sm.abort, p.timeout_ns);
        }
        ++no[0];
        if (!sg.by_keys || sg.T > 1) ++no[1];
        if (!ok) break;
        tc_fence_after();
        float f[2] = {1.0f, 0.0f};
        if (both) {
            sm.ml[slot][tid][0] = m;
            sm.ml[slot][tid][1] = l;
            if (!both_here()) { ok = false; break; }
            const float m2 = sm.ml[slot ^ 1][tid][0], l2 = sm.ml[slot ^ 1][tid][1];
            // in the order of the slots, so that both compute the same
            const float ma = slot ? m2 : m, mb = slot ? m : m2, la = slot ? l2 : l, lb = slot ? l : l2;
            const float mm = fmaxf(ma, mb);
            f[0] = ma == -INFINITY ? 0.0f : exp2_approx(ma - mm);
            f[1] = mb == -INFINITY ? 0.0f : exp2_approx(mb - mm);
            if (ma != ma || mb != mb) f[0] = f[1] = NAN;
            m = mm;
            l = la * f[0] + lb * f[1];
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const float lse2 = l == 0.0f ? -INFINITY : m + log2f(l);
        const bool mend = *reinterpret_cast<volatile int*>(&sm.bad_value) == seg_no + 1;
        const bool writes = busy && (both || !sg.by_keys || slot == 0);
        const int col0 = both ? slot * (D / 2) : 0, cols = both ? D / 2 : D;
        const Slot out = att_slot<D>(p, sg.own, sg.job, blockIdx.x, sg.whole, sg.first);
        if (writes) {
            for (int col = col0; col < col0 + cols; col += 32) {
                float o[32];
                uint32_t y[32];
                if (both) {
                    uint32_t z[32];
                    tc_ld_x32(tmem + kTmemO + lanes + col, y);
                    tc_ld_x32(tmem + kTmemO + 128 + lanes + col, z);
                    tc_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(y[e]) * f[0] + __uint_as_float(z[e]) * f[1];
                } else {
                    tc_ld_x32(to + col, y);
                    tc_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(y[e]);
                }
                if (mend && row.valid) att_add_bad<D, kBf16>(c, p, sg, row, bits, col, o);
                if (row.valid && sg.direct) {
                    uint16_t* to_row = static_cast<uint16_t*>(p.a.out_dev) + (row.tok * p.a.q_heads + row.head) * D + col;
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        *reinterpret_cast<uint4*>(to_row + e) =
                            make_uint4(pack_f16<kBf16>(o[e] * inv, o[e + 1] * inv), pack_f16<kBf16>(o[e + 2] * inv, o[e + 3] * inv),
                                       pack_f16<kBf16>(o[e + 4] * inv, o[e + 5] * inv), pack_f16<kBf16>(o[e + 6] * inv, o[e + 7] * inv));
                } else if (row.valid) {
                    float4* to_slot = reinterpret_cast<float4*>(out.base) + (int64_t)(col / 4) * out.R + r;
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        to_slot[(int64_t)(e / 4) * out.R] = make_float4(o[e] * inv, o[e + 1] * inv, o[e + 2] * inv, o[e + 3] * inv);
                }
                __syncwarp();
            }
            if (col0 == 0 && row.valid) {
                if (!sg.direct) out.base[(int64_t)out.R * D + r] = lse2;
                else if (p.a.lse_dev) p.a.lse_dev[row.tok * p.a.q_heads + row.head] = lse2 * 0.693147180559945309f;
            }
        }
        if (both && !both_here()) { ok = false; break; }      // both have read both accumulators
    }
}

template <int D, bool kBf16>
__global__ void __launch_bounds__(kAttThreads, 1) attend_kernel(const CacheView c, const AttendParams p,
                                                                const __grid_constant__ CUtensorMap kmap,
                                                                const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ __align__(1024) uint8_t raw[];       // the only shared memory: its tiles are 1024-byte aligned
    AttSmem<D>& sm = *reinterpret_cast<AttSmem<D>*>(raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < AttSmem<D>::kStages; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
        }
        mbar_init(&sm.qfull, 8);
        for (int x = 0; x < 2; ++x) {
            mbar_init(&sm.sfull[x], 1);
            mbar_init(&sm.pfull[x], 4);
            mbar_init(&sm.ofull[x], 1);
        }
        mbar_init(&sm.pair, 8);
        mbar_init(&sm.drain, 1);
        sm.abort = 0;
        sm.bad_value = 0;
        fence_barrier_init();
    }
    if (warp == kAttMma) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    const Schedule sc = att_schedule<D>(c, p, sm);      // ends with a CTA barrier
    tc_fence_after();
    grid_dependency_launch();
    const uint32_t tmem = sm.tmem;
    if (warp < 8) {
        reg_grow<208>();
        att_softmax<D, kBf16>(c, p, sc, sm, tmem);
    } else {
        reg_shrink<80>();
        if (warp == kAttProducer) {
            if (lane == 0) {
                prefetch_tensormap(&kmap);
                prefetch_tensormap(&vmap);
            }
            att_produce<D>(c, p, sc, sm, &kmap, &vmap);
        } else if (warp == kAttMma) {
            att_mma<D, kBf16>(c, p, sc, sm, tmem);
            if (lane == 0) {                            // every product has completed before the memory is freed
                tc_commit(&sm.drain);
                const unsigned long long until = globaltimer_ns() + p.timeout_ns;
                while (!mbar_try_wait(&sm.drain, 0))
                    if (globaltimer_ns() > until) break;
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kAttMma) tmem_dealloc(tmem, 512);
    if (threadIdx.x == 0 && sm.abort) raise_status(c.state + kCacheStatus, MOE_ERR_TIMEOUT, blockIdx.x);
}

// ---- merge -----------------------------------------------------------------------------------

// The parts of a job: tiles x0 .. x0 + n of all W, over `grid` CTAs.
struct Parts {
    long long job;
    int c0, c1;
    bool own;
};
__device__ __forceinline__ Parts att_parts(bool own, long long job, long long x0, long long n, long long W, int grid) {
    Parts q;
    q.own = own;
    q.job = job;
    const long long n_cta = min((long long)grid, W);
    q.c0 = (int)min(((x0 + 1) * n_cta - 1) / W, n_cta - 1);
    q.c1 = (int)min(((x0 + n) * n_cta - 1) / W, n_cta - 1);
    return q;
}
template <int D>
__device__ __forceinline__ Slot att_part(const AttendParams& p, const Parts& q, int cta) {
    return att_slot<D>(p, q.own, q.job, cta, q.c0 == q.c1, cta == q.c0);
}

constexpr int kMergeRows = 32;

// A CTA per (head, unit of a stream, 32 rows): out = sum of w_i part_i, w_i = 2^(lse_i - lse).
template <int D, bool kBf16>
__global__ void __launch_bounds__(256) attend_merge_kernel(const CacheView c, const AttendParams p, int grid, int groups) {
    grid_dependency_wait();
    __shared__ float s_m[kMergeRows], s_inv[kMergeRows];
    __shared__ uint2 s_out[kMergeRows][D / 4 + 1];
    const int shared = (int)p.head[kHeadShared];
    const long long W_sh = p.head[kHeadTilesSh], W1 = p.head[kHeadTilesOwn], W = W_sh + (long long)c.Hkv * W1;
    const int units = p.a.streams * p.U;
    long long b = blockIdx.x;
    const int group = (int)(b % groups); b /= groups;
    const int unit = (int)(b % units), h = (int)(b / units);
    const OwnUnit u = att_unit(c, p, unit, shared);
    const int row0 = group * kMergeRows, n = min(kMergeRows, u.nrows - row0);
    if (n <= 0) return;
    const Parts own = att_parts(true, (long long)h * units + unit, W_sh + (long long)h * W1 + p.cum[unit], u.tiles(), W, grid);
    const bool shares = u.begin > 0;
    if (!shares && own.c0 == own.c1) return;            // written by its only segment
    const int s = unit / p.U, tiles_sh = (shared + kKeyTile - 1) / kKeyTile;
    // rows of this stream among the packed rows of all: they may cross from one shared unit to the next
    const long long packed = (long long)s * p.a.block * p.G + u.r0 + row0;
    const auto shared_parts = [&](int row) {
        const long long job = (long long)h * p.U_sh + (packed + row) / kUnitRows;
        return att_parts(false, job, job * tiles_sh, tiles_sh, W, grid);
    };
    const auto each = [&](int row, auto f) {
        for (int i = own.c0; i <= own.c1; ++i) f(att_part<D>(p, own, i), u.r0 % kUnitRows + row0 + row);
        if (!shares) return;
        const Parts q = shared_parts(row);
        for (int i = q.c0; i <= q.c1; ++i) f(att_part<D>(p, q, i), (int)((packed + row) % kUnitRows));
    };
    const int64_t first_tok = (int64_t)s * p.a.block;
    if (threadIdx.x < n) {
        const int row = threadIdx.x;
        float m = -INFINITY, z = 0.0f;
        bool nan = false;
        each(row, [&](const Slot& sl, int r) {
            const float x = sl.base[(int64_t)sl.R * D + r];
            m = fmaxf(m, x);
            nan |= x != x;
        });
        const float ref = m == -INFINITY ? 0.0f : m;
        each(row, [&](const Slot& sl, int r) { z += exp2_approx(sl.base[(int64_t)sl.R * D + r] - ref); });
        if (nan) z = NAN;
        s_m[row] = ref;
        s_inv[row] = z == 0.0f ? 0.0f : 1.0f / z;
        if (p.a.lse_dev) {
            const int i = u.r0 + row0 + row, t = i / p.G;
            p.a.lse_dev[(first_tok + t) * p.a.q_heads + h * p.G + (i - t * p.G)] =
                z == 0.0f ? -INFINITY : (ref + log2f(z)) * 0.693147180559945309f;
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < n * (D / 4); e += 256) {
        const int row = e % n, x = e / n;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const float ref = s_m[row], inv = s_inv[row];
        each(row, [&](const Slot& sl, int r) {
            const float w = exp2_approx(sl.base[(int64_t)sl.R * D + r] - ref) * inv;
            const float4 v = reinterpret_cast<const float4*>(sl.base)[(int64_t)x * sl.R + r];
            if (w != 0.0f) {                             // a part that saw nothing may hold nothing
                acc.x = fmaf(w, v.x, acc.x); acc.y = fmaf(w, v.y, acc.y);
                acc.z = fmaf(w, v.z, acc.z); acc.w = fmaf(w, v.w, acc.w);
            }
        });
        s_out[row][x] = make_uint2(pack_f16<kBf16>(acc.x, acc.y), pack_f16<kBf16>(acc.z, acc.w));
    }
    __syncthreads();
    for (int e = threadIdx.x; e < n * (D / 4); e += 256) {
        const int row = e / (D / 4), x = e % (D / 4);
        const int i = u.r0 + row0 + row, t = i / p.G;
        uint16_t* out = static_cast<uint16_t*>(p.a.out_dev) +
                        ((first_tok + t) * p.a.q_heads + h * p.G + (i - t * p.G)) * (int64_t)D;
        reinterpret_cast<uint2*>(out)[x] = s_out[row][x];
    }
}

}  // namespace moe

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

int check_shape(const moe_mxfp4_cache* c, int32_t streams, int32_t block, int32_t q_heads) {
    if (!c || streams < 0 || streams > c->cfg.num_streams || block < 0 || q_heads < 1) return MOE_ERR_INVALID_ARG;
    if (q_heads % c->cfg.kv_heads || q_heads / c->cfg.kv_heads > 256) return MOE_ERR_INVALID_ARG;
    if ((int64_t)streams * block > 0x7FFFFFFF / q_heads) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// Sections of the workspace.
struct AttendLayout {
    int G, U, U_sh, R_own;
    size_t cum, split, whole_sh, whole_own, total;
};
AttendLayout attend_layout(const moe_mxfp4_cache* c, int streams, int block, int q_heads) {
    AttendLayout L;
    L.G = q_heads / c->cfg.kv_heads;
    const int64_t rows = (int64_t)block * L.G;
    L.U = (int)((rows + moe::kUnitRows - 1) / moe::kUnitRows);
    L.U_sh = (int)((streams * rows + moe::kUnitRows - 1) / moe::kUnitRows);
    L.R_own = (int)(rows < moe::kUnitRows ? (rows + 3) / 4 * 4 : moe::kUnitRows);   // slots are whole float4s
    const size_t row = (size_t)(c->cfg.head_dim + 1) * 4, jobs = (size_t)c->cfg.kv_heads;
    L.cum = 256;
    L.split = L.cum + up256((size_t)streams * L.U * 8);
    L.whole_sh = L.split + up256(2 * (size_t)c->sm_count * moe::kUnitRows * row);
    L.whole_own = L.whole_sh + up256(jobs * L.U_sh * moe::kUnitRows * row);
    L.total = L.whole_own + up256(jobs * streams * L.U * L.R_own * row);
    return L;
}

template <int D, bool kBf16>
int launch_attend(const moe_mxfp4_cache* c, int layer, const moe::CacheView& v, const moe::AttendParams& p, cudaStream_t st) {
    constexpr size_t smem = sizeof(moe::AttSmem<D>);
    static_assert(smem <= 227 * 1024, "a CTA's shared memory");
    auto* kern = moe::attend_kernel<D, kBf16>;
    const int groups = (p.R_own + moe::kMergeRows - 1) / moe::kMergeRows;
    const int64_t merge = (int64_t)c->cfg.kv_heads * p.a.streams * p.U * groups;
    if (merge > 0x7FFFFFFF) return MOE_ERR_UNSUPPORTED;
    kern<<<c->sm_count, moe::kAttThreads, smem, st>>>(v, p, c->maps[2 * layer], c->maps[2 * layer + 1]);
    if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
    return moe::launch_dependent(moe::attend_merge_kernel<D, kBf16>, dim3((unsigned)merge), dim3(256), 0, st, v, p, c->sm_count,
                                 groups) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

}  // namespace

bool moe::attend_prepare() {
    const auto set = [](auto* kern, size_t smem) {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) == cudaSuccess;
    };
    return set(attend_kernel<128, true>, sizeof(AttSmem<128>)) && set(attend_kernel<128, false>, sizeof(AttSmem<128>)) &&
           set(attend_kernel<64, true>, sizeof(AttSmem<64>)) && set(attend_kernel<64, false>, sizeof(AttSmem<64>));
}

extern "C" int moe_mxfp4_cache_attend_bytes(const moe_mxfp4_cache* c, int32_t streams, int32_t block, int32_t q_heads,
                                            size_t* bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    if (const int r = check_shape(c, streams, block, q_heads)) return r;
    *bytes = attend_layout(c, streams, block, q_heads).total;
    return MOE_OK;
}

extern "C" int moe_mxfp4_cache_attend(moe_mxfp4_cache* c, void* state_dev, int32_t layer, const moe_mxfp4_attend_args* args,
                                      void* workspace_dev, size_t workspace_bytes, void* stream) {
    if (!c || !state_dev || !aligned(state_dev, 16) || !args || layer < 0 || layer >= c->cfg.num_layers)
        return MOE_ERR_INVALID_ARG;
    moe::AttendParams p = {};
    p.a = *args;
    moe_mxfp4_attend_args& a = p.a;
    if (const int r = check_shape(c, a.streams, a.block, a.q_heads)) return r;
    const int64_t row = (int64_t)a.q_heads * c->cfg.head_dim;
    if (a.q_stride == 0) a.q_stride = row;
    if (a.q_stride < row || a.q_stride % 8 || !(a.scale - a.scale == 0.0f)) return MOE_ERR_INVALID_ARG;
    if (!aligned(a.lse_dev, 4) || !aligned(a.lengths_dev, 4) || !aligned(a.mask_dev, 8) || (a.mask_dev && a.block > 64))
        return MOE_ERR_INVALID_ARG;
    if (a.shared_tokens < 0 || a.shared_tokens % c->cfg.page_tokens) return MOE_ERR_INVALID_ARG;
    if (a.shared_tokens > 0 && (a.shared_stream < 0 || a.shared_stream >= c->cfg.num_streams ||
                                a.shared_tokens / c->cfg.page_tokens > c->cfg.max_pages))
        return MOE_ERR_INVALID_ARG;
    if (a.streams == 0 || a.block == 0) return MOE_OK;
    if (!a.q_dev || !a.out_dev || !aligned(a.q_dev, 16) || !aligned(a.out_dev, 16)) return MOE_ERR_INVALID_ARG;
    const AttendLayout L = attend_layout(c, a.streams, a.block, a.q_heads);
    if (!workspace_dev || !aligned(workspace_dev, 256) || workspace_bytes < L.total) return MOE_ERR_WORKSPACE;
    const moe::DeviceScope on(c->device);
    if (!on.ok()) return MOE_ERR_CUDA;
    char* ws = static_cast<char*>(workspace_dev);
    p.v_pool = static_cast<const uint16_t*>(c->layers[layer].v_dev);
    p.G = L.G;
    p.U = L.U;
    p.U_sh = L.U_sh;
    p.R_own = L.R_own;
    // a negative scale turns the queries' signs; a scale of zero is one below any score's last bit,
    // which keeps hidden keys (-inf) hidden
    const float s = a.scale < 0.0f ? -a.scale : a.scale;
    p.c = s * 1.44269504088896341f;
    if (p.c < 0x1p-100f) p.c = 0x1p-100f;
    p.q_flip = a.scale < 0.0f ? 0x80008000u : 0u;
    p.timeout_ns = (unsigned long long)c->cfg.timeout_us * 1000ull;
    p.head = reinterpret_cast<long long*>(ws);
    p.cum = reinterpret_cast<long long*>(ws + L.cum);
    p.split = reinterpret_cast<float*>(ws + L.split);
    p.whole_sh = reinterpret_cast<float*>(ws + L.whole_sh);
    p.whole_own = reinterpret_cast<float*>(ws + L.whole_own);
    const moe::CacheView v = moe::cache_view(c, state_dev);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool bf16 = c->cfg.dtype == MOE_DTYPE_BF16;
    if (c->cfg.head_dim == 128)
        return bf16 ? launch_attend<128, true>(c, layer, v, p, st) : launch_attend<128, false>(c, layer, v, p, st);
    return bf16 ? launch_attend<64, true>(c, layer, v, p, st) : launch_attend<64, false>(c, layer, v, p, st);
}
