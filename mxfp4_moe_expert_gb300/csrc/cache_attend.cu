// Attention of a verify block over the paged key/value cache (moe_mxfp4_cache_attend).
//
// Mathematics.  A query row (stream s, position b, head) with scores x_j = scale q.k_j over the
// keys it sees: out = sum_j 2^(t_j - m) v_j / sum_j 2^(t_j - m), t = x log2 e, for any m near the
// largest t; partial results over parts of the keys are merged by their logarithms of sums.
//
// Work.  The G = q_heads / kv_heads rows that read one kv head are packed (b, g) and, over the
// shared prefix, (s, b, g).  A job is a unit of these rows with its run of keys (the shared prefix
// once for the rows of all streams; every stream's own keys), cut into tiles of 128 keys.  There
// are two kinds of units (the rules between them are beside attend_layout and in the entry point).
// Wide ones have 256 rows: both row slots of a CTA take each tile of keys, so that it is read from
// memory once for 256 rows.  Narrow ones have up to 128 rows: the two slots of a CTA work on
// different jobs, or parts of a job, each with a ring of its own, so that the wait for memory in
// one is covered by the other.  The tiles of the wide jobs are dealt out evenly to
// the CTAs (one per SM), those of the narrow ones to their 2 x CTAs slots, in order: a long run of
// keys is split over many, short ones are packed.  What one worker does of a job is a segment.
// A segment that is all its rows need is written straight to the output; the others leave
// normalised partial rows and the logarithm of their sum, which a second kernel merges in a fixed
// order.  The lengths are read on the device, so a captured graph follows the cache.
//
// A slot.  Producer warp: walks the worker's segments, publishes each, and copies the K and V
// tiles (TMA boxes of one head's page) into the ring.  MMA warp: S = Q K^T from shared memory into
// tensor memory, O += P V with P, in 16 bits, from tensor memory over the columns of S.  Softmax
// warpgroup: a thread per row.  The reference of the exponentials follows the running maximum only
// when that passes it by some exponents (kRescale; P stays below 2^8 in bf16 and 2^15 in fp16, sums
// are fp32), so the accumulator is rescaled rarely, by the softmax warps themselves.
//
// What bounds it, on 152 SMs.  Reading keys where there are few rows: 96 streams that decode one
// position over 700..6000 keys (1.32 GB) take 200 us, 6.6 TB/s, 0.97 of the copy rate.  The tensor
// core's chain where a long prefix is shared: 64 streams x 8 positions x 64 heads behind 32768 keys
// (0.57 TFLOP) take 430 us, 1.32 PFLOP/s, 0.68 of the cuBLAS rate.  A wide tile (256 rows x 128
// keys) takes about 2950 cycles for 2048 of products: scores -> softmax (1500) -> P V and the next
// scores (1024) follow one another in each slot, and shared memory is read at its full 128 bytes a
// cycle while Q K^T runs.  The launches, the schedule and the merge where there is little work: one
// stream of 8 positions over 4093 keys takes 16 us, of which its tiles are 3.
#include <cuda_fp16.h>

#include <atomic>

#include "cache.cuh"
#include "mma_f16.cuh"

namespace moe {

constexpr int kKeyTile = 128;
constexpr int kAttThreads = 384;               // softmax warps 0-3 (slot 0), 4-7 (slot 1), producers, MMA
constexpr int kAttProducer = 8, kAttMma = 10;  // + slot
constexpr uint32_t kTmemS = 0, kTmemO = 256;   // columns: S of slot x at 128 x, O at 256 + 128 x
// The reference of a row's exponentials is this many exponents below its maximum when it was set
// (att_below), and follows when the maximum passes that by kRescale.  bf16 terms have fp32's range.
// An fp16 term is exact to half a step down to 2^-14 and at most 2^-25 off below: with terms of up to
// 2^15 that is 2^-26 and 2^-37 of the maximum, so that a tail of many small terms keeps its weight
// (with a reference at the maximum, 65536 terms of 2^-26 of it were lost, 0.07 % of the sum).
// Exponents beyond 2^22 have steps of half and more, and terms no room for them below fp16's largest.
template <bool kBf16>
__device__ __forceinline__ float att_below(float m) { return !kBf16 && fabsf(m) < 0x1p22f ? 12.0f : 0.0f; }
template <bool kBf16> constexpr float kRescale = kBf16 ? 8.0f : 3.0f;
// A segment costs about this many tiles more than its tiles (its queries, its start, its rows' way
// out); dealt out with them.  3 for narrow ones rather than 2: 96 streams decode in 205.7 us
// instead of 209.0, other cases do not change.
constexpr int kPadWide = 1, kPadNarrow = 3;
// Marks of wide segments, in turn.  Slot 0's MMA warp may mark the next segment while slot 1's softmax
// warps have yet to read the mark of this one, but not the one after it: its turn there follows slot
// 1's products of the next segment, whose queries those warps load after they have read.
constexpr int kWideMarks = 2;

struct AttendParams {
    moe_mxfp4_attend_args a;
    const uint16_t* v_pool;
    int G;                     // query heads per kv head
    uint32_t g_mul;            // ceil(2^32 / G): x / G = high word of x g_mul for x < 2^16 (G = 1 apart)
    int wide_sh, wide_own;     // units of 256 rows (else 128) over the shared prefix, over the own keys
    int U, U_sh;               // units of a stream's own rows, of all streams' rows
    int R_own;                 // rows of a slot for a stream's unit, a multiple of 4
    float c;                   // |scale| log2 e
    uint32_t q_flip;           // sign flips of a pair of query elements (a negative scale)
    unsigned long long timeout_ns;
    struct JobList* head;      // workspace: the lists (narrow, wide) for the merge
    int4* units;               // each unit: first own place (of a head), rows, tiles, whether it shares the prefix
    float* split_wide;         // partial rows of split jobs: 2 per worker, 256 rows each, ...
    float* split_narrow;       // ... 128 rows each
    float* whole_sh;           // partial rows of whole jobs: shared, ...
    float* whole_own;          // ... and own
    __device__ __forceinline__ int div_g(int x) const { return G == 1 ? x : (int)__umulhi((uint32_t)x, g_mul); }
    __host__ __device__ int rows_sh() const { return wide_sh ? 256 : 128; }
    __host__ __device__ int rows_own() const { return wide_own ? 256 : 128; }
};
// One worker's part of a job, for one slot.
struct Segment {
    float* out;                // partial rows (nullptr: straight to the output)
    int R, out_row;            // rows of that slot, the first one here
    int own, wide, h, s;
    int r0, nrows;             // first packed row, rows
    int key0, T, key_end, ctx; // first key, tiles (0: no more segments), end of the keys, first block position
    int no, wide_no;           // segments, and wide ones, of this slot before it
};

// The jobs of one list (wide or narrow): shared ones, then own ones, each with its places in a
// row of W (below 2^31: checked on the host): a job with n tiles has pad + n, tile i at place
// pad + i.  Worker w has q places, one more when w < rem.
struct JobList {
    int pad, tiles_sh, has_own;
    int W_sh, W1, W;                  // places of the shared jobs, of one head's own jobs, of all
    int workers, q, rem;
    __device__ int first(int w) const { return q * w + min(w, rem); }
    __device__ int worker(int place) const {
        const int big = rem * (q + 1);
        return min(place < big ? place / (q + 1) : rem + (place - big) / q, workers - 1);
    }
};
// A unit of a stream's own rows: its keys [begin, end) and rows.
struct OwnUnit {
    int r0, nrows, ctx, begin, end;
    __device__ int tiles() const { return (end - begin + kKeyTile - 1) / kKeyTile; }
};
template <int D>
struct AttSmem {
    static constexpr int kPanel = 128 * 128;                 // 128 rows x 64 elements
    static constexpr int kTileBytes = kPanel * (D / 64);     // a K, V or Q tile
    static constexpr int kStages = D == 128 ? 4 : 8;         // of the wide ring; half of them for each narrow one
    uint8_t q[2][kTileBytes];
    uint8_t kv[kStages][kTileBytes];
    uint64_t full[2][kStages], empty[2][kStages];            // [0]: wide, [1]: narrow
    uint64_t mended[kStages];                                // wide: slot 0's MMA warp has mended the V tile
    uint64_t turn[2];                                        // wide: the slot's turn on the tensor core
    uint64_t handover;                                       // the first kind's tiles are used up (att_producer)
    uint64_t segf[2][2], sege[2][2], qfull[2], sfull[2], phalf[2], pfull[2], ofull[2], drain[2];
    Segment seg[2][2];
    int sums[4][kAttThreads / 32];
    uint32_t tmem;
    JobList list[2];                                         // narrow, wide
    int first_h[2], first_unit[2], first_off[2];             // where each slot's own jobs begin,
    OwnUnit first_own[2];                                    // and that unit (no rows: not looked up)
    int bad_value[2], bad_wide[kWideMarks];                  // last narrow (wide) segment (+ 1) with a non-finite block value
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
// Copies and products that are under way end by themselves, whatever the other warps do: a CTA that
// gives up still waits for them, with a limit of its own that does not follow the caller's (two
// seconds, some 10^5 times what they take).
__device__ __forceinline__ void att_drain(uint64_t* bar, uint32_t parity) {
    const unsigned long long until = globaltimer_ns() + 2000000000ull;
    while (!mbar_try_wait(bar, parity) && globaltimer_ns() < until) {}
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
    const int len = c.length()[s], held = c.held()[s], mine = c.table(s)[i], theirs = c.table(p.a.shared_stream)[i];
    return (len >= shared) & (held > i) & (mine == theirs);
}
__device__ __forceinline__ int att_shared(const CacheView& c, const AttendParams& p) {
    const int n = p.a.shared_tokens;
    if (n <= 0) return 0;
    const int len = c.length()[p.a.shared_stream], held = c.held()[p.a.shared_stream];
    return (len >= n) & (held >= (n >> c.page_shift)) ? n : 0;
}

__device__ __forceinline__ OwnUnit att_unit(const CacheView& c, const AttendParams& p, int unit, int shared) {
    OwnUnit w{0, 0, 0, 0, 0};
    const int s = unit / p.U;
    if (s >= p.a.streams) return w;
    w.r0 = (unit - s * p.U) * p.rows_own();
    const int ctx = att_ctx(c, s), used = att_used(p, s), rows = used * p.G;   // (loads side by side)
    const bool shares = att_shares(c, p, s, shared);
    if (w.r0 >= rows) return w;
    w.nrows = min(p.rows_own(), rows - w.r0);
    w.ctx = ctx;
    w.end = ctx + (p.a.mask_dev ? used : (w.r0 + w.nrows - 1) / p.G + 1);
    w.begin = shares ? shared : 0;
    return w;
}

// W1: places of one head's own jobs (with this list's padding).
__device__ __forceinline__ JobList att_list(const CacheView& c, const AttendParams& p, bool wide, int shared, int W1, int grid) {
    JobList L;
    L.pad = wide ? kPadWide : kPadNarrow;
    L.has_own = (p.wide_own != 0) == wide;
    L.tiles_sh = (shared + kKeyTile - 1) / kKeyTile;
    L.W_sh = shared > 0 && (p.wide_sh != 0) == wide ? c.Hkv * p.U_sh * (L.tiles_sh + L.pad) : 0;
    L.W1 = L.has_own ? W1 : 0;
    L.W = L.W_sh + c.Hkv * L.W1;
    L.workers = min(wide ? grid : 2 * grid, L.W);                // none of them without a place
    L.q = L.workers ? L.W / L.workers : 0;
    L.rem = L.W - L.q * L.workers;
    return L;
}

// Exclusive prefix over the CTA's threads of a value per thread, and the sum.
template <int D>
__device__ __forceinline__ int att_scan(AttSmem<D>& sm, int v, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sm.sums[3][warp] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kAttThreads / 32; ++w) {
        if (w < warp) before += sm.sums[3][w];
        all += sm.sums[3][w];
    }
    *total = all;
    __syncthreads();
    return before + x - v;
}

// Shared tokens in use and the places of one head's own jobs; writes what the merge needs, and
// where each slot's own jobs begin.
struct Schedule {
    int shared, W1;
};
template <int D>
__device__ Schedule att_schedule(const CacheView& c, const AttendParams& p, AttSmem<D>& sm) {
    Schedule sc;
    const int units = p.a.streams * p.U, tid = threadIdx.x, pad = p.wide_own ? kPadWide : kPadNarrow;
    const int shared = att_shared(c, p);
    // places of one head's own jobs with and without the shared pass, and the streams that share
    int sum[3] = {0, 0, 0}, mine[2] = {0, 0};
    OwnUnit u{0, 0, 0, 0, 0};                  // (u, mine: of unit `tid`)
    for (int i = tid; i < units; i += kAttThreads) {
        const OwnUnit w = att_unit(c, p, i, shared);
        if (w.nrows == 0) continue;
        const int with = w.tiles() + pad, without = (w.end + kKeyTile - 1) / kKeyTile + pad;
        sum[0] += with;
        sum[1] += without;
        sum[2] += w.r0 == 0 && w.begin > 0;
        if (i == tid) {
            mine[0] = with;
            mine[1] = without;
            u = w;
        }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const int x = __reduce_add_sync(0xFFFFFFFFu, sum[k]);
        if ((tid & 31) == 0) sm.sums[k][tid >> 5] = x;
        sum[k] = 0;
    }
    if (tid < 2) {
        sm.first_unit[tid] = 0;
        sm.first_off[tid] = 0;
        sm.first_own[tid].nrows = 0;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAttThreads / 32; ++w)
#pragma unroll
        for (int k = 0; k < 3; ++k) sum[k] += sm.sums[k][w];
    const bool share = sum[2] > 1;             // one stream alone reads all through its own table
    sc.shared = share ? shared : 0;
    sc.W1 = share ? sum[0] : sum[1];
    // the unit, and the place in it, where each slot's own jobs begin
    const JobList L = att_list(c, p, p.wide_own != 0, sc.shared, sc.W1, gridDim.x);
    if (tid == 0) {
        sm.list[p.wide_own] = L;
        sm.list[p.wide_own ^ 1] = att_list(c, p, !p.wide_own, sc.shared, sc.W1, gridDim.x);
    }
    int y[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int w = p.wide_own ? blockIdx.x : x * gridDim.x + blockIdx.x, at = w < L.workers ? L.first(w) : 0;
        const int h = at > L.W_sh ? (at - L.W_sh) / L.W1 : 0;
        y[x] = at > L.W_sh ? at - L.W_sh - h * L.W1 : 0;
        if (tid == 0) sm.first_h[x] = h;
    }
    if (blockIdx.x == 0 || y[0] > 0 || y[1] > 0) {
        int at = 0;
        for (int i0 = 0; i0 < units; i0 += kAttThreads) {
            const int i = i0 + tid;
            int n = mine[share ? 0 : 1];
            if (i0 > 0) {                      // (units behind the first pass are read again)
                u = i < units ? att_unit(c, p, i, sc.shared) : OwnUnit{0, 0, 0, 0, 0};
                n = u.nrows > 0 ? u.tiles() + pad : 0;
            }
            if (!share) u.begin = 0;
            int all;
            const int x0 = at + att_scan(sm, n, &all);
#pragma unroll
            for (int x = 0; x < 2; ++x)
                if (n > 0 && x0 <= y[x] && y[x] < x0 + n) {
                    sm.first_unit[x] = i;
                    sm.first_off[x] = y[x] - x0;
                    sm.first_own[x] = u;
                }
            if (blockIdx.x == 0 && i < units) p.units[i] = make_int4(x0, u.nrows, n - pad, u.begin > 0);
            at += all;
        }
    }
    __syncthreads();
    if (blockIdx.x == 0 && tid < 2) p.head[tid] = sm.list[tid];
    return sc;
}

// Partial rows of a part of a job: rows run fastest, then the columns in fours; the logarithms of
// the sums are behind them.
struct Slot {
    float* base;
    int R;
};
template <int D>
__device__ __forceinline__ Slot att_slot(const AttendParams& p, bool wide, bool own, int job, int worker, bool whole, bool first) {
    if (!whole) {                              // at most one part of a job it does not begin and one that it does
        const int R = wide ? 256 : 128;
        return {(wide ? p.split_wide : p.split_narrow) + (2 * (int64_t)worker + (first ? 1 : 0)) * R * (D + 1), R};
    }
    const int R = own ? p.R_own : p.rows_sh();
    return {(own ? p.whole_own : p.whole_sh) + (int64_t)job * R * (D + 1), R};
}

// A producer warp's walk over the segments of one list; all lanes hold the same values but `n`.
struct Walk {
    int v, end;                // places
    int h, unit, off;
    int base, n;               // tiles of the units base + lane
    bool known;                // the first unit has been looked up
};
template <int D>
__device__ __forceinline__ Walk att_walk(const JobList& L, const AttSmem<D>& sm, int slot, int worker) {
    Walk w;
    w.v = worker < L.workers ? L.first(worker) : 0;
    w.end = worker < L.workers ? L.first(worker + 1) : 0;
    w.h = 0;
    w.unit = 0;
    w.off = 0;
    w.known = false;
    if (L.has_own && w.v >= L.W_sh && w.v < w.end) {
        w.h = sm.first_h[slot];
        w.unit = sm.first_unit[slot];
        w.off = sm.first_off[slot];
        w.known = sm.first_own[slot].nrows > 0;
    }
    w.base = -1;
    w.n = 0;
    return w;
}
template <int D>
__device__ bool att_next(const CacheView& c, const AttendParams& p, const Schedule& sc, const JobList& L, const AttSmem<D>& sm,
                         bool wide, int slot, int worker, Walk& w, Segment& sg) {
    for (;;) {
        if (w.v >= w.end) return false;
        int n, begin, o0, job;                 // tiles of the job, first key; first place of it here
        if (w.v < L.W_sh) {
            job = w.v / (L.tiles_sh + L.pad);
            o0 = w.v - job * (L.tiles_sh + L.pad);
            n = L.tiles_sh;
            begin = 0;
            sg.own = 0;
            sg.h = job / p.U_sh;
            sg.r0 = (job - sg.h * p.U_sh) * p.rows_sh();
            sg.nrows = min(p.rows_sh(), p.a.streams * p.a.block * p.G - sg.r0);
            sg.s = p.a.shared_stream;
            sg.key_end = sg.ctx = sc.shared;
        } else {
            const int units = p.a.streams * p.U, lane = threadIdx.x & 31;
            while (!w.known) {                 // the next unit with tiles
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
            const OwnUnit u = w.known ? sm.first_own[slot] : att_unit(c, p, w.unit, sc.shared);
            w.known = false;
            n = u.tiles();
            begin = u.begin;
            o0 = w.off;
            job = w.h * units + w.unit;
            sg.own = 1;
            sg.h = w.h;
            sg.s = w.unit / p.U;
            sg.r0 = u.r0;
            sg.nrows = u.nrows;
            sg.key_end = u.end;
            sg.ctx = u.ctx;
            w.off = 0;
            ++w.unit;
        }
        const int o1 = min(L.pad + n, o0 + (w.end - w.v));
        w.v += o1 - o0;
        const int t0 = max(o0 - L.pad, 0), t1 = max(o1 - L.pad, 0);
        if (t1 <= t0) continue;                // places without a tile
        const bool whole = t1 - t0 == n;
        const Slot to = att_slot<D>(p, wide, sg.own, job, worker, whole, t0 == 0);
        sg.out = whole && sg.own && begin == 0 ? nullptr : to.base;
        sg.R = to.R;
        sg.out_row = wide ? 128 * slot : 0;
        sg.r0 += sg.out_row;
        sg.nrows = min(128, sg.nrows - sg.out_row);
        sg.wide = wide;
        sg.key0 = begin + t0 * kKeyTile;
        sg.T = t1 - t0;
        return true;
    }
}

// ---- producer ------------------------------------------------------------------------------

// The ring of a list's tiles: K and V of each tile in turn.
template <int D>
struct Ring {
    AttSmem<D>* sm;
    int wide, first, stages, log;                            // stages = 2^log
    __device__ Ring(AttSmem<D>& s, bool w, int slot)
        : sm(&s), wide(w), first(w ? 0 : slot * (AttSmem<D>::kStages / 2)), stages(w ? AttSmem<D>::kStages : AttSmem<D>::kStages / 2),
          log((AttSmem<D>::kStages == 4 ? 2 : 3) - (w ? 0 : 1)) {}
    __device__ int stage(uint32_t i) const { return first + (int)(i & (stages - 1)); }
    __device__ uint32_t round(uint32_t i) const { return (i >> log) & 1; }
    __device__ uint64_t* full(uint32_t i) const { return &sm->full[wide ? 0 : 1][stage(i)]; }
    __device__ uint64_t* empty(uint32_t i) const { return &sm->empty[wide ? 0 : 1][stage(i)]; }
};

// Limit of a wait for work on `tiles` tiles (of K or V) that are under way.
__device__ __forceinline__ unsigned long long att_limit(const AttendParams& p, uint32_t tiles) { return p.timeout_ns + 10000ull * tiles; }

// Makes a segment known to the slot's other warps.
template <int D>
__device__ __forceinline__ bool att_publish(const AttendParams& p, AttSmem<D>& sm, int slot, const Segment& sg, uint32_t tiles) {
    const int e = sg.no & 1;
    if (!att_warp_wait(&sm.sege[slot][e], ((sg.no >> 1) & 1) ^ 1, &sm.abort, att_limit(p, tiles))) return false;
    if ((threadIdx.x & 31) == 0) {
        sm.seg[slot][e] = sg;
        mbar_arrive(&sm.segf[slot][e]);
    }
    __syncwarp();
    return true;
}

// One list.  Returns false when a wait gave up; *n: tiles of the ring.
template <int D>
__device__ bool att_produce(const CacheView& c, const AttendParams& p, const Schedule& sc, AttSmem<D>& sm, const CUtensorMap* kmap,
                            const CUtensorMap* vmap, bool wide, int slot, Segment& sg, uint32_t& n) {
    using SM = AttSmem<D>;
    const int lane = threadIdx.x & 31, per_tile = kKeyTile >> c.page_shift;
    const JobList L = sm.list[wide];
    const int worker = wide ? blockIdx.x : slot * gridDim.x + blockIdx.x;
    const bool loads = !wide || slot == 0;
    const Ring<D> ring(sm, wide, slot);
    Walk w = att_walk<D>(L, sm, slot, worker);
    while (att_next<D>(c, p, sc, L, sm, wide, slot, worker, w, sg)) {
        const int* table = c.table(sg.s);
        const int pages = min(min(c.held()[sg.s], c.L.M), (sg.key_end + c.page - 1) >> c.page_shift);
        // the page that this lane copies of a tile; outside the pool (zeros) where there is none
        const auto page_of = [&](int t) {
            const int i = ((sg.key0 + t * kKeyTile) >> c.page_shift) + lane;
            const int id = lane < per_tile && t < sg.T && i < pages ? table[i] : -1;
            return (unsigned)id < (unsigned)c.L.P ? id : c.L.P;
        };
        int id = page_of(0);
        if (!att_publish<D>(p, sm, slot, sg, n)) return false;
        ++sg.no;
        sg.wide_no += wide;
        if (!loads) {
            n += 2 * sg.T;
            continue;
        }
        for (int t = 0; t < sg.T; ++t) {
            const int next = page_of(t + 1);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv, ++n) {
                if (!att_warp_wait(ring.empty(n), ring.round(n) ^ 1, &sm.abort, p.timeout_ns)) return false;
                uint64_t* full = ring.full(n);
                if (lane == 0) mbar_arrive_expect_tx(full, SM::kTileBytes);
                __syncwarp();
                if (lane < per_tile) {
                    const uint32_t dst = smem_u32(sm.kv[ring.stage(n)]) + lane * c.page * 128;
#pragma unroll
                    for (int x = 0; x < D / 64; ++x)
                        tma_load_3d(dst + x * SM::kPanel, kv ? vmap : kmap, 64 * x, sg.h * c.page, id, full);
                }
            }
            id = next;
        }
    }
    return true;
}

template <int D>
__device__ void att_producer(const CacheView& c, const AttendParams& p, const Schedule& sc, AttSmem<D>& sm, const CUtensorMap* kmap,
                             const CUtensorMap* vmap, int slot) {
    Segment sg;
    sg.no = sg.wide_no = 0;
    uint32_t nw = 0, nn = 0;
    const Ring<D> wide(sm, true, slot), narrow(sm, false, slot);
    const auto used_up = [&](const Ring<D>& ring, uint32_t n) {   // all tiles of a ring
        for (uint32_t i = n > (uint32_t)ring.stages ? n - ring.stages : 0; i < n; ++i)
            if (!att_warp_wait(ring.empty(i), ring.round(i), &sm.abort, p.timeout_ns)) return false;
        return true;
    };
    // Wide jobs keep the tensor core busy, narrow ones the memory: half of the CTAs begin with one
    // kind and half with the other (64 streams behind 32768 keys: 445 -> 410 us).  The rings share
    // their stages, so one kind's tiles are all used up before the other's are copied.
    bool ok = true;
    for (int phase = 0; phase < 2 && ok; ++phase) {
        const bool is_wide = (phase ^ blockIdx.x & 1) == 0;
        if (sm.list[is_wide].W == 0) continue;
        uint32_t& n = is_wide ? nw : nn;
        ok = att_produce<D>(c, p, sc, sm, kmap, vmap, is_wide, slot, sg, n);
        if (phase == 1 || !ok) break;
        // The warp that copied the last tiles waits for their ring (the other one has not followed its
        // phases) and tells the other: slot 0 after the wide jobs; after the narrow ones slot 1 tells
        // slot 0, which then copies into both.
        if (!is_wide || slot == 0) ok = used_up(is_wide ? wide : narrow, n);
        if (slot == (is_wide ? 0 : 1)) {
            if (ok && (threadIdx.x & 31) == 0) mbar_arrive(&sm.handover);
            __syncwarp();
        } else {
            ok = ok && att_warp_wait(&sm.handover, 0, &sm.abort, att_limit(p, n));
        }
    }
    sg.T = 0;
    if (ok) att_publish<D>(p, sm, slot, sg, nw + nn);
    // Every copy has landed before the CTA leaves, also where another warp gives up after this one is done.
    if (slot == 0)
        for (uint32_t i = nw > (uint32_t)wide.stages ? nw - wide.stages : 0; i < nw; ++i) att_drain(wide.full(i), wide.round(i));
    for (uint32_t i = nn > (uint32_t)narrow.stages ? nn - narrow.stages : 0; i < nn; ++i) att_drain(narrow.full(i), narrow.round(i));
}

// ---- MMA -------------------------------------------------------------------------------------

// Rows of a V tile that no product may see: positions behind the unit's keys become zero, and so
// do non-finite elements at block positions, which some rows may not see (0 x NaN is NaN); the
// epilogue adds those to the rows that do see them.  Whole warp; true in every lane when there
// were any.
template <int D, bool kBf16>
__device__ __noinline__ bool att_mend_v(uint8_t* tile, int from, int end) {
    const int lane = threadIdx.x & 31;
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
    fence_proxy_async_shared();
    __syncwarp();
    return __any_sync(0xFFFFFFFFu, bad);
}

template <int D, bool kBf16>
__device__ void att_mma(const AttendParams& p, AttSmem<D>& sm, uint32_t tmem, int slot) {
    using SM = AttSmem<D>;
    constexpr uint32_t idesc_s = idesc_f16(128, 128, kBf16, false), idesc_o = idesc_f16(128, D, kBf16, true);
    const bool issues = elect_one();
    const uint32_t ts = tmem + kTmemS + 128 * slot, to = tmem + kTmemO + 128 * slot, q = smem_u32(sm.q[slot]);
    uint32_t used_wide = 0, used_narrow = 0, np = 0, turns = 0, mends = 0;   // mends: a bit per stage
    const auto wait = [&](uint64_t* bar, uint32_t parity) { return att_warp_wait(bar, parity, &sm.abort, p.timeout_ns); };
    uint32_t tiles = 0;                                    // so far
    for (int no = 0;; ++no) {
        if (!att_warp_wait(&sm.segf[slot][no & 1], (no >> 1) & 1, &sm.abort, att_limit(p, tiles))) return;
        const Segment& sg = sm.seg[slot][no & 1];
        tiles += 2 * sg.T;
        const int T = uniform(sg.T), wide = uniform(sg.wide), key0 = uniform(sg.key0), ctx = uniform(sg.ctx);
        const int key_end = uniform(sg.key_end), wide_no = uniform(sg.wide_no);
        if (issues) mbar_arrive(&sm.sege[slot][no & 1]);
        if (T == 0) return;
        const Ring<D> ring(sm, wide, slot);
        uint32_t n = wide ? used_wide : used_narrow;       // (next tile of the ring)
        if (wide) used_wide += 2 * T;
        else used_narrow += 2 * T;
        const auto scores = [&]() {                        // S of the tile whose K is tile n of the ring
            if (!wait(ring.full(n), ring.round(n))) return false;
            tc_fence_after();
            if (issues) {
                const uint32_t k = smem_u32(sm.kv[ring.stage(n)]);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint32_t o = (i / 4) * SM::kPanel + (i % 4) * 32;
                    tc_mma_f16_ss(ts, smem_desc_sw128(q + o), smem_desc_sw128(k + o), idesc_s, i > 0);
                }
                tc_commit(&sm.sfull[slot]);
                tc_commit(ring.empty(n));
            }
            __syncwarp();
            return true;
        };
        // Wide units: the slots take turns, each with the products of a step in one go, so that one
        // slot's scores are ready while the other's products run (interleaved, both would wait for all:
        // 473 us instead of 450 for 64 streams behind 32768 keys).
        const auto begin_turn = [&]() { return !wide || wait(&sm.turn[slot], (turns & 1) ^ (slot == 0)); };
        const auto end_turn = [&]() {
            if (!wide) return;
            ++turns;
            if (issues) mbar_arrive(&sm.turn[slot ^ 1]);
            __syncwarp();
        };
        if (!wait(&sm.qfull[slot], no & 1)) return;
        if (!begin_turn() || !scores()) return;
        end_turn();
        for (int t = 0; t < T; ++t, ++n) {
            ++n;                                           // V of tile t
            if (!wait(ring.full(n), ring.round(n))) return;
            const int st = ring.stage(n), j0 = key0 + t * kKeyTile;
            if (j0 + kKeyTile > ctx) {                     // block positions, or the end of the keys
                if (!wide || slot == 0) {
                    const bool bad = att_mend_v<D, kBf16>(sm.kv[st], min(max(ctx - j0, 0), kKeyTile), min(max(key_end - j0, 0), kKeyTile));
                    if (issues) {
                        if (bad) {
                            *reinterpret_cast<volatile int*>(wide ? &sm.bad_wide[wide_no % kWideMarks] : &sm.bad_value[slot]) =
                                (wide ? wide_no : no) + 1;
                            __threadfence_block();
                        }
                        if (wide) mbar_arrive(&sm.mended[st]);
                    }
                    __syncwarp();
                } else {
                    if (!wait(&sm.mended[st], mends >> st & 1)) return;
                    mends ^= 1u << st;
                }
            }
            const uint32_t v = smem_u32(sm.kv[st]);
            if (!wait(&sm.phalf[slot], np & 1) || !begin_turn()) return;
            tc_fence_after();
            if (issues) {
#pragma unroll
                for (int i = 0; i < kKeyTile / 32; ++i)
                    tc_mma_f16_ts(to, ts + 8 * i, smem_desc_mn_sw128(v + i * 2048, SM::kPanel), idesc_o, t > 0 || i > 0);
            }
            __syncwarp();
            if (!wait(&sm.pfull[slot], np++ & 1)) return;
            tc_fence_after();
            if (issues) {
#pragma unroll
                for (int i = kKeyTile / 32; i < kKeyTile / 16; ++i)
                    tc_mma_f16_ts(to, ts + 8 * i, smem_desc_mn_sw128(v + i * 2048, SM::kPanel), idesc_o, 1);
                tc_commit(ring.empty(n));
                if (t + 1 == T) tc_commit(&sm.ofull[slot]);
            }
            __syncwarp();
            if (t + 1 < T) {
                ++n;
                if (!scores()) return;
                --n;
            }
            end_turn();
        }
    }
}

// ---- softmax ---------------------------------------------------------------------------------

// A row of a segment: its token (stream * block + position) and query head.
struct Row {
    int64_t tok;
    int b, head;
    bool valid;
};
__device__ __forceinline__ Row att_row(const CacheView& c, const AttendParams& p, int shared, const Segment& sg, int r) {
    Row x;
    const int i = sg.r0 + r, q = i / p.G;
    x.head = sg.h * p.G + (i - q * p.G);
    x.valid = r < sg.nrows;
    x.b = q;
    x.tok = q;
    if (sg.own) {
        x.tok += (int64_t)sg.s * p.a.block;
    } else if (x.valid) {
        const int s = q / p.a.block;
        x.b = q - s * p.a.block;
        x.valid = x.b < att_used(p, s) && att_shares(c, p, s, shared);
    }
    return x;
}

// The query rows of a segment into its Q tile (128-byte swizzle), zeros behind them.  128 threads;
// 16-byte chunks of a row on neighbouring lanes.
template <int D>
__device__ __forceinline__ void att_load_q(const AttendParams& p, const Segment& sg, uint8_t* tile) {
    constexpr int kChunks = D / 8;
    const int tid = threadIdx.x & 127, x = tid % kChunks;
    const uint16_t* q = static_cast<const uint16_t*>(p.a.q_dev) + x * 8;
    const int64_t tok0 = sg.own ? (int64_t)sg.s * p.a.block : 0;
    const int nrows = sg.nrows, t0 = sg.r0 / p.G, g0 = sg.r0 - t0 * p.G;     // first row's token and head
    q += (tok0 + t0) * p.a.q_stride + (int64_t)sg.h * p.G * D;
    uint4 v[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int row = tid / kChunks + i * (128 / kChunks), g = g0 + row, t = p.div_g(g);
        v[i] = load_or_zero(q + t * p.a.q_stride + (g - t * p.G) * D, row < nrows);
    }
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int row = tid / kChunks + i * (128 / kChunks);
        *reinterpret_cast<uint4*>(tile + (x / 8) * AttSmem<D>::kPanel + row * 128 + (((x & 7) ^ (row & 7)) << 4)) =
            make_uint4(v[i].x ^ p.q_flip, v[i].y ^ p.q_flip, v[i].z ^ p.q_flip, v[i].w ^ p.q_flip);
    }
}

// Bit i: the row sees key j0 + i.
__device__ __forceinline__ void att_visible(bool masked, int ctx, int key_end, int lim, uint64_t bits, int j0, uint32_t (&vis)[4]) {
    const int n = min(max(lim - j0, 0), kKeyTile);                                       // keys below lim are seen
    uint64_t lo = n >= 64 ? ~0ull : (1ull << n) - 1, hi = n >= 128 ? ~0ull : n > 64 ? (1ull << (n - 64)) - 1 : 0ull;
    if (masked) {
        const int len = key_end - ctx;                                                   // block positions, at most 64
        bits &= len >= 64 ? ~0ull : (1ull << len) - 1;
        const int at = ctx - j0;                                                         // of block position 0 in the tile
        if (at <= -64 || at >= kKeyTile) bits = 0;
        else if (at < 0) lo |= bits >> -at;
        else if (at < 64) { lo |= bits << at; if (at) hi |= bits >> (64 - at); }
        else hi |= bits << (at - 64);
    }
    vis[0] = (uint32_t)lo; vis[1] = (uint32_t)(lo >> 32); vis[2] = (uint32_t)hi; vis[3] = (uint32_t)(hi >> 32);
}

// Columns of a row whose values at the block positions that it sees are not all finite, which the
// products left out: any sum with one is not finite either, and is the sum of those alone (NaN, or
// infinities of one sign, or of both: NaN).  Whole warp: each key's row of values is one load of the
// warp's, eight keys at a time; a lane keeps for its own query row a bit per column for either sign
// (bit l of word e: column l D/32 + e).  16384 positions of 8 heads of 128 take 1.6 ms, with a bad
// value every 64 positions 3.7; with a lane that reads its own row's columns one by one, the waits
// of the other warps ran out (200 ms).  2048 of 64 heads: 0.27 and 0.60 ms, against 166.
template <int D, bool kBf16>
__device__ __noinline__ void att_put_bad(const CacheView& c, const AttendParams& p, const Segment& sg, bool valid, int b, uint64_t bits,
                                         int64_t at, int r, float inv) {
    constexpr int kE = D / 32, kKeys = 8;                        // elements of a lane; keys under way together
    constexpr uint32_t kExp = kBf16 ? 0x7F80u : 0x7C00u, kMan = kBf16 ? 0x007Fu : 0x03FFu;
    const int lane = threadIdx.x & 31, from = max(sg.ctx, sg.key0), end = min(sg.key_end, sg.key0 + sg.T * kKeyTile);
    const int held = min(c.held()[sg.s], c.L.M);
    const int* table = c.table(sg.s);
    uint32_t pos[kE] = {}, neg[kE] = {};
    for (int pi = from >> c.page_shift; pi << c.page_shift < end && pi < held; ++pi) {
        const int page = table[pi];
        if ((unsigned)page >= (unsigned)c.L.P) continue;
        const int j1 = min(end, (pi + 1) << c.page_shift);
        const uint16_t* base = p.v_pool + page * c.page_stride + (int64_t)sg.h * c.page * D + lane * kE;
        for (int j0 = max(from, pi << c.page_shift); j0 < j1; j0 += kKeys) {
            uint32_t v[kKeys][kE / 2];
            bool hit = false;
#pragma unroll
            for (int k = 0; k < kKeys; ++k) {
                const uint32_t* row = reinterpret_cast<const uint32_t*>(base + (int64_t)((j0 + k) & (c.page - 1)) * D);
#pragma unroll
                for (int x = 0; x < kE / 2; ++x) v[k][x] = j0 + k < j1 ? row[x] : 0u;
            }
#pragma unroll
            for (int k = 0; k < kKeys; ++k)
#pragma unroll
                for (int x = 0; x < kE / 2; ++x) hit |= (v[k][x] & kExp) == kExp || (v[k][x] >> 16 & kExp) == kExp;
            if (!__any_sync(0xFFFFFFFFu, hit)) continue;
#pragma unroll
            for (int k = 0; k < kKeys; ++k) {
                const int i = j0 + k - sg.ctx;                   // block position
                const bool sees = valid && j0 + k < j1 && (p.a.mask_dev ? bits >> i & 1 : i <= b);
#pragma unroll
                for (int e = 0; e < kE; ++e) {
                    const uint32_t u = v[k][e / 2] >> 16 * (e & 1);
                    const bool bad = (u & kExp) == kExp, nan = (u & kMan) != 0;
                    const uint32_t plus = __ballot_sync(0xFFFFFFFFu, bad && (nan || !(u & 0x8000u)));
                    const uint32_t minus = __ballot_sync(0xFFFFFFFFu, bad && (nan || (u & 0x8000u)));
                    if (sees) {
                        pos[e] |= plus;
                        neg[e] |= minus;
                    }
                }
            }
        }
    }
#pragma unroll
    for (int e = 0; e < kE; ++e)
        for (uint32_t any = pos[e] | neg[e]; any; any &= any - 1) {
            const int l = __ffs(any) - 1, col = l * kE + e;
            const bool plus = pos[e] >> l & 1, minus = neg[e] >> l & 1;
            const float sum = (plus && minus ? NAN : plus ? INFINITY : -INFINITY) * inv;
            if (sg.out) sg.out[((col / 4) * sg.R + r) * 4 + col % 4] = sum;
            else static_cast<uint16_t*>(p.a.out_dev)[at * D + col] = (uint16_t)pack_f16<kBf16>(sum, 0.0f);
        }
}

template <int D, bool kBf16>
__device__ void att_softmax(const CacheView& c, const AttendParams& p, int shared, AttSmem<D>& sm, uint32_t tmem) {
    const int slot = threadIdx.x >> 7, tid = threadIdx.x & 127, lane = threadIdx.x & 31;
    const uint32_t lanes = (uint32_t)(tid & ~31) << 16;          // this warp's quarter of the tensor memory
    const uint32_t ts = tmem + kTmemS + 128 * slot + lanes, to = tmem + kTmemO + 128 * slot + lanes;
    uint32_t ns = 0;
    const auto wait = [&](uint64_t* bar, uint32_t parity) { return att_warp_wait(bar, parity, &sm.abort, p.timeout_ns); };
    uint32_t tiles = 0;                                          // so far
    for (int no = 0;; ++no) {
        if (!att_warp_wait(&sm.segf[slot][no & 1], (no >> 1) & 1, &sm.abort, att_limit(p, tiles))) return;
        const Segment& sg = sm.seg[slot][no & 1];
        const int T = sg.T;
        if (T == 0) return;
        tiles += 2 * T;
        // the query rows; the products that read the last ones have completed (ofull, below)
        att_load_q<D>(p, sg, sm.q[slot]);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.qfull[slot]);
        const Row row = att_row(c, p, shared, sg, tid);
        const bool busy = __any_sync(0xFFFFFFFFu, row.valid);
        const bool masked = sg.own && p.a.mask_dev;
        const uint64_t bits = masked && row.valid ? p.a.mask_dev[row.tok] : 0;
        const int lim = !sg.own ? sg.key_end : masked ? sg.ctx : sg.ctx + row.b + 1;
        float m = -INFINITY, l = 0.0f;
        int j0 = sg.key0;
        const int tail = sg.ctx - kKeyTile;                      // tiles from behind here on have hidden keys
        for (int t = 0; t < T; ++t, j0 += kKeyTile) {
            if (!wait(&sm.sfull[slot], ns++ & 1)) return;
            tc_fence_after();
            if (busy) {
                uint32_t x[4][32], vis[4];
                const bool hidden = j0 > tail;
                if (hidden) att_visible(masked, sg.ctx, sg.key_end, lim, bits, j0, vis);
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                tc_ld_x32(ts, x[0]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {                    // the next 32 keys load while these are looked over
                    tc_wait_ld(x[k]);
                    if (k < 3) tc_ld_x32(ts + 32 * (k + 1), x[k < 3 ? k + 1 : 3]);
                    if (hidden)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(vis[k] >> e & 1)) x[k][e] = 0xFF800000u;
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        mx[(e / 2) & 3] = max3(mx[(e / 2) & 3], __uint_as_float(x[k][e]), __uint_as_float(x[k][e + 1]));
                }
                const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * p.c;
                const bool passed = m != -INFINITY && top > m + (att_below<kBf16>(m) + kRescale<kBf16>);
                if (__any_sync(0xFFFFFFFFu, passed)) {
                    const float f = passed ? exp2_approx(m - (top - att_below<kBf16>(top))) : 1.0f;
                    l *= f;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        uint32_t o[16];
                        tc_ld_x16(to + 16 * k, o);
                        tc_wait_ld(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tc_st_x16(to + 16 * k, o);
                    }
                }
                if (passed || m == -INFINITY) m = top - att_below<kBf16>(top);
                const float ref = m == -INFINITY ? 0.0f : m;
                float sum[4][2] = {};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float a, b;
                        fma_x2(a, b, __uint_as_float(x[k][e]), __uint_as_float(x[k][e + 1]), p.c, -ref);
                        a = exp2_approx(a);
                        b = exp2_approx(b);
                        add_x2(sum[(e / 2) & 3][0], sum[(e / 2) & 3][1], a, b);
                        pk[e / 2] = pack_f16<kBf16>(a, b);
                    }
                    tc_st_x16(ts + 16 * k, pk);
                    if (k == 1) {                                // the first half of the keys can go
                        tc_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm.phalf[slot]);
                    }
                }
                l += ((sum[0][0] + sum[0][1]) + (sum[1][0] + sum[1][1])) + ((sum[2][0] + sum[2][1]) + (sum[3][0] + sum[3][1]));
                tc_wait_st();
            } else if (lane == 0) {
                mbar_arrive(&sm.phalf[slot]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.pfull[slot]);
        }
        // the rows, out of tensor memory
        if (!wait(&sm.ofull[slot], no & 1)) return;
        tc_fence_after();
        if (busy) {
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const float lse2 = l == 0.0f ? -INFINITY : m + log2f(l);
            const bool mend = sg.own && *reinterpret_cast<volatile int*>(sg.wide ? &sm.bad_wide[sg.wide_no % kWideMarks]
                                                                                 : &sm.bad_value[slot]) ==
                                            (sg.wide ? sg.wide_no : no) + 1;
            float* const out = sg.out;
            const int R = sg.R, r = sg.out_row + tid;
            const int64_t at = row.tok * p.a.q_heads + row.head;
#pragma unroll
            for (int col = 0; col < D; col += 64) {
                uint32_t y[2][32];
                tc_ld_x32(to + col, y[0]);
                tc_ld_x32(to + col + 32, y[1]);
                tc_wait_ld(y[0]);
                tc_wait_ld(y[1]);
                const auto f = [&](int e) { return __uint_as_float(y[e / 32][e % 32]) * inv; };
                if (row.valid && !out) {
                    uint4* to_row = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.a.out_dev) + at * D + col);
#pragma unroll
                    for (int e = 0; e < 64; e += 8)
                        to_row[e / 8] = make_uint4(pack_f16<kBf16>(f(e), f(e + 1)), pack_f16<kBf16>(f(e + 2), f(e + 3)),
                                                   pack_f16<kBf16>(f(e + 4), f(e + 5)), pack_f16<kBf16>(f(e + 6), f(e + 7)));
                } else if (row.valid) {
                    float4* to_slot = reinterpret_cast<float4*>(out) + (col / 4) * R + r;
#pragma unroll
                    for (int e = 0; e < 64; e += 4) to_slot[(e / 4) * R] = make_float4(f(e), f(e + 1), f(e + 2), f(e + 3));
                }
                __syncwarp();
            }
            if (__any_sync(0xFFFFFFFFu, mend)) att_put_bad<D, kBf16>(c, p, sg, row.valid, row.b, bits, at, r, inv);
            if (row.valid) {
                if (out) out[(int64_t)R * D + r] = lse2;
                else if (p.a.lse_dev) p.a.lse_dev[at] = lse2 * 0.693147180559945309f;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.sege[slot][no & 1]);
    }
}

template <int D, bool kBf16>
__global__ void __launch_bounds__(kAttThreads, 1) attend_kernel(const CacheView c, const AttendParams p,
                                                                const __grid_constant__ CUtensorMap kmap,
                                                                const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ __align__(1024) uint8_t raw[];       // the only shared memory: its tiles are 1024-byte aligned
    AttSmem<D>& sm = *reinterpret_cast<AttSmem<D>*>(raw);
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < AttSmem<D>::kStages; ++i) {
            mbar_init(&sm.full[0][i], 1);
            mbar_init(&sm.full[1][i], 1);
            mbar_init(&sm.empty[0][i], 2);                 // both slots' MMA warps
            mbar_init(&sm.empty[1][i], 1);
            mbar_init(&sm.mended[i], 1);
        }
        for (int x = 0; x < 2; ++x) {
            for (int e = 0; e < 2; ++e) {
                mbar_init(&sm.segf[x][e], 1);
                mbar_init(&sm.sege[x][e], 5);              // MMA warp, softmax warps
            }
            mbar_init(&sm.turn[x], 1);
            mbar_init(&sm.qfull[x], 4);
            mbar_init(&sm.sfull[x], 1);
            mbar_init(&sm.phalf[x], 4);
            mbar_init(&sm.pfull[x], 4);
            mbar_init(&sm.ofull[x], 1);
            mbar_init(&sm.drain[x], 1);
            sm.bad_value[x] = 0;
        }
        mbar_init(&sm.handover, 1);
        for (int i = 0; i < kWideMarks; ++i) sm.bad_wide[i] = 0;
        sm.abort = 0;
        fence_barrier_init();
    }
    if (warp == kAttMma) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    grid_dependency_wait();
    const Schedule sc = att_schedule<D>(c, p, sm);         // ends with a CTA barrier
    tc_fence_after();
    grid_dependency_launch();
    const uint32_t tmem = uniform(sm.tmem);
    if (warp < 8) {
        reg_grow<216>();
        att_softmax<D, kBf16>(c, p, sc.shared, sm, tmem);
    } else {
        reg_shrink<72>();
        if (warp < kAttMma) {
            if (lane == 0) {
                prefetch_tensormap(&kmap);
                prefetch_tensormap(&vmap);
            }
            att_producer<D>(c, p, sc, sm, &kmap, &vmap, warp - kAttProducer);
        } else {
            const int slot = warp - kAttMma;
            att_mma<D, kBf16>(p, sm, tmem, slot);
            if (elect_one()) {                             // every product has completed before the memory is freed
                tc_commit(&sm.drain[slot]);
                att_drain(&sm.drain[slot], 0);
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

constexpr int kMergeThreads = 256;
constexpr int kMergeCols = 16;                 // columns of a thread

// One job's parts, in order: part i is worker c0 + i's.
struct Parts {
    float* base;               // of the first part
    int64_t step;              // floats from part 1 to part 2 and so on ...
    int64_t gap;               // ... and from part 0 to part 1
    int n, R;
};
template <int D>
__device__ __forceinline__ Parts att_parts(const AttendParams& p, const JobList& L, bool wide, bool own, int job, int first, int tiles) {
    const int c0 = L.worker(first), c1 = L.worker(first + tiles - 1);
    const Slot s = att_slot<D>(p, wide, own, job, c0, c0 == c1, true);
    const int64_t row = (int64_t)s.R * (D + 1);
    return {s.base, 2 * row, row, c1 - c0 + 1, s.R};           // (the first part begins the job: slot 2 c0 + 1)
}

// out = sum of w_i part_i / sum of w_i, w_i = 2^lse_i, over the parts of a row's own job and, where
// its stream shares the prefix, of the shared job.  A CTA per (unit of a stream, `rows` rows,
// head); a thread has 16 columns of a row (rows on neighbouring lanes, as the parts store them);
// where there are few rows, several threads take the parts in turn, each with the running maximum
// and sum of a softmax, and are joined pairwise in a fixed order.  Bound by latency (the schedule,
// then the parts, from L2): 5 us after the attention for one stream, about 10 for 14336 rows with
// 5.7 parts each (42 MB).
// kDeep parts are under way together: 4 where one wave of CTAs holds all rows (one stream: 16.5 us
// against 17.3 with 2), 2 where the registers would cost CTAs (96 streams: 201.4 against 202.9).
template <int D, bool kBf16, int kDeep>
__global__ void __launch_bounds__(kMergeThreads) attend_merge_kernel(const AttendParams p, int log_rows) {
    constexpr int kGroups = D / kMergeCols;
    __shared__ float s_acc[kMergeThreads][kMergeCols + 3];     // sums, maximum, weight (odd stride: no bank twice)
    const int tid = threadIdx.x, units = p.a.streams * p.U, unit = blockIdx.x, h = blockIdx.z, row0 = blockIdx.y << log_rows;
    const int rows = 1 << log_rows, row = tid & (rows - 1), group = (tid >> log_rows) & (kGroups - 1);
    const int turn = (tid >> log_rows) / kGroups, turns = (kMergeThreads >> log_rows) / kGroups;
    grid_dependency_wait();
    const int4 u = p.units[unit];                              // first place, rows, tiles, shares
    const JobList Lo = p.head[p.wide_own], Ls = p.head[p.wide_sh];
    if (row0 >= u.y) return;
    Parts sh = {nullptr, 0, 0, 0, 0};
    const Parts own = att_parts<D>(p, Lo, p.wide_own, true, h * units + unit, Lo.W_sh + h * Lo.W1 + u.x + Lo.pad, u.z);
    if (!u.w && own.n == 1) return;                            // written by its only segment
    const int s = p.U == 1 ? unit : unit / p.U, u0 = (unit - s * p.U) * p.rows_own();
    const int r = u0 + row0 + row, packed = s * p.a.block * p.G + r;
    if (u.w) {                                                 // the shared unit that this row lies in
        const int job = h * p.U_sh + (packed >> (p.wide_sh ? 8 : 7));
        sh = att_parts<D>(p, Ls, p.wide_sh, false, job, job * (Ls.tiles_sh + Ls.pad) + Ls.pad, Ls.tiles_sh);
    }
    const bool valid = row0 + row < u.y;
    float m = -INFINITY, z = 0.0f, acc[kMergeCols] = {};
    if (valid) {
        const int n = own.n + sh.n, r_sh = packed & (p.rows_sh() - 1);
        for (int i0 = turn; i0 < n; i0 += kDeep * turns) {
            float lse[kDeep];
            float4 v[kDeep][kMergeCols / 4];
#pragma unroll
            for (int d = 0; d < kDeep; ++d) {
                const int i = i0 + d * turns;
                const bool there = i < n, mine = i < own.n;
                const int k = mine ? i : i - own.n, R = mine ? own.R : sh.R, at = mine ? row0 + row : r_sh;
                const float* part = (mine ? own.base : sh.base) + (k ? (mine ? own.gap : sh.gap) + (k - 1) * (mine ? own.step : sh.step) : 0);
                lse[d] = load_cg_or(part + R * D + at, there, -INFINITY);
#pragma unroll
                for (int x = 0; x < kMergeCols / 4; ++x)
                    v[d][x] = load_cg_or_zero(reinterpret_cast<const float4*>(part) + (group * (kMergeCols / 4) + x) * R + at, there);
            }
#pragma unroll
            for (int d = 0; d < kDeep; ++d) {
                if (lse[d] == -INFINITY) continue;             // a part that saw nothing, or none
                const float top = fmaxf(m, lse[d]), f = exp2_approx(m - top), w = exp2_approx(lse[d] - top);
                m = top;
                z = z * f + w;
#pragma unroll
                for (int x = 0; x < kMergeCols / 4; ++x) {
                    acc[4 * x] = fmaf(w, v[d][x].x, acc[4 * x] * f);
                    acc[4 * x + 1] = fmaf(w, v[d][x].y, acc[4 * x + 1] * f);
                    acc[4 * x + 2] = fmaf(w, v[d][x].z, acc[4 * x + 2] * f);
                    acc[4 * x + 3] = fmaf(w, v[d][x].w, acc[4 * x + 3] * f);
                }
            }
        }
    }
    for (int half = turns / 2; half > 0; half /= 2) {          // the upper half of the turns joins the lower
        if (turn >= half && turn < 2 * half) {
#pragma unroll
            for (int x = 0; x < kMergeCols; ++x) s_acc[tid][x] = acc[x];
            s_acc[tid][kMergeCols] = m;
            s_acc[tid][kMergeCols + 1] = z;
        }
        __syncthreads();
        if (turn < half) {
            const float* o = s_acc[tid + half * rows * kGroups];
            const float mk = o[kMergeCols], zk = o[kMergeCols + 1];
            if (zk != 0.0f) {
                const float top = fmaxf(m, mk), f = exp2_approx(m - top), w = exp2_approx(mk - top);
                m = top;
                z = z * f + zk * w;
#pragma unroll
                for (int x = 0; x < kMergeCols; ++x) acc[x] = fmaf(w, o[x], acc[x] * f);
            }
        }
        __syncthreads();
    }
    if (!valid || turn > 0) return;
    const float inv = z == 0.0f ? 0.0f : 1.0f / z;
    const int t = r / p.G;
    const int64_t at = ((int64_t)s * p.a.block + t) * p.a.q_heads + h * p.G + (r - t * p.G);
    uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.a.out_dev) + at * D + group * kMergeCols);
#pragma unroll
    for (int x = 0; x < kMergeCols / 8; ++x)
        out[x] = make_uint4(pack_f16<kBf16>(acc[8 * x] * inv, acc[8 * x + 1] * inv), pack_f16<kBf16>(acc[8 * x + 2] * inv, acc[8 * x + 3] * inv),
                            pack_f16<kBf16>(acc[8 * x + 4] * inv, acc[8 * x + 5] * inv), pack_f16<kBf16>(acc[8 * x + 6] * inv, acc[8 * x + 7] * inv));
    if (p.a.lse_dev && group == 0) p.a.lse_dev[at] = z == 0.0f ? -INFINITY : (m + log2f(z)) * 0.693147180559945309f;
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

// Sections of the workspace, and the units.
struct AttendLayout {
    int G, wide_own, U, U_wide, R_own;
    size_t units, split_wide, split_narrow, whole_sh, whole_own, total;
};
AttendLayout attend_layout(const moe_mxfp4_cache* c, int streams, int block, int q_heads) {
    AttendLayout L;
    L.G = q_heads / c->cfg.kv_heads;
    const int64_t rows = (int64_t)block * L.G, all = streams * rows;
    // A stream's own rows in wide units wherever one of 128 rows would not do (32 streams over
    // 3500 keys: 136 rows 101 us against 158 in narrow units, 256 rows 111 against 167).
    L.wide_own = rows > 128;
    const int ro = L.wide_own ? 256 : 128;
    L.U = (int)((rows + ro - 1) / ro);
    L.U_wide = (int)((all + 255) / 256);
    L.R_own = (int)(rows < ro ? (rows + 3) / 4 * 4 : ro);   // slots are whole float4s
    const size_t row = (size_t)(c->cfg.head_dim + 1) * 4, jobs = (size_t)c->cfg.kv_heads;
    const size_t split = up256(4 * (size_t)c->sm_count * 128 * row);
    L.units = 256;
    L.split_wide = L.units + up256((size_t)streams * L.U * 16);
    L.split_narrow = L.split_wide + split;
    L.whole_sh = L.split_narrow + split;
    L.whole_own = L.whole_sh + up256(jobs * L.U_wide * 256 * row);   // (units of 128 rows need no more)
    L.total = L.whole_own + up256(jobs * streams * L.U * L.R_own * row);
    return L;
}

template <int D, bool kBf16>
int launch_attend(const moe_mxfp4_cache* c, int layer, const moe::CacheView& v, const moe::AttendParams& p, cudaStream_t st) {
    constexpr size_t smem = sizeof(moe::AttSmem<D>);
    static_assert(smem <= 227 * 1024, "a CTA's shared memory");
    // Rows of a merging CTA (a power of two): as few as keep all rows in two CTAs for every SM, else 32
    // (with 16 they take two waves of CTAs: 84.4 instead of 82.1 us for 32 streams behind 8192 keys).
    const int64_t jobs = (int64_t)c->cfg.kv_heads * p.a.streams * p.U;
    const auto ctas = [&](int log) { return jobs * ((p.R_own + (1 << log) - 1) >> log); };
    int log_rows = 5;
    while (log_rows > 1 && (1 << (log_rows - 1) >= p.R_own || ctas(log_rows - 1) <= 2 * c->sm_count)) --log_rows;
    if (moe::launch_dependent(moe::attend_kernel<D, kBf16>, dim3(c->sm_count), dim3(moe::kAttThreads), smem, st, v, p,
                              c->maps[2 * layer], c->maps[2 * layer + 1]) != cudaSuccess)
        return MOE_ERR_CUDA;
    const bool one_wave = ctas(log_rows) <= 2 * c->sm_count;
    return moe::launch_dependent(one_wave ? moe::attend_merge_kernel<D, kBf16, 4> : moe::attend_merge_kernel<D, kBf16, 2>,
                                 dim3(p.a.streams * p.U, (p.R_own + (1 << log_rows) - 1) >> log_rows, c->cfg.kv_heads),
                                 dim3(moe::kMergeThreads), 0, st, p, log_rows) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

}  // namespace

bool moe::attend_prepare(int device) {
    static std::atomic<uint64_t> done{0};          // a bit per device (more than 64: set every time)
    const uint64_t bit = device < 64 ? 1ull << device : 0;
    if (done.load() & bit) return true;
    const auto set = [](auto* kern, size_t smem) {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) == cudaSuccess;
    };
    if (!set(attend_kernel<128, true>, sizeof(AttSmem<128>)) || !set(attend_kernel<128, false>, sizeof(AttSmem<128>)) ||
        !set(attend_kernel<64, true>, sizeof(AttSmem<64>)) || !set(attend_kernel<64, false>, sizeof(AttSmem<64>)))
        return false;
    done.fetch_or(bit);
    return true;
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
    // places of the schedule, with every stream as long as its table
    const double tiles = ((double)c->cfg.max_pages * c->cfg.page_tokens + a.block) / moe::kKeyTile + 2 + moe::kPadNarrow;
    if (c->cfg.kv_heads * (2.0 * L.U_wide + (double)a.streams * L.U) * tiles >= 2147483647.0) return MOE_ERR_UNSUPPORTED;
    const moe::DeviceScope on(c->device);
    if (!on.ok()) return MOE_ERR_CUDA;
    char* ws = static_cast<char*>(workspace_dev);
    p.v_pool = static_cast<const uint16_t*>(c->layers[layer].v_dev);
    p.G = L.G;
    p.g_mul = 0xFFFFFFFFu / (uint32_t)L.G + 1;
    // The shared prefix in wide units where that makes 20 tiles or more for every CTA: a wide tile
    // costs less than two narrow ones (64 streams behind 32768 keys, 216 tiles: 395 us against 499;
    // 32 behind 8192, 24 tiles: 82.3 against 84.8), but few of them leave slots without work (16
    // behind 8192, 13 tiles: 54.1 against 48.6; 4, 3 tiles: 32.0 against 24.8; all with 8 heads of 128).
    const int64_t rows = (int64_t)a.streams * a.block * L.G;
    p.wide_sh = rows > 128 && (int64_t)c->cfg.kv_heads * L.U_wide * (a.shared_tokens / moe::kKeyTile) >= 20 * (int64_t)c->sm_count;
    p.wide_own = L.wide_own;
    p.U = L.U;
    p.U_sh = p.wide_sh ? L.U_wide : (int)((rows + 127) / 128);
    p.R_own = L.R_own;
    // a negative scale turns the queries' signs; a scale of zero is the smallest above it, which keeps
    // hidden keys (-inf) hidden and takes the largest score (2^128) to 2^-21
    const float s = a.scale < 0.0f ? -a.scale : a.scale;
    p.c = s * 1.44269504088896341f;
    if (p.c < 0x1p-149f) p.c = 0x1p-149f;
    p.q_flip = a.scale < 0.0f ? 0x80008000u : 0u;
    p.timeout_ns = (unsigned long long)c->cfg.timeout_us * 1000ull;
    p.head = reinterpret_cast<moe::JobList*>(ws);
    p.units = reinterpret_cast<int4*>(ws + L.units);
    p.split_wide = reinterpret_cast<float*>(ws + L.split_wide);
    p.split_narrow = reinterpret_cast<float*>(ws + L.split_narrow);
    p.whole_sh = reinterpret_cast<float*>(ws + L.whole_sh);
    p.whole_own = reinterpret_cast<float*>(ws + L.whole_own);
    const moe::CacheView v = moe::cache_view(c, state_dev);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool bf16 = c->cfg.dtype == MOE_DTYPE_BF16;
    if (c->cfg.head_dim == 128)
        return bf16 ? launch_attend<128, true>(c, layer, v, p, st) : launch_attend<128, false>(c, layer, v, p, st);
    return bf16 ? launch_attend<64, true>(c, layer, v, p, st) : launch_attend<64, false>(c, layer, v, p, st);
}
