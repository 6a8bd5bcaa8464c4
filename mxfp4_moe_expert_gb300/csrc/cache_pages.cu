// Page operations of the paged key/value cache: reserve (with copy on write), append,
// truncate / commit, fork, compact; the handle's life cycle.
//
// The books (lengths, page tables, counts) are a few words per stream and page, so the
// operations that hand out or move pages decide everything in one CTA, in the order of the
// streams and pages (prefix sums, no atomics whose order matters); what follows from the
// decision (copying pages in every layer, rewriting tables) is spread over the GPU by a
// second kernel whose launch overlaps the first.  Atomics are integer sums, minima and
// maxima, whose order cannot be seen.
#include <cudaTypedefs.h>

#include <new>

#include "cache.cuh"

namespace moe {

constexpr int kPlanThreads = 1024;   // of a planning CTA, at most
constexpr int kNoStream = 0x7FFFFFFF;

__device__ __forceinline__ void cache_error(const CacheView& c, int code, int detail) {
    raise_status(c.state + kCacheStatus, code, detail);
}

// Exclusive prefix sum over the CTA's threads; *total: the CTA's sum.
__device__ __forceinline__ long long block_scan(long long v, long long* total) {
    __shared__ long long sums[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        long long t = lane < (int)(blockDim.x >> 5) ? sums[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xFFFFFFFFu, t, o);
            if (lane >= o) t += y;
        }
        sums[lane] = t;
    }
    __syncthreads();
    const long long before = (warp ? sums[warp - 1] : 0) + x - v;
    *total = sums[31];
    __syncthreads();
    return before;
}

// ---- reserve -------------------------------------------------------------------------

// One CTA, bound by the latency of its passes (5 to 9 us).  Every stream's wish; the writers of each shared page; the pages wanted in all;
// as many free pages, lowest first; and, when there are enough, the books.
__global__ void __launch_bounds__(kPlanThreads) cache_reserve_kernel(CacheView c, const int* __restrict__ add, int add_all) {
    __shared__ int s_bad;
    const int tid = threadIdx.x, threads = blockDim.x, S = c.L.S, P = c.L.P;
    int* const writers = c.state + c.L.writers;
    int* const first = c.state + c.L.first;
    int* const ref = c.refcount();
    int* const fl = c.state + c.L.free_list;
    int* const need = c.state + c.L.need;
    int* const last = c.state + c.L.last;
    int* const off = c.state + c.L.off;
    int* const mv_src = c.state + c.L.move_src;
    if (tid == 0) s_bad = kNoStream;
    grid_dependency_wait();
    __syncthreads();
    for (int s = tid; s < S; s += threads) {
        const int len = c.length()[s], held = c.held()[s], n = add ? add[s] : add_all;
        int want = held, page = -1;
        if (n > 0) {
            const long long tokens = (long long)len + n;
            bool bad = len < 0 || held < 0 || held > c.L.M || tokens > ((long long)c.L.M << c.page_shift) ||
                       len > ((long long)held << c.page_shift);
            if (!bad) {
                want = max(held, (int)((tokens + c.page - 1) >> c.page_shift));
                if (len & (c.page - 1)) {
                    page = c.table(s)[len >> c.page_shift];
                    bad = (unsigned)page >= (unsigned)P;
                }
            }
            if (bad) {
                atomicMin(&s_bad, s);
                want = held;
                page = -1;
            }
        }
        if (page >= 0 && ref[page] > 1) {
            atomicAdd(writers + page, 1);
            atomicMax(first + page, S - s);
        } else {
            page = -1;
        }
        need[s] = want;
        last[s] = page < 0 ? -1 : 2 * page;
    }
    __syncthreads();
    // Whether a stream copies its last page: its writers do, but the first of them where
    // they are its only holders.  Pages and copies are summed in the order of the streams.
    long long total = 0;
    int moves = 0;
    for (int s0 = 0; s0 < S; s0 += threads) {
        const int s = s0 + tid;
        int want = 0, copy = 0;
        if (s < S) {
            const int page = last[s] >> 1;
            if (last[s] >= 0) copy = !(ref[page] == writers[page] && first[page] == S - s);
            want = need[s] - c.held()[s] + copy;
        }
        long long sum;
        const long long at = block_scan(((long long)want << 20) | copy, &sum);
        if (s < S) {
            off[s] = (int)min(total + (at >> 20), (long long)P);
            if (copy) {
                last[s] |= 1;
                mv_src[moves + (int)(at & 0xFFFFF)] = s;
            }
        }
        total += sum >> 20;
        moves += (int)(sum & 0xFFFFF);
    }
    bool ok = s_bad == kNoStream;
    long long found = 0;
    if (ok && total <= P) {
        for (int p0 = 0; p0 < P && found < total; p0 += 4 * threads) {
            const int p = p0 + 4 * tid;
            bool r[4];
            int n = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                r[i] = p + i < P && ref[p + i] == 0;
                n += r[i];
            }
            long long sum;
            long long at = found + block_scan(n, &sum);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (r[i]) {
                    if (at < total) fl[at] = p + i;
                    ++at;
                }
            found += sum;
        }
    }
    if (tid == 0) {
        if (!ok) cache_error(c, MOE_ERR_CACHE_STATE, s_bad);
        else if (found < total) cache_error(c, MOE_ERR_CACHE_FULL, (int)min(total, (long long)kNoStream));
        c.state[kCacheMoves] = ok && found >= total ? moves : 0;
    }
    ok = ok && found >= total;
    __syncthreads();
    for (int s = tid; s < S; s += threads)
        if (last[s] >= 0) {                       // the marks back to rest
            writers[last[s] >> 1] = 0;
            first[last[s] >> 1] = 0;
        }
    if (!ok) return;
    for (int m = tid; m < moves; m += threads) {
        const int s = mv_src[m], len = c.length()[s], old = last[s] >> 1, to = fl[off[s]];
        mv_src[m] = old;
        c.state[c.L.move_dst + m] = to;
        c.state[c.L.move_used + m] = len & (c.page - 1);
        c.table(s)[len >> c.page_shift] = to;
        atomicSub(ref + old, 1);
    }
    for (int i = tid; i < (int)total; i += threads) ref[fl[i]] = 1;
    const int lane = tid & 31;
    for (int s = tid >> 5; s < S; s += threads / 32) {   // a warp per stream
        const int held = c.held()[s], n = need[s];
        const int* from = fl + off[s] + (last[s] >= 0 ? last[s] & 1 : 0);
        for (int i = held + lane; i < n; i += 32) c.table(s)[i] = from[i - held];
        __syncwarp();
        if (lane == 0 && n > held) c.held()[s] = n;
    }
}

// ---- copying pages -------------------------------------------------------------------

constexpr int kMaxPools = 256;    // pools of one launch (2 KB of kernel parameters)
struct PoolList {
    void* base[kMaxPools];
};

constexpr int kCopyThreads = 512;
constexpr int kPiece = 4096;      // bytes a warp copies at a time: 8 independent 16-byte loads per lane

// move_src[m] -> move_dst[m] in every pool of the list, the first move_used[m] tokens of
// every head (a warp takes pieces of one head's page); with `remap`, the tables after a
// compact too: entries at U or above have moved.  Bound by HBM: it reads and writes each
// byte once (2.24 GB of a compact in 343 to 365 us from GPU to GPU, with its plan and two copies of
// books: 6.2 to 6.5 TB/s, 0.91 to 0.97 of the copy rate).  Where these took 343, 2 KB pieces took
// 372, 8 KB ones and fewer CTAs the same.
__global__ void __launch_bounds__(kCopyThreads) cache_copy_kernel(CacheView c, const __grid_constant__ PoolList pools, int n_pools, int remap) {
    grid_dependency_wait();
    const int moves = c.state[kCacheMoves];
    const int row = c.D * 2, head = c.page * row;            // bytes of a token, of a head's page
    const int pieces = (head + kPiece - 1) / kPiece;
    const int lane = threadIdx.x & 31, warp0 = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5);
    const int warps = gridDim.x * (kCopyThreads / 32);
    const long long n = (long long)moves * n_pools * c.Hkv * pieces;
    for (long long u = warp0; u < n; u += warps) {
        const int m = (int)(u / (n_pools * c.Hkv * pieces));
        int w = (int)(u - (long long)m * (n_pools * c.Hkv * pieces));
        const int pool = w / (c.Hkv * pieces);
        w -= pool * (c.Hkv * pieces);
        const int h = w / pieces, piece = w - h * pieces;
        const int bytes = c.state[c.L.move_used + m] * row;
        char* const base = static_cast<char*>(pools.base[pool]);
        const int64_t at = (int64_t)h * head + (int64_t)piece * kPiece;
        const uint4* src = reinterpret_cast<const uint4*>(base + c.state[c.L.move_src + m] * c.page_stride * 2 + at);
        uint4* dst = reinterpret_cast<uint4*>(base + c.state[c.L.move_dst + m] * c.page_stride * 2 + at);
        const int left = (min(bytes, (piece + 1) * kPiece) - piece * kPiece) / 16;   // 16-byte words of this piece
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i * 32 + lane < left) v[i] = __ldcs(src + i * 32 + lane);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i * 32 + lane < left) __stcs(dst + i * 32 + lane, v[i]);
    }
    if (!remap) return;
    const int U = c.state[kCacheLive];
    const int* to = c.state + c.L.free_list;
    for (int s = warp0; s < c.L.S; s += warps) {
        const int held = min(c.held()[s], c.L.M);
        for (int i = lane; i < held; i += 32) {
            const int p = c.table(s)[i];
            if (p >= U && p < c.L.P) c.table(s)[i] = to[p];
            else if ((unsigned)p >= (unsigned)c.L.P) cache_error(c, MOE_ERR_CACHE_STATE, s);
        }
    }
}

// ---- append --------------------------------------------------------------------------

// A warp has 32 16-byte words of a token's keys and of its values, which are under way while the
// page is looked up.  Bound by HBM for long blocks (24 x 1999 tokens of 4 heads of 64, 98 MB read
// and written: 16.7 us, 5.9 TB/s), by the launch and that look-up for short ones (8 tokens of 8
// heads of 128: 1.4 us in a graph).  Warps with four tokens at a time measured 17.0 and 1.9 us.
__global__ void __launch_bounds__(256) cache_append_kernel(CacheView c, const char* __restrict__ k, const char* __restrict__ v,
                                                           int64_t row_bytes, char* __restrict__ kp, char* __restrict__ vp,
                                                           int streams, int block, const int* __restrict__ lengths) {
    const int lane = threadIdx.x & 31, log_head = c.D == 128 ? 4 : 3;        // words of a head: 16 or 8
    const int words = c.Hkv << log_head, parts = (words + 31) / 32;
    const int n = streams * block * parts;
    grid_dependency_wait();
    for (int u = blockIdx.x * 8 + (threadIdx.x >> 5); u < n; u += gridDim.x * 8) {
        const int tok = u / parts, w = (u - tok * parts) * 32 + lane;
        const int s = tok / block, i = tok - s * block;
        if (lengths && i >= lengths[s]) continue;
        const bool mine = w < words;
        uint4 a, b;
        if (mine) {
            a = __ldcs(reinterpret_cast<const uint4*>(k + tok * row_bytes) + w);
            b = __ldcs(reinterpret_cast<const uint4*>(v + tok * row_bytes) + w);
        }
        const int len = c.length()[s], held = min(c.held()[s], c.L.M);
        const int64_t pos = (int64_t)len + i;
        int page = -1;
        if (len >= 0 && (pos >> c.page_shift) < held) page = c.table(s)[pos >> c.page_shift];
        if ((unsigned)page >= (unsigned)c.L.P || c.refcount()[page] > 1) {
            if (w == 0) cache_error(c, MOE_ERR_CACHE_STATE, s);
            continue;
        }
        if (!mine) continue;
        const int64_t e = page * c.page_stride + ((int64_t)(w >> log_head) * c.page + (pos & (c.page - 1))) * c.D +
                          (w & ((1 << log_head) - 1)) * 8;
        *reinterpret_cast<uint4*>(kp + e * 2) = a;
        *reinterpret_cast<uint4*>(vp + e * 2) = b;
    }
}

// ---- truncate, commit ----------------------------------------------------------------

// A warp per stream: gives back the pages behind its new length.
__global__ void __launch_bounds__(256) cache_truncate_kernel(CacheView c, const int* __restrict__ value, int relative) {
    const int s = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    grid_dependency_wait();
    if (s >= c.L.S || value[s] < 0) return;
    const int len = c.length()[s], held = c.held()[s];
    const long long to = (long long)value[s] + (relative ? len : 0);
    if (len < 0 || held < 0 || held > c.L.M || to > ((long long)held << c.page_shift)) {
        if (lane == 0) cache_error(c, MOE_ERR_CACHE_STATE, s);
        return;
    }
    const int keep = (int)((to + c.page - 1) >> c.page_shift);
    for (int i = keep + lane; i < held; i += 32) {
        const int p = c.table(s)[i];
        if ((unsigned)p < (unsigned)c.L.P) atomicSub(c.refcount() + p, 1);
        else cache_error(c, MOE_ERR_CACHE_STATE, s);
        c.table(s)[i] = -1;
    }
    __syncwarp();
    if (lane == 0) {
        c.length()[s] = (int)to;
        if (keep < held) c.held()[s] = keep;
    }
}

// ---- fork ----------------------------------------------------------------------------

// A CTA per pair.  Every CTA checks the whole list (against the lengths and the pages held,
// which no CTA changes before all are done), so that all or none take effect; the last CTA
// to finish writes the lengths and the pages held.
__global__ void __launch_bounds__(256) cache_fork_kernel(CacheView c, const int* __restrict__ src, const int* __restrict__ dst, int n) {
    extern __shared__ unsigned taken[];          // a bit per stream: it is a dst
    __shared__ int s_bad, s_last;
    const int tid = threadIdx.x, S = c.L.S;
    for (int i = tid; i < (S + 31) / 32; i += 256) taken[i] = 0;
    if (tid == 0) s_bad = kNoStream;
    grid_dependency_wait();
    __syncthreads();
    for (int i = tid; i < n; i += 256) {
        const int a = src[i], b = dst[i];
        bool bad = (unsigned)a >= (unsigned)S || (unsigned)b >= (unsigned)S;
        if (!bad) {
            const int len = c.length()[a], held = c.held()[a];
            bad = c.held()[b] != 0 || len < 0 || held > c.L.M || len > ((long long)held << c.page_shift);
            if (atomicOr(taken + (b >> 5), 1u << (b & 31)) >> (b & 31) & 1u) bad = true;   // twice
        }
        if (bad) atomicMin(&s_bad, i);
    }
    __syncthreads();
    for (int i = tid; i < n; i += 256) {
        const int a = src[i];
        if ((unsigned)a < (unsigned)S && (taken[a >> 5] >> (a & 31) & 1u)) atomicMin(&s_bad, i);
    }
    __syncthreads();
    const bool ok = s_bad == kNoStream;
    if (ok) {
        const int a = src[blockIdx.x], b = dst[blockIdx.x];
        const int pages = (c.length()[a] + c.page - 1) >> c.page_shift;
        for (int i = tid; i < pages; i += 256) {
            const int p = c.table(a)[i];
            c.table(b)[i] = p;
            if ((unsigned)p < (unsigned)c.L.P) atomicAdd(c.refcount() + p, 1);
            else cache_error(c, MOE_ERR_CACHE_STATE, blockIdx.x);
        }
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) s_last = atomicAdd(c.state + kCacheArrived, 1) == (int)gridDim.x - 1;
    __syncthreads();
    if (!s_last) return;
    if (ok)
        for (int i = tid; i < n; i += 256) {
            const int len = c.length()[src[i]];
            c.length()[dst[i]] = len;
            c.held()[dst[i]] = (len + c.page - 1) >> c.page_shift;
        }
    if (tid == 0) {
        c.state[kCacheArrived] = 0;
        if (!ok) cache_error(c, MOE_ERR_CACHE_STATE, s_bad);
    }
}

// ---- compact -------------------------------------------------------------------------

// One CTA.  U = pages in use; the i-th used page at U or above goes to the i-th free one
// below U (there are as many of one as of the other).
__global__ void __launch_bounds__(kPlanThreads) cache_compact_kernel(CacheView c) {
    const int tid = threadIdx.x, threads = blockDim.x, P = c.L.P;
    int* const ref = c.refcount();
    int* const to = c.state + c.L.free_list;     // old page -> new page, for the pages that move
    int* const src = c.state + c.L.move_src;
    int* const dst = c.state + c.L.move_dst;
    long long sum;
    int mine = 0;
    grid_dependency_wait();
    for (int p = tid; p < P; p += threads) mine += ref[p] != 0;
    block_scan(mine, &sum);
    const int U = (int)sum;
    int n_src = 0, n_dst = 0;
    for (int p0 = 0; p0 < P; p0 += threads) {
        const int p = p0 + tid;
        const bool used = p < P && ref[p] != 0;
        const bool up = used && p >= U, hole = p < U && !used;
        const long long at = block_scan(((long long)up << 32) | hole, &sum);
        if (up) src[n_src + (int)(at >> 32)] = p;
        if (hole) dst[n_dst + (int)(at & 0xFFFFFFFF)] = p;
        n_src += (int)(sum >> 32);
        n_dst += (int)(sum & 0xFFFFFFFF);
    }
    __syncthreads();
    for (int m = tid; m < n_src; m += threads) {
        const int a = src[m], b = dst[m];
        to[a] = b;
        c.state[c.L.move_used + m] = c.page;
        ref[b] = ref[a];
        ref[a] = 0;
    }
    if (tid == 0) {
        c.state[kCacheMoves] = n_src;
        c.state[kCacheLive] = U;
    }
}

}  // namespace moe

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool good_state(const moe_mxfp4_cache* c, const void* state) { return c && state && aligned16(state); }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

bool device_memory(const void* p, int device) {
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return a.type == cudaMemoryTypeManaged || (a.type == cudaMemoryTypeDevice && a.device == device);
}

// A pool as a tensor of [pages][kv_heads * page_tokens][head_dim] 16-bit elements, read in
// boxes of one head's page (up to 128 tokens) x 64 elements, in the 128-byte swizzle.
bool encode_pool(CUtensorMap* m, const void* base, const moe_mxfp4_cache_config& c) {
    static const PFN_cuTensorMapEncodeTiled_v12000 enc = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.kv_heads * c.page_tokens, (cuuint64_t)c.num_pages};
    const cuuint64_t strides[2] = {(cuuint64_t)c.head_dim * 2, (cuuint64_t)c.page_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)c.page_tokens, 1};
    const cuuint32_t step[3] = {1, 1, 1};
    return enc(m, c.dtype == MOE_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
               const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// Threads of a planning CTA.  A barrier of 8 warps is cheaper than one of 32, and few streams and
// pages need no more: reserving for 32 streams of 521 pages takes 5.8 us with 256 threads and 6.4
// with 1024, for 256 streams 10.1 and 8.5; compacting 10 pages 3.1 and 3.5, 521 pages 4.0 and 3.4
// (with the copying kernel that follows, in a graph).
int reserve_threads(const moe_mxfp4_cache* c) { return c->cfg.num_streams <= 64 && c->cfg.num_pages <= 1024 ? 256 : moe::kPlanThreads; }
int compact_threads(const moe_mxfp4_cache* c) { return c->cfg.num_pages <= 256 ? 256 : moe::kPlanThreads; }

// Copies the pages of the move list (at most `moves` of them) in every pool, kMaxPools pools a
// launch; the last launch also rewrites the tables, with `remap`.
int launch_copies(const moe_mxfp4_cache* c, const moe::CacheView& v, int64_t moves, int remap, cudaStream_t st) {
    for (int l0 = 0; l0 < c->cfg.num_layers; l0 += moe::kMaxPools / 2) {
        moe::PoolList pools = {};
        int n = 0;
        for (int l = l0; l < c->cfg.num_layers && n < moe::kMaxPools; ++l) {
            pools.base[n++] = c->layers[l].k_dev;
            pools.base[n++] = c->layers[l].v_dev;
        }
        const int64_t head = (int64_t)c->cfg.page_tokens * c->cfg.head_dim * 2;
        int64_t warps = moves * n * c->cfg.kv_heads * ((head + moe::kPiece - 1) / moe::kPiece);
        if (remap && warps < c->cfg.num_streams) warps = c->cfg.num_streams;
        const int64_t per_cta = moe::kCopyThreads / 32, want = (warps + per_cta - 1) / per_cta, most = 4 * c->sm_count;
        if (moe::launch_dependent(moe::cache_copy_kernel, dim3((unsigned)(want < most ? want : most)), dim3(moe::kCopyThreads), 0, st,
                                  v, pools, n, remap && l0 + moe::kMaxPools / 2 >= c->cfg.num_layers) != cudaSuccess)
            return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_mxfp4_cache_create(const moe_mxfp4_cache_config* cfg, const moe_mxfp4_cache_layer* layers, moe_mxfp4_cache** out) {
    if (!cfg || !layers || !out) return MOE_ERR_INVALID_ARG;
    *out = nullptr;
    moe_mxfp4_cache_config c = *cfg;
    if (c.num_layers < 1 || c.num_layers > 1024 || c.num_streams < 1 || c.num_streams > 65536) return MOE_ERR_INVALID_ARG;
    if (c.num_pages < 1 || c.num_pages > (1 << 24)) return MOE_ERR_INVALID_ARG;
    if (c.page_tokens != 16 && c.page_tokens != 32 && c.page_tokens != 64 && c.page_tokens != 128) return MOE_ERR_INVALID_ARG;
    if (c.max_pages < 1 || (int64_t)c.max_pages * c.page_tokens >= (1 << 30)) return MOE_ERR_INVALID_ARG;
    if (c.kv_heads < 1 || c.kv_heads > 256) return MOE_ERR_INVALID_ARG;
    if (c.head_dim != 64 && c.head_dim != 128) return MOE_ERR_INVALID_ARG;
    if (c.dtype != MOE_DTYPE_BF16 && c.dtype != MOE_DTYPE_FP16) return MOE_ERR_INVALID_ARG;
    const int64_t page = (int64_t)c.kv_heads * c.page_tokens * c.head_dim;
    if (c.page_stride == 0) c.page_stride = page;
    if (c.page_stride < page || c.page_stride % 8 || c.page_stride >= ((int64_t)1 << 38)) return MOE_ERR_INVALID_ARG;
    if (c.timeout_us < 0) return MOE_ERR_INVALID_ARG;
    if (c.timeout_us == 0) c.timeout_us = 200000;
    for (int l = 0; l < c.num_layers; ++l)
        if (!layers[l].k_dev || !layers[l].v_dev || !aligned16(layers[l].k_dev) || !aligned16(layers[l].v_dev))
            return MOE_ERR_INVALID_ARG;
    int dev = 0, major = 0, minor = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return MOE_ERR_CUDA;
    if (major != 10 || minor != 3) return MOE_ERR_UNSUPPORTED;
    for (int l = 0; l < c.num_layers; ++l)
        if (!device_memory(layers[l].k_dev, dev) || !device_memory(layers[l].v_dev, dev)) return MOE_ERR_INVALID_ARG;
    if (!moe::attend_prepare(dev)) return MOE_ERR_CUDA;
    try {
        moe_mxfp4_cache* h = new moe_mxfp4_cache();
        h->cfg = c;
        h->device = dev;
        h->sm_count = sms;
        h->layers.assign(layers, layers + c.num_layers);
        h->maps.resize(2 * (size_t)c.num_layers);
        for (int l = 0; l < c.num_layers; ++l)
            if (!encode_pool(&h->maps[2 * l], layers[l].k_dev, c) || !encode_pool(&h->maps[2 * l + 1], layers[l].v_dev, c)) {
                delete h;
                return MOE_ERR_CUDA;
            }
        *out = h;
    } catch (...) {
        return MOE_ERR_INVALID_ARG;
    }
    return MOE_OK;
}

void moe_mxfp4_cache_destroy(moe_mxfp4_cache* c) { delete c; }

int moe_mxfp4_cache_state_bytes(const moe_mxfp4_cache* c, size_t* bytes) {
    if (!c || !bytes) return MOE_ERR_INVALID_ARG;
    *bytes = (size_t)moe::cache_layout(c->cfg.num_streams, c->cfg.max_pages, c->cfg.num_pages).total * 4;
    return MOE_OK;
}

int moe_mxfp4_cache_reserve(moe_mxfp4_cache* c, void* state_dev, const int32_t* add_dev, int32_t add, void* stream) {
    if (!good_state(c, state_dev) || !aligned4(add_dev)) return MOE_ERR_INVALID_ARG;
    const moe::DeviceScope on(c->device);
    if (!on.ok()) return MOE_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const moe::CacheView v = moe::cache_view(c, state_dev);
    if (moe::launch_dependent(moe::cache_reserve_kernel, dim3(1), dim3(reserve_threads(c)), 0, st, v, add_dev, add) != cudaSuccess)
        return MOE_ERR_CUDA;
    return launch_copies(c, v, c->cfg.num_streams, 0, st);
}

int moe_mxfp4_cache_append(moe_mxfp4_cache* c, void* state_dev, int32_t layer, const void* k_dev, const void* v_dev,
                           int64_t row_stride, int32_t streams, int32_t block, const int32_t* lengths_dev, void* stream) {
    if (!good_state(c, state_dev) || layer < 0 || layer >= c->cfg.num_layers) return MOE_ERR_INVALID_ARG;
    if (streams < 0 || streams > c->cfg.num_streams || block < 0 || !aligned4(lengths_dev)) return MOE_ERR_INVALID_ARG;
    const int64_t row = (int64_t)c->cfg.kv_heads * c->cfg.head_dim;
    if (row_stride == 0) row_stride = row;
    if (row_stride < row || row_stride % 8) return MOE_ERR_INVALID_ARG;
    if (streams == 0 || block == 0) return MOE_OK;
    if (!k_dev || !v_dev || !aligned16(k_dev) || !aligned16(v_dev)) return MOE_ERR_INVALID_ARG;
    const moe::DeviceScope on(c->device);
    if (!on.ok()) return MOE_ERR_CUDA;
    const int64_t warps = (int64_t)streams * block * ((row / 8 + 31) / 32);
    if (warps > 1 << 30) return MOE_ERR_UNSUPPORTED;
    const int64_t want = (warps + 7) / 8, most = 64 * (int64_t)c->sm_count;
    return status_of(moe::launch_dependent(
        moe::cache_append_kernel, dim3((unsigned)(want < most ? want : most)), dim3(256), 0, static_cast<cudaStream_t>(stream),
        moe::cache_view(c, state_dev), static_cast<const char*>(k_dev), static_cast<const char*>(v_dev), row_stride * 2,
        static_cast<char*>(c->layers[layer].k_dev), static_cast<char*>(c->layers[layer].v_dev), streams, block, lengths_dev));
}

static int cache_truncate(moe_mxfp4_cache* c, void* state_dev, const int32_t* value, int relative, void* stream) {
    if (!good_state(c, state_dev) || !value || !aligned4(value)) return MOE_ERR_INVALID_ARG;
    const moe::DeviceScope on(c->device);
    if (!on.ok()) return MOE_ERR_CUDA;
    return status_of(moe::launch_dependent(moe::cache_truncate_kernel, dim3((c->cfg.num_streams + 7) / 8), dim3(256), 0,
                                           static_cast<cudaStream_t>(stream), moe::cache_view(c, state_dev), value, relative));
}

int moe_mxfp4_cache_truncate(moe_mxfp4_cache* c, void* state_dev, const int32_t* new_length_dev, void* stream) {
    return cache_truncate(c, state_dev, new_length_dev, 0, stream);
}

int moe_mxfp4_cache_commit(moe_mxfp4_cache* c, void* state_dev, const int32_t* accepted_dev, void* stream) {
    return cache_truncate(c, state_dev, accepted_dev, 1, stream);
}

int moe_mxfp4_cache_fork(moe_mxfp4_cache* c, void* state_dev, const int32_t* src_dev, const int32_t* dst_dev, int32_t n,
                         void* stream) {
    if (!good_state(c, state_dev) || n < 0 || n > c->cfg.num_streams) return MOE_ERR_INVALID_ARG;
    if (n == 0) return MOE_OK;
    if (!src_dev || !dst_dev || !aligned4(src_dev) || !aligned4(dst_dev)) return MOE_ERR_INVALID_ARG;
    const moe::DeviceScope on(c->device);
    if (!on.ok()) return MOE_ERR_CUDA;
    const size_t smem = (size_t)((c->cfg.num_streams + 31) / 32) * 4;
    return status_of(moe::launch_dependent(moe::cache_fork_kernel, dim3(n), dim3(256), smem, static_cast<cudaStream_t>(stream),
                                           moe::cache_view(c, state_dev), src_dev, dst_dev, n));
}

int moe_mxfp4_cache_compact(moe_mxfp4_cache* c, void* state_dev, void* stream) {
    if (!good_state(c, state_dev)) return MOE_ERR_INVALID_ARG;
    const moe::DeviceScope on(c->device);
    if (!on.ok()) return MOE_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const moe::CacheView v = moe::cache_view(c, state_dev);
    if (moe::launch_dependent(moe::cache_compact_kernel, dim3(1), dim3(compact_threads(c)), 0, st, v) != cudaSuccess) return MOE_ERR_CUDA;
    return launch_copies(c, v, c->cfg.num_pages / 2, 1, st);
}

int moe_mxfp4_cache_check(moe_mxfp4_cache* c, void* state_dev, void* stream) {
    if (!good_state(c, state_dev)) return MOE_ERR_INVALID_ARG;
    const moe::DeviceScope on(c->device);
    if (!on.ok()) return MOE_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int s[2] = {0, 0};
    if (cudaMemcpyAsync(s, state_dev, sizeof(s), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return MOE_ERR_CUDA;
    if (s[0] == MOE_OK) return MOE_OK;
    if (cudaMemsetAsync(state_dev, 0, sizeof(s), st) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess)
        return MOE_ERR_CUDA;
    return s[0];
}

}  // extern "C"
