// The paged key/value cache: its handle, the layout of its state words, and what the
// page operations (cache_pages.cu) and the attention (cache_attend.cu) share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <vector>

#include "common.cuh"

struct moe_mxfp4_cache {
    moe_mxfp4_cache_config cfg;                  // page_stride and timeout_us resolved
    std::vector<moe_mxfp4_cache_layer> layers;
    std::vector<CUtensorMap> maps;               // per layer: K pool, V pool
    int device = 0;
    int sm_count = 0;
};

namespace moe {

// Word offsets of the state (moe_mxfp4.h states the first five; the rest is the library's):
// the marks are zero at rest, the others are written before they are read.
struct CacheLayout {
    int S, M, P;                  // streams, pages per stream, pages of the pool
    int64_t length, held, table, refcount;
    int64_t writers, first;       // [P] at rest 0: streams of a reserve that write the page, the lowest of them
    int64_t free_list;            // [P] free pages found by a reserve; old -> new page of a compact
    int64_t need, last;           // [S] reserve: pages held afterwards; 2 * the page written in place + copied, or -1
    int64_t off;                  // [S] reserve: first entry of the stream's pages in free_list
    int64_t move_src, move_dst, move_used;   // [moves] pages to copy and the tokens to copy of each
    int64_t total;
};

enum : int {                      // header words
    kCacheStatus = 0,             // status code, detail
    kCacheMoves = 2,              // number of pages to copy
    kCacheLive = 3,               // pages in use (compact)
    kCacheArrived = 4,            // CTAs of a fork that are done (0 at rest)
    kCacheHeader = 16,
};

__host__ __device__ inline CacheLayout cache_layout(int S, int M, int P) {
    CacheLayout L;
    L.S = S; L.M = M; L.P = P;
    const int64_t moves = S > P ? S : P;
    L.length = kCacheHeader;
    L.held = L.length + S;
    L.table = L.held + S;
    L.refcount = L.table + (int64_t)S * M;
    L.writers = L.refcount + P;
    L.first = L.writers + P;
    L.free_list = L.first + P;
    L.need = L.free_list + P;
    L.last = L.need + S;
    L.off = L.last + S;
    L.move_src = L.off + S;
    L.move_dst = L.move_src + moves;
    L.move_used = L.move_dst + moves;
    L.total = L.move_used + moves;
    return L;
}

// What a kernel gets of a cache.
struct CacheView {
    int* state;
    CacheLayout L;
    int page, page_shift;         // tokens per page, its logarithm
    int Hkv, D;
    int64_t page_stride;          // elements
    __device__ int* length() const { return state + L.length; }
    __device__ int* held() const { return state + L.held; }
    __device__ int* table(int s) const { return state + L.table + (int64_t)s * L.M; }
    __device__ int* refcount() const { return state + L.refcount; }
};

inline CacheView cache_view(const moe_mxfp4_cache* c, void* state) {
    CacheView v;
    v.state = static_cast<int*>(state);
    v.L = cache_layout(c->cfg.num_streams, c->cfg.max_pages, c->cfg.num_pages);
    v.page = c->cfg.page_tokens;
    v.page_shift = 0;
    while ((1 << v.page_shift) < v.page) ++v.page_shift;
    v.Hkv = c->cfg.kv_heads;
    v.D = c->cfg.head_dim;
    v.page_stride = c->cfg.page_stride;
    return v;
}

// Allows the attention's kernels their shared memory on the current device, once for each.
bool attend_prepare(int device);

// The handle's device for the duration of a call.
class DeviceScope {
  public:
    explicit DeviceScope(int device) {
        ok_ = cudaGetDevice(&was_) == cudaSuccess;
        if (ok_ && was_ != device) {
            ok_ = cudaSetDevice(device) == cudaSuccess;
            back_ = ok_;
        }
    }
    ~DeviceScope() {
        if (back_) cudaSetDevice(was_);
    }
    bool ok() const { return ok_; }

  private:
    int was_ = 0;
    bool ok_ = false, back_ = false;
};

// A launch that may begin while the kernel before it on the stream still runs; the kernel
// calls grid_dependency_wait before it reads what that one wrote.
template <class... P, class... A>
inline cudaError_t launch_dependent(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dependency_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace moe
