// Attention of a verify block over the paged key/value cache.
//
// One warp per query row: 32 keys at a time (a lane per key for q.k, a lane per four
// elements for p.v), one pass with the running maximum and sum of the softmax.
#include <cuda_fp16.h>

#include "cache.cuh"

namespace moe {

template <bool kBf16>
__device__ __forceinline__ float2 pair_to_f32(uint32_t v) {
    if (kBf16) return make_float2(bf16_lo(v), bf16_hi(v));
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

template <int D, bool kBf16>
__global__ void __launch_bounds__(128) attend_simple_kernel(CacheView c, const uint16_t* __restrict__ kp,
                                                            const uint16_t* __restrict__ vp, moe_mxfp4_attend_args a) {
    __shared__ float qs[4][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = (int64_t)blockIdx.x * 4 + warp;
    if (row >= (int64_t)a.streams * a.block * a.q_heads) return;
    const int h = (int)(row % a.q_heads);
    const int64_t tok = row / a.q_heads;
    const int s = (int)(tok / a.block), b = (int)(tok % a.block);
    const int used = a.lengths_dev ? min(a.lengths_dev[s], a.block) : a.block;
    if (b >= used) return;
    const int ctx = c.length()[s], held = min(c.held()[s], c.L.M), hk = h / (a.q_heads / c.Hkv);
    const uint16_t* q = static_cast<const uint16_t*>(a.q_dev) + tok * a.q_stride + (int64_t)h * D;
    for (int i = lane; i < D / 2; i += 32) {
        const float2 x = pair_to_f32<kBf16>(reinterpret_cast<const uint32_t*>(q)[i]);
        qs[warp][2 * i] = x.x * a.scale;
        qs[warp][2 * i + 1] = x.y * a.scale;
    }
    __syncwarp();
    const uint64_t bits = a.mask_dev ? a.mask_dev[tok] : 0;
    const int end = ctx + (a.mask_dev ? used : b + 1);
    float m = -INFINITY, l = 0.0f, acc[D / 32] = {};
    for (int j0 = 0; j0 < end; j0 += 32) {
        const int j = j0 + lane;
        bool seen = j < end && (j < ctx || !a.mask_dev || (bits >> (j - ctx) & 1));
        int64_t at = 0;
        if (seen) {
            const int i = j >> c.page_shift;
            const int page = i < held ? c.table(s)[i] : -1;
            seen = (unsigned)page < (unsigned)c.L.P;
            at = page * c.page_stride + ((int64_t)hk * c.page + (j & (c.page - 1))) * D;
        }
        float x = -INFINITY;
        if (seen) {
            x = 0.0f;
            for (int i = 0; i < D / 2; ++i) {
                const float2 k = pair_to_f32<kBf16>(reinterpret_cast<const uint32_t*>(kp + at)[i]);
                x = fmaf(k.x, qs[warp][2 * i], x);
                x = fmaf(k.y, qs[warp][2 * i + 1], x);
            }
        }
        float mx = x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
        mx = fmaxf(m, mx);
        if (mx == -INFINITY && !__any_sync(0xFFFFFFFFu, x != x)) continue;   // nothing seen yet
        const float base = mx == -INFINITY ? 0.0f : mx;
        const float p = seen ? expf(x - base) : 0.0f;
        const float f = expf(m - base);
        l = l * f + warp_sum(p);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) acc[i] *= f;
        m = mx;
        unsigned who = __ballot_sync(0xFFFFFFFFu, seen);
        while (who) {
            const int k = __ffs(who) - 1;
            who &= who - 1;
            const float pk = __shfl_sync(0xFFFFFFFFu, p, k);
            const uint16_t* v = vp + __shfl_sync(0xFFFFFFFFu, at, k);
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const float2 x2 = pair_to_f32<kBf16>(reinterpret_cast<const uint32_t*>(v)[i * 32 + lane]);
                acc[2 * i] = fmaf(pk, x2.x, acc[2 * i]);
                acc[2 * i + 1] = fmaf(pk, x2.y, acc[2 * i + 1]);
            }
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out_dev) + row * D);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        uint32_t v;
        if (kBf16) {
            const __nv_bfloat162 y = __floats2bfloat162_rn(acc[2 * i] * inv, acc[2 * i + 1] * inv);
            v = *reinterpret_cast<const uint32_t*>(&y);
        } else {
            const __half2 y = __floats2half2_rn(acc[2 * i] * inv, acc[2 * i + 1] * inv);
            v = *reinterpret_cast<const uint32_t*>(&y);
        }
        out[i * 32 + lane] = v;
    }
    if (a.lse_dev && lane == 0) a.lse_dev[row] = l == 0.0f ? -INFINITY : (m == -INFINITY ? 0.0f : m) + logf(l);
}

}  // namespace moe

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_shape(const moe_mxfp4_cache* c, int32_t streams, int32_t block, int32_t q_heads) {
    if (!c || streams < 0 || streams > c->cfg.num_streams || block < 0 || q_heads < 1) return MOE_ERR_INVALID_ARG;
    if (q_heads % c->cfg.kv_heads || q_heads / c->cfg.kv_heads > 256) return MOE_ERR_INVALID_ARG;
    if ((int64_t)streams * block > 0x7FFFFFFF / q_heads) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

}  // namespace

extern "C" int moe_mxfp4_cache_attend_bytes(const moe_mxfp4_cache* c, int32_t streams, int32_t block, int32_t q_heads,
                                            size_t* bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    if (const int r = check_shape(c, streams, block, q_heads)) return r;
    *bytes = 256;
    return MOE_OK;
}

extern "C" int moe_mxfp4_cache_attend(moe_mxfp4_cache* c, void* state_dev, int32_t layer, const moe_mxfp4_attend_args* args,
                                      void* workspace_dev, size_t workspace_bytes, void* stream) {
    if (!c || !state_dev || !aligned(state_dev, 16) || !args || layer < 0 || layer >= c->cfg.num_layers)
        return MOE_ERR_INVALID_ARG;
    moe_mxfp4_attend_args a = *args;
    size_t need = 0;
    if (const int r = moe_mxfp4_cache_attend_bytes(c, a.streams, a.block, a.q_heads, &need)) return r;
    const int64_t row = (int64_t)a.q_heads * c->cfg.head_dim;
    if (a.q_stride == 0) a.q_stride = row;
    if (a.q_stride < row || a.q_stride % 8 || !(a.scale == a.scale)) return MOE_ERR_INVALID_ARG;
    if (!aligned(a.lse_dev, 4) || !aligned(a.lengths_dev, 4) || !aligned(a.mask_dev, 8) || (a.mask_dev && a.block > 64))
        return MOE_ERR_INVALID_ARG;
    if (a.shared_tokens < 0 || a.shared_tokens % c->cfg.page_tokens) return MOE_ERR_INVALID_ARG;
    if (a.shared_tokens > 0 && (a.shared_stream < 0 || a.shared_stream >= c->cfg.num_streams ||
                                a.shared_tokens / c->cfg.page_tokens > c->cfg.max_pages))
        return MOE_ERR_INVALID_ARG;
    if (a.streams == 0 || a.block == 0) return MOE_OK;
    if (!a.q_dev || !a.out_dev || !aligned(a.q_dev, 16) || !aligned(a.out_dev, 16)) return MOE_ERR_INVALID_ARG;
    if (!workspace_dev || !aligned(workspace_dev, 256) || workspace_bytes < need) return MOE_ERR_WORKSPACE;
    const moe::DeviceScope on(c->device);
    if (!on.ok()) return MOE_ERR_CUDA;
    const int64_t rows = (int64_t)a.streams * a.block * a.q_heads;
    const auto* kp = static_cast<const uint16_t*>(c->layers[layer].k_dev);
    const auto* vp = static_cast<const uint16_t*>(c->layers[layer].v_dev);
    const moe::CacheView v = moe::cache_view(c, state_dev);
    const dim3 grid((unsigned)((rows + 3) / 4));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool bf16 = c->cfg.dtype == MOE_DTYPE_BF16;
    if (c->cfg.head_dim == 128) {
        if (bf16) moe::attend_simple_kernel<128, true><<<grid, 128, 0, st>>>(v, kp, vp, a);
        else moe::attend_simple_kernel<128, false><<<grid, 128, 0, st>>>(v, kp, vp, a);
    } else {
        if (bf16) moe::attend_simple_kernel<64, true><<<grid, 128, 0, st>>>(v, kp, vp, a);
        else moe::attend_simple_kernel<64, false><<<grid, 128, 0, st>>>(v, kp, vp, a);
    }
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
