// Edits of a verify block's logits (moe_mxfp4_edit_logits) and acceptance of chains and trees of drafts with
// them (moe_mxfp4_accept_edited): penalties for tokens that a stream has said or was prompted with, biases and
// grammar masks.
//
// How often a token was said is counted where it is needed: a CTA has a run of tokens of the vocabulary and
// counts those of the stream's history that lie in it in shared memory, so nothing is kept from call to call.
#include <cuda_fp16.h>

#include <cmath>

#include "cache.cuh"

namespace moe {

constexpr int kEditThreads = 256;
constexpr int kEditRun = 4096;              // tokens of the vocabulary of a CTA
constexpr uint32_t kPrompted = 1u << 31;    // of a count: the prompt has the token

struct EditView {
    moe_mxfp4_edit_args a;
    void* out;
    int64_t out_stride;
    unsigned long long* best;               // acceptance: [rows, runs] largest (key, ~token) of a run, 0 = none
    int runs;
};

template <int kType>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
    if (kType == MOE_DTYPE_FP32) return static_cast<const float*>(p)[i];
    const uint16_t x = static_cast<const uint16_t*>(p)[i];
    return kType == MOE_DTYPE_BF16 ? __uint_as_float((uint32_t)x << 16) : __half2float(__ushort_as_half(x));
}
template <int kType>
__device__ __forceinline__ void store_logit(void* p, int64_t i, float z) {
    if (kType == MOE_DTYPE_FP32) static_cast<float*>(p)[i] = z;
    else static_cast<uint16_t*>(p)[i] = kType == MOE_DTYPE_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(z)) : __half_as_ushort(__float2half_rn(z));
}

struct Penalty {
    float repetition, frequency, presence;
};

// The order of the operations and their roundings are fixed: both entry points give the same value.
__device__ __forceinline__ float edited(float z, uint32_t count, const Penalty& p) {
    if (count) z = z > 0 ? __fdiv_rn(z, p.repetition) : __fmul_rn(z, p.repetition);
    const uint32_t c = count & ~kPrompted;
    if (c) z = __fsub_rn(__fmaf_rn(-p.frequency, (float)c, z), p.presence);
    return z;
}

// Orderable key of a logit (larger logit, larger key; equal ones, -0 and +0 among them, have one key; NaN ranks as -inf).
__device__ __forceinline__ uint32_t logit_key(float v) {
    uint32_t u = __float_as_uint(v == 0.0f ? 0.0f : v);
    if (v != v) u = 0xFF800000u;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int used_positions(const moe_mxfp4_edit_args& a, int s) {
    return a.lengths_dev ? min(a.lengths_dev[s], a.block) : a.block;
}
// Block positions before b that b sees.
__device__ __forceinline__ bool sees(const moe_mxfp4_edit_args& a, int64_t row, int b, int j) {
    return j == b || (j < b && (!a.mask_dev || (a.mask_dev[row] >> j & 1)));
}

// A CTA per (position, run of the vocabulary).
template <int kType, bool kAccept>
__global__ void __launch_bounds__(kEditThreads) edit_kernel(EditView e) {
    __shared__ uint32_t count[kEditRun];
    __shared__ int entry[kEditRun];         // 1 + the last entry of the stream's biases for the token
    __shared__ unsigned long long red[kEditThreads / 32];
    const moe_mxfp4_edit_args& a = e.a;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / e.runs;
    const int run = blockIdx.x - row * e.runs;
    const int s = row / a.block, b = row - (int64_t)s * a.block;
    const int64_t v0 = (int64_t)run * kEditRun;
    const int n = (int)min((int64_t)kEditRun, a.vocab - v0);
    grid_dependency_wait();
    if (b >= used_positions(a, s)) return;
    for (int i = tid; i < kEditRun; i += kEditThreads) {
        count[i] = 0;
        entry[i] = 0;
    }
    __syncthreads();
    if (a.history_dev) {
        const int64_t len = min((int64_t)a.history_lengths_dev[s], a.history_room);
        const int64_t prompt = a.prompt_lengths_dev ? a.prompt_lengths_dev[s] : 0;
        for (int64_t i = tid; i < len; i += kEditThreads) {
            const int64_t v = a.history_dev[s * a.history_stride + i] - v0;
            if (v < 0 || v >= n) continue;
            if (i < prompt) atomicOr(count + v, kPrompted);
            else atomicAdd(count + v, 1u);
        }
    }
    if (a.tokens_dev)
        for (int j = tid; j <= b; j += kEditThreads) {
            const int64_t v = a.tokens_dev[(int64_t)s * a.block + j] - v0;
            if (v >= 0 && v < n && sees(a, row, b, j)) atomicAdd(count + v, 1u);
        }
    if (a.bias_begin_dev) {
        const int64_t end = min((int64_t)a.bias_begin_dev[s + 1], a.bias_entries);
        for (int64_t i = (int64_t)max(a.bias_begin_dev[s], 0) + tid; i < end; i += kEditThreads) {
            const int64_t v = a.bias_ids_dev[i] - v0;
            if (v >= 0 && v < n) atomicMax(entry + v, (int)i + 1);
        }
    }
    __syncthreads();
    const Penalty p{a.repetition_dev ? a.repetition_dev[s] : 1.0f, a.frequency_dev ? a.frequency_dev[s] : 0.0f,
                    a.presence_dev ? a.presence_dev[s] : 0.0f};
    unsigned long long best = 0;
    for (int i = tid; i < n; i += kEditThreads) {
        const int64_t v = v0 + i;
        const bool ok = !a.allowed_dev || (a.allowed_dev[row * a.allowed_stride + (v >> 5)] >> (v & 31) & 1);
        float z = edited(load_logit<kType>(a.logits_dev, row * a.row_stride + v), count[i], p);
        if (entry[i]) z += a.bias_dev[entry[i] - 1];
        if (!kAccept) {
            store_logit<kType>(e.out, row * e.out_stride + v, ok ? z : -INFINITY);
        } else if (ok) {
            const unsigned long long cand = (unsigned long long)logit_key(z) << 32 | (0xFFFFFFFFu - (uint32_t)v);
            best = cand > best ? cand : best;
        }
    }
    if (!kAccept) return;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long other = __shfl_xor_sync(0xFFFFFFFFu, best, o);
        best = other > best ? other : best;
    }
    if ((tid & 31) == 0) red[tid >> 5] = best;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kEditThreads / 32; ++w) best = red[w] > best ? red[w] : best;
        e.best[blockIdx.x] = best;
    }
}

// A CTA per stream: the targets of its positions, and the path of accepted nodes.
__global__ void __launch_bounds__(256) accept_path_kernel(EditView e, int* __restrict__ target, int* __restrict__ accepted,
                                                          int* __restrict__ next_token, int* __restrict__ path) {
    __shared__ int s_target[1024], s_token[1024], s_parent[1024];
    const moe_mxfp4_edit_args& a = e.a;
    const int s = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    grid_dependency_wait();
    const int used = used_positions(a, s);
    const int64_t row0 = (int64_t)s * a.block;
    for (int b = tid >> 5; b < a.block; b += 8) {
        unsigned long long best = 0;
        if (b < used)
            for (int i = lane; i < e.runs; i += 32) {
                const unsigned long long x = e.best[(row0 + b) * e.runs + i];
                best = x > best ? x : best;
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long other = __shfl_xor_sync(0xFFFFFFFFu, best, o);
            best = other > best ? other : best;
        }
        if (lane == 0) {
            s_target[b] = best ? (int)(0xFFFFFFFFu - (uint32_t)best) : -1;
            target[row0 + b] = s_target[b];
            s_token[b] = a.tokens_dev[row0 + b];
            int up = b - 1;
            if (a.mask_dev) {
                const unsigned long long below = a.mask_dev[row0 + b] & ((1ull << b) - 1);
                up = 63 - __clzll(below);
            }
            s_parent[b] = up;
        }
    }
    __syncthreads();
    if (tid >= 32) return;
    int at = 0, n = 0;
    while (n < used) {
        if (lane == 0 && path) path[row0 + n] = at;
        ++n;
        int child = a.block;
        if (s_target[at] >= 0)
            for (int c = at + 1 + lane; c < used; c += 32)
                if (s_parent[c] == at && s_token[c] == s_target[at]) {
                    child = c;
                    break;
                }
        child = __reduce_min_sync(0xFFFFFFFFu, child);
        if (child >= used) break;
        at = child;
    }
    if (path)
        for (int i = n + lane; i < a.block; i += 32) path[row0 + i] = -1;
    if (lane == 0) {
        accepted[s] = n;
        if (next_token) next_token[s] = n ? s_target[at] : -1;
    }
}

}  // namespace moe

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int edit_runs(int64_t vocab) { return (int)((vocab + moe::kEditRun - 1) / moe::kEditRun); }

// Checks the arguments and resolves the strides.
int check_edit(moe_mxfp4_edit_args* a) {
    if (a->dtype != MOE_DTYPE_BF16 && a->dtype != MOE_DTYPE_FP16 && a->dtype != MOE_DTYPE_FP32) return MOE_ERR_INVALID_ARG;
    if (a->streams < 0 || a->block < 1 || a->block > 1024 || a->vocab < 1 || a->vocab > 0x7FFFFFFF) return MOE_ERR_INVALID_ARG;
    if ((int64_t)a->streams * a->block > 0x7FFFFFFF || (a->mask_dev && a->block > 64)) return MOE_ERR_INVALID_ARG;
    if (a->row_stride == 0) a->row_stride = a->vocab;
    if (a->allowed_stride == 0) a->allowed_stride = (a->vocab + 31) / 32;
    if (a->row_stride < a->vocab || a->allowed_stride < (a->vocab + 31) / 32) return MOE_ERR_INVALID_ARG;
    if (a->streams == 0) return MOE_OK;
    if (!a->logits_dev || !aligned(a->logits_dev, a->dtype == MOE_DTYPE_FP32 ? 4 : 2)) return MOE_ERR_INVALID_ARG;
    if (a->history_dev && (!a->history_lengths_dev || a->history_room < 0 || a->history_stride < a->history_room)) return MOE_ERR_INVALID_ARG;
    if (a->bias_begin_dev && (a->bias_entries < 0 || a->bias_entries > 0x7FFFFFFF)) return MOE_ERR_INVALID_ARG;
    if (a->bias_begin_dev && a->bias_entries && (!a->bias_ids_dev || !a->bias_dev)) return MOE_ERR_INVALID_ARG;
    if (!aligned(a->mask_dev, 8)) return MOE_ERR_INVALID_ARG;
    for (const void* p : {(const void*)a->tokens_dev, (const void*)a->lengths_dev, (const void*)a->history_dev, (const void*)a->history_lengths_dev,
                          (const void*)a->prompt_lengths_dev, (const void*)a->repetition_dev, (const void*)a->frequency_dev,
                          (const void*)a->presence_dev, (const void*)a->bias_begin_dev, (const void*)a->bias_ids_dev,
                          (const void*)a->bias_dev, (const void*)a->allowed_dev})
        if (!aligned(p, 4)) return MOE_ERR_INVALID_ARG;
    return (int64_t)a->streams * a->block * edit_runs(a->vocab) > 0x7FFFFFFF ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

template <bool kAccept>
int launch_edit(const moe::EditView& e, cudaStream_t st) {
    const dim3 grid((unsigned)(e.a.streams * (int64_t)e.a.block * e.runs));
    auto go = [&](auto kern) { return moe::launch_dependent(kern, grid, dim3(moe::kEditThreads), 0, st, e); };
    const cudaError_t r = e.a.dtype == MOE_DTYPE_FP32   ? go(moe::edit_kernel<MOE_DTYPE_FP32, kAccept>)
                          : e.a.dtype == MOE_DTYPE_BF16 ? go(moe::edit_kernel<MOE_DTYPE_BF16, kAccept>)
                                                        : go(moe::edit_kernel<MOE_DTYPE_FP16, kAccept>);
    return r == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace

extern "C" {

int moe_mxfp4_edit_logits(const moe_mxfp4_edit_args* args, void* out_dev, int64_t out_stride, void* stream) {
    if (!args) return MOE_ERR_INVALID_ARG;
    moe::EditView e = {};
    e.a = *args;
    const int st = check_edit(&e.a);
    if (st != MOE_OK) return st;
    if (out_stride == 0) out_stride = e.a.vocab;
    if (out_stride < e.a.vocab) return MOE_ERR_INVALID_ARG;
    if (e.a.streams == 0) return MOE_OK;
    if (!out_dev || !aligned(out_dev, e.a.dtype == MOE_DTYPE_FP32 ? 4 : 2)) return MOE_ERR_INVALID_ARG;
    if (out_dev == e.a.logits_dev && out_stride != e.a.row_stride) return MOE_ERR_INVALID_ARG;
    e.out = out_dev;
    e.out_stride = out_stride;
    e.runs = edit_runs(e.a.vocab);
    return launch_edit<false>(e, static_cast<cudaStream_t>(stream));
}

int moe_mxfp4_accept_edited_bytes(int32_t streams, int32_t block, int64_t vocab, size_t* bytes) {
    if (streams < 0 || block < 1 || block > 1024 || vocab < 1 || vocab > 0x7FFFFFFF || !bytes) return MOE_ERR_INVALID_ARG;
    *bytes = (size_t)streams * block * edit_runs(vocab) * sizeof(unsigned long long);
    return MOE_OK;
}

int moe_mxfp4_accept_edited(const moe_mxfp4_edit_args* args, int32_t* target_dev, int32_t* accepted_dev,
                            int32_t* next_token_dev, int32_t* path_dev, void* workspace_dev, size_t workspace_bytes,
                            void* stream) {
    if (!args) return MOE_ERR_INVALID_ARG;
    moe::EditView e = {};
    e.a = *args;
    int st = check_edit(&e.a);
    if (st != MOE_OK || e.a.streams == 0) return st;
    if (!e.a.tokens_dev || !target_dev || !accepted_dev) return MOE_ERR_INVALID_ARG;
    if (!aligned(target_dev, 4) || !aligned(accepted_dev, 4) || !aligned(next_token_dev, 4) || !aligned(path_dev, 4)) return MOE_ERR_INVALID_ARG;
    size_t need = 0;
    moe_mxfp4_accept_edited_bytes(e.a.streams, e.a.block, e.a.vocab, &need);
    if (!workspace_dev || !aligned(workspace_dev, 8) || workspace_bytes < need) return MOE_ERR_WORKSPACE;
    e.best = static_cast<unsigned long long*>(workspace_dev);
    e.runs = edit_runs(e.a.vocab);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    st = launch_edit<true>(e, cs);
    if (st != MOE_OK) return st;
    return moe::launch_dependent(moe::accept_path_kernel, dim3((unsigned)e.a.streams), dim3(256), 0, cs, e, target_dev, accepted_dev,
                                 next_token_dev, path_dev) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
