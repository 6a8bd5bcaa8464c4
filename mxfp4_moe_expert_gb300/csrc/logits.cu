// Edits of a verify block's logits (moe_mxfp4_edit_logits) and acceptance of chains and trees of drafts with
// them (moe_mxfp4_accept_edited): penalties for tokens that a stream has said or was prompted with, biases and
// grammar masks.
//
// How often a token was said is counted where it is needed: a CTA has a run of tokens of the vocabulary and
// counts those of the stream's history that lie in it in shared memory, once for some positions of the block, so
// nothing is kept from call to call.
#include <cuda_fp16.h>

#include <cmath>

#include "cache.cuh"

namespace moe {

constexpr int kEditThreads = 256;
constexpr int kEach = 16;                          // tokens of the vocabulary of a thread, the same ones for every position
constexpr int kEditRun = kEach * kEditThreads;     // ... and of a CTA
constexpr int kMostRows = 16;                      // positions of a CTA, at most
constexpr uint32_t kPrompted = 1u << 31;           // of a count: the prompt has the token, ...
constexpr uint32_t kInBlock = 1u << 30;            // ... and so has the block, at positions that not all of the CTA's see

struct EditView {
    moe_mxfp4_edit_args a;
    void* out;
    int64_t out_stride;
    unsigned long long* best;                      // acceptance: [rows, runs] largest (key, ~token) of a run, 0 = none
    int runs, rows, groups;                        // of a CTA's positions: how many, and groups of them in a block
};

struct Penalty {
    float repetition, inverse, frequency, presence;
};

// What is taken off a token that was said c times.
__device__ __forceinline__ float penalty_of(uint32_t c, const Penalty& p) {
    return c ? __fmaf_rn(p.frequency, (float)c, p.presence) : 0.0f;
}
// z / r as z (1 / r): half a step more than a division, and a fifth of its instructions.  The operations and their
// roundings are fixed: both entry points give the same value.
__device__ __forceinline__ float edited(float z, bool seen, float off, const Penalty& p) {
    const float factor = seen ? (z > 0 ? p.inverse : p.repetition) : 1.0f;
    return __fsub_rn(__fmul_rn(z, factor), off);
}

// Orderable key of a logit (larger logit, larger key; equal ones, -0 and +0 among them, have one key; NaN ranks as -inf).
__device__ __forceinline__ uint32_t logit_key(float v) {
    uint32_t u = __float_as_uint(v == 0.0f ? 0.0f : v);
    if (v != v) u = 0xFF800000u;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ bool aligned_to_16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

__device__ __forceinline__ int used_positions(const moe_mxfp4_edit_args& a, int s) {
    return a.lengths_dev ? min(a.lengths_dev[s], a.block) : a.block;
}

// What a CTA knows of its run of the vocabulary.
struct EditRun {
    uint32_t count[kEditRun];
    union {
        int entry[kEditRun];                       // 1 + the last entry of the stream's biases for the token, then
        float off[kEditRun];                       // what is taken off it (of one in the block: the bias alone)
    };
    int block_token[64], block_at[64], n_block;    // tokens of the block in the run that only some of the CTA's positions see
    uint32_t top[kMostRows];                       // acceptance: largest key so far of a position,
    unsigned long long best[kMostRows][kEditThreads / 32];   // and each warp's with its token (0: another warp has a larger one)
};

// A token of the block: its edited logit at position b.
__device__ __noinline__ float edited_in_block(const EditView& e, const EditRun& r, const Penalty& p, float z, int i, int64_t row, int b) {
    uint32_t count = r.count[i] & ~kInBlock;
    const bool tree = e.a.mask_dev != nullptr;
    const unsigned long long seen = tree ? (e.a.mask_dev[row] & ((1ull << b) - 1)) | 1ull << b : 0;
    for (int k = 0; k < r.n_block; ++k)
        if (r.block_token[k] == i && (tree ? seen >> r.block_at[k] & 1 : r.block_at[k] <= b)) ++count;
    return edited(z, count != 0, __fadd_rn(penalty_of(count & ~kPrompted, p), r.off[i]), p);
}

// Counts a token of the history.
__device__ __forceinline__ void count_token(EditRun& r, int token, int64_t v0, int n, bool prompt) {
    const uint32_t v = (uint32_t)token - (uint32_t)v0;
    if (v >= (uint32_t)n) return;
    if (prompt) atomicOr(r.count + v, kPrompted);
    else atomicAdd(r.count + v, 1u);
}

template <int kType>
__device__ __forceinline__ float to_f32(uint16_t x) {
    return kType == MOE_DTYPE_BF16 ? __uint_as_float((uint32_t)x << 16) : __half2float(__ushort_as_half(x));
}
template <int kType>
__device__ __forceinline__ uint16_t from_f32(float x) {
    return kType == MOE_DTYPE_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
}

// A thread's kEach tokens of the run, as bits of the logits' type: words of 16 bytes that lie kEditThreads apart
// (kWords, where rows begin on 16 bytes), or single ones.
template <int kType, bool kWords>
struct Mine {
    static constexpr int kSize = kType == MOE_DTYPE_FP32 ? 4 : 2, kPer = 16 / kSize;
    uint32_t bits[kEach * kSize / 4];
    static __device__ __forceinline__ int at(int i) {      // ascending in i
        return kWords ? (i / kPer * kEditThreads + (int)threadIdx.x) * kPer + i % kPer : i * kEditThreads + (int)threadIdx.x;
    }
    __device__ __forceinline__ float get(int i) const {
        if (kType == MOE_DTYPE_FP32) return __uint_as_float(bits[i]);
        return to_f32<kType>((uint16_t)(i & 1 ? bits[i / 2] >> 16 : bits[i / 2]));
    }
    // The largest of the tokens of `which` (-inf: of none; NaN is not taken).  16-bit logits in pairs: -inf is added to those left out.
    __device__ __forceinline__ float most(uint32_t which) const {
        constexpr uint32_t all = (1u << kEach) - 1;
        if (kType == MOE_DTYPE_FP32) {
            float m = -INFINITY;
            if (__all_sync(0xFFFFFFFFu, which == all)) {
#pragma unroll
                for (int i = 0; i < kEach; ++i) m = fmaxf(m, get(i));
            } else {
#pragma unroll
                for (int i = 0; i < kEach; ++i)
                    if (which >> i & 1) m = fmaxf(m, get(i));
            }
            return m;
        }
        uint32_t m = kNone * 0x10001u;
        if (__all_sync(0xFFFFFFFFu, which == all)) {
#pragma unroll
            for (int i = 0; i < kEach / 2; ++i) m = max2(m, bits[i]);
        } else {
#pragma unroll
            for (int w = 0; w < kEach / 8; ++w) {
                const uint32_t out = (~which >> (8 * w) & 0xFFu) * 0x8001u;      // bits 2 p and 2 p + 1 of eight, 16 apart
#pragma unroll
                for (int i = 0; i < 4; ++i) m = max2(m, add2(bits[4 * w + i], (out >> (2 * i) & 0x10001u) * kNone));
            }
        }
        return fmaxf(to_f32<kType>((uint16_t)m), to_f32<kType>((uint16_t)(m >> 16)));
    }
    static constexpr uint32_t kNone = kType == MOE_DTYPE_FP32 ? 0xFF800000u : kType == MOE_DTYPE_BF16 ? 0xFF80u : 0xFC00u;   // -inf
    static __device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y) {
        if (kType == MOE_DTYPE_BF16) asm("max.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(y));
        else asm("max.f16x2 %0, %0, %1;" : "+r"(x) : "r"(y));
        return x;
    }
    static __device__ __forceinline__ uint32_t add2(uint32_t x, uint32_t y) {
        if (kType == MOE_DTYPE_BF16) asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(y));
        else asm("add.rn.f16x2 %0, %0, %1;" : "+r"(x) : "r"(y));
        return x;
    }
    __device__ __forceinline__ void raw(int i, uint32_t x) {
        if (kType == MOE_DTYPE_FP32) bits[i] = x;
        else bits[i / 2] = i & 1 ? (bits[i / 2] & 0xFFFFu) | x << 16 : (bits[i / 2] & 0xFFFF0000u) | x;
    }
    __device__ __forceinline__ void set(int i, float z) {
        if (kType == MOE_DTYPE_FP32) bits[i] = __float_as_uint(z);
        else raw(i, from_f32<kType>(z));
    }
    __device__ __forceinline__ void load(const void* p, int64_t first, int n) {   // first: of the run's first token; n: tokens in it
        if (kWords) {
#pragma unroll
            for (int w = 0; w < kEach / kPer; ++w) {
                const int v = at(w * kPer);
                if (v + kPer <= n) {
                    const uint4 x = __ldcs(reinterpret_cast<const uint4*>(static_cast<const char*>(p) + (first + v) * kSize));
                    bits[4 * w] = x.x;
                    bits[4 * w + 1] = x.y;
                    bits[4 * w + 2] = x.z;
                    bits[4 * w + 3] = x.w;
                } else {
#pragma unroll
                    for (int i = 0; i < kPer; ++i) one(p, first, n, w * kPer + i);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kEach; ++i) one(p, first, n, i);
        }
    }
    __device__ __forceinline__ void one(const void* p, int64_t first, int n, int i) {
        const int v = at(i);
        if (kType == MOE_DTYPE_FP32) raw(i, v < n ? __ldcs(static_cast<const uint32_t*>(p) + first + v) : 0);
        else raw(i, v < n ? __ldcs(static_cast<const uint16_t*>(p) + first + v) : 0);
    }
    // The words (tokens) that have changed, or all.
    __device__ __forceinline__ void store(void* p, int64_t first, int n, uint32_t which) const {
        if (kWords) {
#pragma unroll
            for (int w = 0; w < kEach / kPer; ++w) {
                const int v = at(w * kPer);
                if (!(which >> (w * kPer) & ((1u << kPer) - 1))) continue;
                if (v + kPer <= n) {
                    *reinterpret_cast<uint4*>(static_cast<char*>(p) + (first + v) * kSize) =
                        make_uint4(bits[4 * w], bits[4 * w + 1], bits[4 * w + 2], bits[4 * w + 3]);
                } else {
#pragma unroll
                    for (int i = 0; i < kPer; ++i) put(p, first, n, w * kPer + i);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (which >> i & 1) put(p, first, n, i);
        }
    }
    __device__ __forceinline__ void put(void* p, int64_t first, int n, int i) const {
        const int v = at(i);
        if (v >= n) return;
        if (kType == MOE_DTYPE_FP32) static_cast<uint32_t*>(p)[first + v] = bits[i];
        else static_cast<uint16_t*>(p)[first + v] = (uint16_t)(i & 1 ? bits[i / 2] >> 16 : bits[i / 2]);
    }
    // A bit for each token that the grammar allows and the vocabulary has.
    static __device__ __forceinline__ uint32_t allowed(const uint32_t* words, int n) {   // words: of the run
        uint32_t ok = 0;
        if (kWords) {
#pragma unroll
            for (int w = 0; w < kEach / kPer; ++w) {
                const int v = at(w * kPer);
                if (v < n) ok |= (__ldg(words + (v >> 5)) >> (v & 31) & ((1u << kPer) - 1)) << (w * kPer);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int v = at(i);
                if (v < n) ok |= (__ldg(words + (v >> 5)) >> (v & 31) & 1) << i;
            }
        }
        return ok & in_run(n);
    }
    static __device__ __forceinline__ uint32_t in_run(int n) {
        if (n == kEditRun) return (1u << kEach) - 1;
        uint32_t in = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) in |= (uint32_t)(at(i) < n) << i;
        return in;
    }
};

// A CTA per stream, group of positions and run of the vocabulary.  The next position's logits are under way while
// one's are edited.
template <int kType, bool kWords, bool kAccept>
__global__ void __launch_bounds__(kEditThreads, 3) edit_kernel(EditView e) {
    using M = Mine<kType, kWords>;
    __shared__ EditRun r;
    const moe_mxfp4_edit_args& a = e.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int run = blockIdx.x % e.runs, sg = blockIdx.x / e.runs, s = sg / e.groups, b0 = (sg - s * e.groups) * e.rows;
    const int64_t v0 = (int64_t)run * kEditRun, row0 = (int64_t)s * a.block;
    const int n = (int)min((int64_t)kEditRun, a.vocab - v0);
    grid_dependency_wait();
    const int b1 = min(min(b0 + e.rows, a.block), used_positions(a, s));
    if (b0 >= b1) return;
    M next;
    uint32_t next_ok = M::in_run(n);
    auto fetch = [&](int b) {
        next.load(a.logits_dev, (row0 + b) * a.row_stride + v0, n);
        if (a.allowed_dev) next_ok = M::allowed(a.allowed_dev + (row0 + b) * a.allowed_stride + (v0 >> 5), n);
    };
    fetch(b0);
    // what is known of the run's tokens
    for (int i = tid; i < kEditRun / 4; i += kEditThreads) {
        reinterpret_cast<uint4*>(r.count)[i] = make_uint4(0, 0, 0, 0);
        if (a.bias_begin_dev) reinterpret_cast<uint4*>(r.entry)[i] = make_uint4(0, 0, 0, 0);
    }
    if (tid < kMostRows) r.top[tid] = 0;
    if (tid == 0) r.n_block = 0;
    __syncthreads();
    if (a.history_dev) {
        const int len = (int)min((int64_t)a.history_lengths_dev[s], a.history_room);
        const int prompt = a.prompt_lengths_dev ? a.prompt_lengths_dev[s] : 0;
        const int* h = a.history_dev + s * a.history_stride;
        // (many loads at once, before any of them is counted: one after the other takes a round trip each)
        int i0 = 0;
        if (aligned_to_16(h))
            for (; i0 + 16 * kEditThreads <= len; i0 += 16 * kEditThreads) {
                int4 t[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) t[k] = reinterpret_cast<const int4*>(h + i0)[k * kEditThreads + tid];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int i = i0 + 4 * (k * kEditThreads + tid);
                    count_token(r, t[k].x, v0, n, i < prompt);
                    count_token(r, t[k].y, v0, n, i + 1 < prompt);
                    count_token(r, t[k].z, v0, n, i + 2 < prompt);
                    count_token(r, t[k].w, v0, n, i + 3 < prompt);
                }
            }
        for (; i0 < len; i0 += 8 * kEditThreads) {
            int t[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) t[k] = i0 + k * kEditThreads + tid < len ? h[i0 + k * kEditThreads + tid] : -1;
#pragma unroll
            for (int k = 0; k < 8; ++k) count_token(r, t[k], v0, n, i0 + k * kEditThreads + tid < prompt);
        }
    }
    if (a.tokens_dev)
        for (int j = tid; j < b1; j += kEditThreads) {
            const int64_t v = a.tokens_dev[row0 + j] - v0;
            if (v < 0 || v >= n) continue;
            if (!a.mask_dev && j <= b0) {
                atomicAdd(r.count + v, 1u);        // all positions here see it
            } else {
                atomicOr(r.count + v, kInBlock);
                const int k = atomicAdd(&r.n_block, 1);
                r.block_token[k] = (int)v;
                r.block_at[k] = j;
            }
        }
    if (a.bias_begin_dev) {
        const int64_t end = min((int64_t)a.bias_begin_dev[s + 1], a.bias_entries);
        for (int64_t i = (int64_t)max(a.bias_begin_dev[s], 0) + tid; i < end; i += kEditThreads) {
            const int64_t v = a.bias_ids_dev[i] - v0;
            if (v >= 0 && v < n) atomicMax(r.entry + v, (int)i + 1);
        }
    }
    __syncthreads();
    Penalty p{a.repetition_dev ? a.repetition_dev[s] : 1.0f, 1.0f, a.frequency_dev ? a.frequency_dev[s] : 0.0f,
              a.presence_dev ? a.presence_dev[s] : 0.0f};
    p.inverse = __frcp_rn(p.repetition);
    uint32_t known = 0, seen = 0, in_block = 0;    // bits of the thread's tokens
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const uint32_t c = r.count[M::at(i)];
        seen |= (uint32_t)(c != 0) << i;
        in_block |= (c >> 30 & 1) << i;
    }
    known = seen;
    if (a.bias_begin_dev)
#pragma unroll
        for (int i = 0; i < kEach; ++i) known |= (uint32_t)(r.entry[M::at(i)] != 0) << i;
    // where no lane of the warp knows anything of its i-th token, the warp passes it over together
    const uint32_t warp_knows = __reduce_or_sync(0xFFFFFFFFu, known);
    for (uint32_t left = known; left; left &= left - 1) {
        const int i = __ffs(left) - 1, at = M::at(i), entry = a.bias_begin_dev ? r.entry[at] : 0;
        const float bias = entry ? a.bias_dev[entry - 1] : 0.0f;
        r.off[at] = __fsub_rn(in_block >> i & 1 ? 0.0f : penalty_of(r.count[at] & ~kPrompted, p), bias);
    }
    auto edit = [&](float z, int i, int64_t row, int b) {
        return in_block >> i & 1 ? edited_in_block(e, r, p, z, M::at(i), row, b) : edited(z, seen >> i & 1, r.off[M::at(i)], p);
    };
    for (int b = b0; b < b1; ++b) {
        M z = next;
        const uint32_t ok = next_ok;
        if (b + 1 < b1) fetch(b + 1);
        const int64_t row = row0 + b;
        if (kAccept) {
            // what is known of is edited one by one, in fp32; the rest is compared as it is
            const uint32_t rest = ok & ~known;
            float most = -INFINITY;
            int which = -1;
            if (warp_knows)
#pragma unroll
                for (int i = 0; i < kEach; ++i)
                    if (warp_knows >> i & 1)
                        if ((known & ok) >> i & 1) {
                            const float x = edit(z.get(i), i, row, b);
                            if (x > most) {
                                most = x;
                                which = i;
                            }
                        }
            const float clean = z.most(rest);
            const float all = fmaxf(clean, most);
            const uint32_t key = ok ? logit_key(all) : 0, top = __reduce_max_sync(0xFFFFFFFFu, key);
            unsigned long long best = 0;
            if (top && top >= *static_cast<volatile uint32_t*>(r.top + (b - b0))) {
                uint32_t v = 0xFFFFFFFFu;
                if (key == top) {                  // the first of the thread's largest; of no numbers, the first that is allowed
                    uint32_t is = ok;
                    if (all > -INFINITY) {
                        is = most == all ? 1u << which : 0;
                        if (clean == all)
#pragma unroll
                            for (int i = 0; i < kEach; ++i) is |= (uint32_t)(z.get(i) == all) << i & rest;
                    }
                    v = (uint32_t)(v0 + M::at(__ffs(is) - 1));
                }
                v = __reduce_min_sync(0xFFFFFFFFu, v);
                best = (unsigned long long)top << 32 | (0xFFFFFFFFu - v);
                if (lane == 0) atomicMax(r.top + (b - b0), top);
            }
            if (lane == 0) r.best[b - b0][warp] = best;
        } else {
            if (warp_knows)
#pragma unroll
                for (int i = 0; i < kEach; ++i)
                    if (warp_knows >> i & 1)
                        if (known >> i & 1) z.set(i, edit(z.get(i), i, row, b));
            if (ok != (1u << kEach) - 1)
#pragma unroll
                for (int i = 0; i < kEach; ++i)
                    if (!(ok >> i & 1)) z.raw(i, M::kNone);
            const bool in_place = e.out == a.logits_dev;
            z.store(e.out, row * e.out_stride + v0, n, in_place ? known | ~ok : ~0u);
        }
    }
    if (!kAccept) return;
    __syncthreads();
    if (tid < b1 - b0) {
        unsigned long long best = 0;
        for (int w = 0; w < kEditThreads / 32; ++w) best = r.best[tid][w] > best ? r.best[tid][w] : best;
        e.best[(row0 + b0 + tid) * e.runs + run] = best;
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
    if (a->history_dev && (!a->history_lengths_dev || a->history_room < 0 || a->history_room >= 1 << 29 ||
                           a->history_stride < a->history_room))
        return MOE_ERR_INVALID_ARG;
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

// Positions of a CTA: as many as leave four CTAs for every SM.
void group_rows(moe::EditView* e) {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) sms = 1;
    e->runs = edit_runs(e->a.vocab);
    const int64_t ctas = (int64_t)e->a.streams * e->a.block * e->runs, most = ctas / (4 * sms);
    e->rows = (int)(most < 1 ? 1 : most > moe::kMostRows ? moe::kMostRows : most);
    if (e->rows > e->a.block) e->rows = e->a.block;
    e->groups = (e->a.block + e->rows - 1) / e->rows;
}

template <bool kAccept>
int launch_edit(const moe::EditView& e, cudaStream_t st) {
    const dim3 grid((unsigned)((int64_t)e.a.streams * e.groups * e.runs));
    const int size = e.a.dtype == MOE_DTYPE_FP32 ? 4 : 2;
    const bool words = aligned(e.a.logits_dev, 16) && e.a.row_stride * size % 16 == 0 &&
                       (kAccept || (aligned(e.out, 16) && e.out_stride * size % 16 == 0));
    auto go = [&](auto kern) { return moe::launch_dependent(kern, grid, dim3(moe::kEditThreads), 0, st, e); };
    cudaError_t r;
    if (e.a.dtype == MOE_DTYPE_FP32)
        r = words ? go(moe::edit_kernel<MOE_DTYPE_FP32, true, kAccept>) : go(moe::edit_kernel<MOE_DTYPE_FP32, false, kAccept>);
    else if (e.a.dtype == MOE_DTYPE_BF16)
        r = words ? go(moe::edit_kernel<MOE_DTYPE_BF16, true, kAccept>) : go(moe::edit_kernel<MOE_DTYPE_BF16, false, kAccept>);
    else
        r = words ? go(moe::edit_kernel<MOE_DTYPE_FP16, true, kAccept>) : go(moe::edit_kernel<MOE_DTYPE_FP16, false, kAccept>);
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
    group_rows(&e);
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
    group_rows(&e);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    st = launch_edit<true>(e, cs);
    if (st != MOE_OK) return st;
    return moe::launch_dependent(moe::accept_path_kernel, dim3((unsigned)e.a.streams), dim3(256), 0, cs, e, target_dev, accepted_dev,
                                 next_token_dev, path_dev) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
