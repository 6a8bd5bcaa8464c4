// Edits of a verify block's logits (moe_mxfp4_edit_logits) and acceptance of chains and trees of drafts with
// them (moe_mxfp4_accept_edited): penalties for tokens that a stream has said or was prompted with, biases and
// grammar masks.
//
// How often a token was said is counted where it is needed: a CTA has a run of tokens of the vocabulary and
// counts those of the stream's history that lie in it in shared memory, once for some positions of the block, so
// nothing is kept from call to call.
#include <cuda_fp16.h>

#include <atomic>
#include <cmath>

#include "cache.cuh"

namespace moe {

constexpr int kEditThreads = 256;
constexpr int kEach = 16;                          // tokens of the vocabulary of a thread, the same ones for every position
constexpr int kEditRun = kEach * kEditThreads;     // ... and of a CTA
constexpr int kMostRows = 16;                      // positions of a CTA, at most
constexpr int kMostStages = 5;                     // of the ring of logits on their way
constexpr int kEditShared = 70 * 1024;             // shared memory of a CTA, at most: three fit an SM
constexpr uint32_t kPrompted = 1u << 31;           // of a count: the prompt has the token, ...
constexpr uint32_t kInBlock = 1u << 30;            // ... and so has the block, at positions that not all of the CTA's see

struct EditView {
    moe_mxfp4_edit_args a;
    void* out;
    int64_t out_stride;
    unsigned long long* best;                      // acceptance: [rows, runs] largest (key, ~token) of a run, 0 = none
    int runs, rows, groups;                        // of a CTA's positions: how many, and groups of them in a block
    int stages;                                    // rows of the ring
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

template <int kType>
__device__ __forceinline__ float to_f32(uint16_t x) {
    return kType == MOE_DTYPE_BF16 ? __uint_as_float((uint32_t)x << 16) : __half2float(__ushort_as_half(x));
}
template <int kType>
__device__ __forceinline__ uint16_t from_f32(float x) {
    return kType == MOE_DTYPE_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
}

__device__ __forceinline__ void copy_16(void* smem, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_4(void* smem, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits for the oldest stage of a ring that is full.
__device__ __forceinline__ void copies_wait(int stages) {
    if (stages == 1) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (stages == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else if (stages == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (stages == 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
    else asm volatile("cp.async.wait_group 4;" ::: "memory");
}

// A position's logits of the run, in shared memory: token v at place v.
template <int kType>
struct Row {
    static constexpr int kSize = kType == MOE_DTYPE_FP32 ? 4 : 2;
    static constexpr uint32_t kNone = kType == MOE_DTYPE_FP32 ? 0xFF800000u : kType == MOE_DTYPE_BF16 ? 0xFF80u : 0xFC00u;   // -inf
    char* p;
    __device__ __forceinline__ float get(int v) const {
        if (kType == MOE_DTYPE_FP32) return reinterpret_cast<const float*>(p)[v];
        return to_f32<kType>(reinterpret_cast<const uint16_t*>(p)[v]);
    }
    __device__ __forceinline__ void put(int v, float z) const {
        if (kType == MOE_DTYPE_FP32) reinterpret_cast<float*>(p)[v] = z;
        else reinterpret_cast<uint16_t*>(p)[v] = from_f32<kType>(z);
    }
    __device__ __forceinline__ void put_none(int v) const {
        if (kType == MOE_DTYPE_FP32) reinterpret_cast<uint32_t*>(p)[v] = kNone;
        else reinterpret_cast<uint16_t*>(p)[v] = (uint16_t)kNone;
    }
};

// A thread's kEach tokens of the run, as bits of the logits' type: words of 16 bytes that lie kEditThreads apart
// (kWords, where rows begin on 16 bytes), or single ones.  Pointers are of the run's first token; n: tokens of the run.
template <int kType, bool kWords>
struct Mine {
    static constexpr int kSize = Row<kType>::kSize, kPer = 16 / kSize, kWarps = kEditThreads / 32;
    static constexpr uint32_t kAll = (1u << kEach) - 1, kNone = Row<kType>::kNone;
    uint32_t bits[kEach * kSize / 4];
    static __device__ __forceinline__ int at(int i) {      // ascending in i
        return kWords ? (i / kPer * kEditThreads + (int)threadIdx.x) * kPer + i % kPer : i * kEditThreads + (int)threadIdx.x;
    }
    __device__ __forceinline__ float get(int i) const {
        if (kType == MOE_DTYPE_FP32) return __uint_as_float(bits[i]);
        return to_f32<kType>((uint16_t)(i & 1 ? bits[i / 2] >> 16 : bits[i / 2]));
    }
    __device__ __forceinline__ void raw(int i, uint32_t x) {
        if (kType == MOE_DTYPE_FP32) bits[i] = x;
        else bits[i / 2] = i & 1 ? (bits[i / 2] & 0xFFFFu) | x << 16 : (bits[i / 2] & 0xFFFF0000u) | x;
    }
    __device__ __forceinline__ uint32_t raw(int i) const {
        return kType == MOE_DTYPE_FP32 ? bits[i] : i & 1 ? bits[i / 2] >> 16 : bits[i / 2] & 0xFFFFu;
    }
    static __device__ __forceinline__ uint32_t read(const void* p, int v) {
        return kType == MOE_DTYPE_FP32 ? static_cast<const uint32_t*>(p)[v] : static_cast<const uint16_t*>(p)[v];
    }
    static __device__ __forceinline__ void write(void* p, int v, uint32_t x) {
        if (kType == MOE_DTYPE_FP32) static_cast<uint32_t*>(p)[v] = x;
        else static_cast<uint16_t*>(p)[v] = (uint16_t)x;
    }

    // kWords: the thread's words into a row of the ring.
    static __device__ __forceinline__ void copy(char* row, const char* src, int n) {
#pragma unroll
        for (int w = 0; w < kEach / kPer; ++w) {
            const int v = at(w * kPer);
            if (n == kEditRun || v + kPer <= n) copy_16(row + v * kSize, src + v * kSize);
            else
                for (int i = v; i < n; ++i) write(row, i, read(src, i));   // (the vocabulary's last word)
        }
    }
    __device__ __forceinline__ void take(const char* row) {
        if (kWords) {
#pragma unroll
            for (int w = 0; w < kEach / kPer; ++w) {
                const uint4 x = *reinterpret_cast<const uint4*>(row + at(w * kPer) * kSize);
                bits[4 * w] = x.x;
                bits[4 * w + 1] = x.y;
                bits[4 * w + 2] = x.z;
                bits[4 * w + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kEach; ++i) raw(i, read(row, at(i)));
        }
    }
    // Single tokens: from memory into registers, and on into the ring.
    __device__ __forceinline__ void load(const char* src, int n) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) raw(i, at(i) < n ? read(src, at(i)) : 0);
    }
    __device__ __forceinline__ void spill(char* row) const {
#pragma unroll
        for (int i = 0; i < kEach; ++i) write(row, at(i), raw(i));
    }
    // To the output: the tokens of `which`, and what shares a word with them.
    __device__ __forceinline__ void store(char* dst, int n, uint32_t which) const {
        if (kWords) {
#pragma unroll
            for (int w = 0; w < kEach / kPer; ++w) {
                const int v = at(w * kPer);
                if (!(which >> (w * kPer) & ((1u << kPer) - 1))) continue;
                if (n == kEditRun || v + kPer <= n) {
                    *reinterpret_cast<uint4*>(dst + v * kSize) = make_uint4(bits[4 * w], bits[4 * w + 1], bits[4 * w + 2], bits[4 * w + 3]);
                } else {
#pragma unroll
                    for (int i = w * kPer; i < w * kPer + kPer; ++i)
                        if (at(i) < n) write(dst, at(i), raw(i));
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if ((which >> i & 1) && at(i) < n) write(dst, at(i), raw(i));
        }
    }

    // The grammar's words of a warp's tokens: kEach of them, on their way (kWords) ...
    static __device__ __forceinline__ int word_of(int k) { return (k / kPer * kWarps + (int)(threadIdx.x >> 5)) * kPer + k % kPer; }
    static __device__ __forceinline__ void copy_allowed(uint32_t* to, const uint32_t* words, int n) {
        const int lane = threadIdx.x & 31;
        if (lane < kEach && 32 * word_of(lane) < n) copy_4(to + lane, words + word_of(lane));
    }
    // ... and a bit for each of the thread's tokens, ...
    static __device__ __forceinline__ uint32_t take_allowed(const uint32_t* from) {
        uint32_t x = 0;
#pragma unroll
        for (int w = 0; w < kEach / kPer; ++w) {
            const int bit = (threadIdx.x & 31) * kPer;
            x |= (from[w * kPer + bit / 32] >> (bit & 31) & ((1u << kPer) - 1)) << (w * kPer);
        }
        return x;
    }
    // ... or for token v of the warp's.
    static __device__ __forceinline__ bool is_allowed(const uint32_t* from, int v) {
        return from[(v >> 5) / (kPer * kWarps) * kPer + (v >> 5) % kPer] >> (v & 31) & 1;
    }
    static __device__ __forceinline__ uint32_t load_allowed(const uint32_t* words, int n) {
        uint32_t ok = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (at(i) < n) ok |= (__ldg(words + (at(i) >> 5)) >> (at(i) & 31) & 1) << i;
        return ok;
    }
    static __device__ __forceinline__ uint32_t in_run(int n) {
        if (n == kEditRun) return kAll;
        uint32_t in = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) in |= (uint32_t)(at(i) < n) << i;
        return in;
    }

    // The largest of the tokens of `which` (-inf: of none; NaN is not taken).  16-bit logits in pairs: -inf is added to those left out.
    __device__ __forceinline__ float most(uint32_t which) const {
        const bool all = __all_sync(0xFFFFFFFFu, which == kAll);
        if (kType == MOE_DTYPE_FP32) {
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (all || (which >> i & 1)) m = fmaxf(m, get(i));
            return m;
        }
        uint32_t m = kNone * 0x10001u;
        if (all) {
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
};

// Counts a token of the history.
__device__ __forceinline__ void count_token(uint32_t* count, int token, int64_t v0, int n, bool prompt) {
    const uint32_t v = (uint32_t)token - (uint32_t)v0;
    if (v >= (uint32_t)n) return;
    if (prompt) atomicOr(count + v, kPrompted);
    else atomicAdd(count + v, 1u);
}
__device__ __forceinline__ void count_history(uint32_t* count, const int* h, int len, int prompt, int64_t v0, int n) {
    // (many loads at once, before any of them is counted: one after the other takes a round trip each)
    const int tid = threadIdx.x;
    int i0 = 0;
    if (aligned_to_16(h))
        for (; i0 + 16 * kEditThreads <= len; i0 += 16 * kEditThreads) {
            int4 t[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) t[k] = reinterpret_cast<const int4*>(h + i0)[k * kEditThreads + tid];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = i0 + 4 * (k * kEditThreads + tid);
                count_token(count, t[k].x, v0, n, i < prompt);
                count_token(count, t[k].y, v0, n, i + 1 < prompt);
                count_token(count, t[k].z, v0, n, i + 2 < prompt);
                count_token(count, t[k].w, v0, n, i + 3 < prompt);
            }
        }
    for (; i0 < len; i0 += 8 * kEditThreads) {
        int t[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) t[k] = i0 + k * kEditThreads + tid < len ? h[i0 + k * kEditThreads + tid] : -1;
#pragma unroll
        for (int k = 0; k < 8; ++k) count_token(count, t[k], v0, n, i0 + k * kEditThreads + tid < prompt);
    }
}

// A CTA per stream, group of positions and run of the vocabulary.  It counts the run's tokens of the history once;
// each warp lists those of its tokens that something is known of, with what is taken off them.  The logits of the
// positions to come are on their way meanwhile, into a ring of rows in shared memory, which each thread copies its own
// words of (rows that do not begin on 16 bytes: the next one, in registers).  Of each position a warp edits the tokens on its
// list in the ring, a lane a token, and then takes its row as it is: a vocabulary has few tokens that a stream has
// said, and looking for them in every row took four times what the rest does.
template <int kType, bool kWords, bool kAccept>
__global__ void __launch_bounds__(kEditThreads, 3) edit_kernel(EditView e) {
    using M = Mine<kType, kWords>;
    constexpr int kWarps = kEditThreads / 32, kRowBytes = kEditRun * M::kSize;
    constexpr uint32_t kListSeen = 1u << 15, kListInBlock = 1u << 14;
    extern __shared__ uint4 dynamic[];
    __shared__ int block_token[64], block_at[64], n_block;      // tokens of the block that only some of the CTA's positions see
    __shared__ uint32_t top_key[kMostRows];                     // acceptance: largest key so far of a position,
    __shared__ unsigned long long warp_best[kMostRows][kWarps]; // and each warp's with its token (0: another warp has a larger one)
    __shared__ uint32_t grammar[kMostStages][kWarps][kEach];
    const moe_mxfp4_edit_args& a = e.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int run = blockIdx.x % e.runs, sg = blockIdx.x / e.runs, s = sg / e.groups, b0 = (sg - s * e.groups) * e.rows;
    const int64_t v0 = (int64_t)run * kEditRun, row0 = (int64_t)s * a.block;
    const int n = (int)min((int64_t)kEditRun, a.vocab - v0);
    uint32_t* const count = reinterpret_cast<uint32_t*>(dynamic);              // later, as fp32: what is taken off the token
    uint16_t* const list = reinterpret_cast<uint16_t*>(count + kEditRun) + warp * 32 * kEach;
    int* const entry = a.bias_begin_dev ? reinterpret_cast<int*>(dynamic + kEditRun / 4 + kEditRun / 8) : nullptr;
    float* const bias = reinterpret_cast<float*>(entry);       // 1 + the last entry of a token, then its bias
    char* const ring = reinterpret_cast<char*>(dynamic + kEditRun / 4 + kEditRun / 8 + (entry ? kEditRun / 4 : 0));
    grid_dependency_wait();
    const int b1 = min(min(b0 + e.rows, a.block), used_positions(a, s));
    if (b0 >= b1) return;
    // rows on their way
    const char* src = static_cast<const char*>(a.logits_dev) + ((row0 + b0) * a.row_stride + v0) * M::kSize;
    const uint32_t* words = a.allowed_dev ? a.allowed_dev + (row0 + b0) * a.allowed_stride + (v0 >> 5) : nullptr;
    const uint32_t in_run = M::in_run(n);
    M next;
    uint32_t next_ok = in_run;
    int ahead = b0, ahead_stage = 0, stage = 0;
    auto fetch = [&] {
        if (ahead < b1) {
            if (kWords) {
                M::copy(ring + ahead_stage * kRowBytes, src, n);
                if (words) M::copy_allowed(grammar[ahead_stage][warp], words, n);
                if (++ahead_stage == e.stages) ahead_stage = 0;
            } else {
                next.load(src, n);
                if (words) next_ok = M::load_allowed(words, n);
            }
            src += a.row_stride * M::kSize;
            if (words) words += a.allowed_stride;
            ++ahead;
        }
        if (kWords) copies_commit();
    };
    for (int i = 0; i < (kWords ? e.stages : 1); ++i) fetch();
    // what is known of the run's tokens
    for (int i = tid; i < kEditRun / 4; i += kEditThreads) {
        reinterpret_cast<uint4*>(count)[i] = make_uint4(0, 0, 0, 0);
        if (entry) reinterpret_cast<uint4*>(entry)[i] = make_uint4(0, 0, 0, 0);
    }
    if (tid < kMostRows) top_key[tid] = 0;
    if (tid == 0) n_block = 0;
    __syncthreads();
    if (a.history_dev)
        count_history(count, a.history_dev + s * a.history_stride, (int)min((int64_t)a.history_lengths_dev[s], a.history_room),
                      a.prompt_lengths_dev ? a.prompt_lengths_dev[s] : 0, v0, n);
    if (a.tokens_dev)
        for (int j = tid; j < b1; j += kEditThreads) {
            const int64_t v = a.tokens_dev[row0 + j] - v0;
            if (v < 0 || v >= n) continue;
            if (!a.mask_dev && j <= b0) {
                atomicAdd(count + v, 1u);          // all positions here see it
            } else {
                atomicOr(count + v, kInBlock);
                const int k = atomicAdd(&n_block, 1);
                block_token[k] = (int)v;
                block_at[k] = j;
            }
        }
    if (entry) {
        const int64_t end = min((int64_t)a.bias_begin_dev[s + 1], a.bias_entries);
        for (int64_t i = (int64_t)max(a.bias_begin_dev[s], 0) + tid; i < end; i += kEditThreads) {
            const int64_t v = a.bias_ids_dev[i] - v0;
            if (v >= 0 && v < n) atomicMax(entry + v, (int)i + 1);
        }
    }
    Penalty p{a.repetition_dev ? a.repetition_dev[s] : 1.0f, 1.0f, a.frequency_dev ? a.frequency_dev[s] : 0.0f,
              a.presence_dev ? a.presence_dev[s] : 0.0f};
    p.inverse = __frcp_rn(p.repetition);
    __syncthreads();
    uint32_t known = 0;                            // bits of the thread's tokens
#pragma unroll
    for (int i = 0; i < kEach; ++i) known |= (uint32_t)(count[M::at(i)] != 0) << i;
    if (entry)
#pragma unroll
        for (int i = 0; i < kEach; ++i) known |= (uint32_t)(entry[M::at(i)] != 0) << i;
    int place = __popc(known), listed;             // of the thread's tokens in the warp's list
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, place, o);
        if (lane >= o) place += x;
    }
    listed = __shfl_sync(0xFFFFFFFFu, place, 31);
    place -= __popc(known);
    for (uint32_t left = known; left; left &= left - 1) {
        const int v = M::at(__ffs(left) - 1);
        const uint32_t c = count[v];
        if (entry && entry[v]) bias[v] = a.bias_dev[entry[v] - 1];
        list[place++] = (uint16_t)(v | (c ? kListSeen : 0) | (c & kInBlock ? kListInBlock : 0));
        if (!(c & kInBlock)) reinterpret_cast<float*>(count)[v] = __fsub_rn(penalty_of(c & ~kPrompted, p), entry ? bias[v] : 0.0f);
    }
    __syncwarp();
    char* dst = static_cast<char*>(e.out) + ((row0 + b0) * e.out_stride + v0) * M::kSize;
    const uint32_t changed = e.out == a.logits_dev ? known : M::kAll;
    for (int b = b0; b < b1; ++b) {
        M z;
        uint32_t ok = in_run;
        const Row<kType> row{ring + stage * kRowBytes};
        const uint32_t* const allowed = grammar[stage][warp];
        if (kWords) {
            copies_wait(e.stages);
            __syncwarp();
            if (a.allowed_dev) ok &= M::take_allowed(allowed);
        } else {
            next.spill(row.p);
            ok = next_ok;
            __syncwarp();
        }
        float most = -INFINITY;                    // of the tokens on the list
        int which = kEditRun;
        for (int k = lane; k < listed; k += 32) {
            const uint32_t item = list[k];
            const int v = item & (kEditRun - 1);
            float off = reinterpret_cast<const float*>(count)[v];
            bool seen = item & kListSeen;
            if (item & kListInBlock) {
                uint32_t c = count[v] & ~kInBlock;
                const bool tree = a.mask_dev != nullptr;
                const unsigned long long sees = tree ? (a.mask_dev[row0 + b] & ((1ull << b) - 1)) | 1ull << b : 0;
                for (int j = 0; j < n_block; ++j)
                    if (block_token[j] == v && (tree ? sees >> block_at[j] & 1 : block_at[j] <= b)) ++c;
                seen = c != 0;
                off = __fsub_rn(penalty_of(c & ~kPrompted, p), entry ? bias[v] : 0.0f);
            }
            const float x = edited(row.get(v), seen, off, p);
            if (!kAccept) {
                row.put(v, x);
            } else {
                row.put_none(v);
                const bool may = !a.allowed_dev || (kWords ? M::is_allowed(allowed, v)
                                                           : a.allowed_dev[(row0 + b) * a.allowed_stride + ((v0 + v) >> 5)] >> (v & 31) & 1);
                if (may && (x > most || (x == most && v < which))) {
                    most = x;
                    which = v;
                }
            }
        }
        __syncwarp();
        z.take(row.p);
        if (kWords) {
            if (++stage == e.stages) stage = 0;
            __syncwarp();                          // (the grammar's words are copied by other lanes)
        }
        fetch();
        if (kAccept) {
            const float rest = z.most(ok), all = fmaxf(rest, most);
            const uint32_t key = ok || which < kEditRun ? logit_key(all) : 0, top = __reduce_max_sync(0xFFFFFFFFu, key);
            unsigned long long best = 0;
            if (top && top >= *static_cast<volatile uint32_t*>(top_key + (b - b0))) {
                uint32_t v = 0xFFFFFFFFu;
                if (key == top) {                  // the first of the largest; of no numbers, the first that is allowed
                    uint32_t is = ok;
                    if (all > -INFINITY) {
                        is = 0;
#pragma unroll
                        for (int i = 0; i < kEach; ++i) is |= (uint32_t)(z.get(i) == all) << i;
                        is &= ok;
                    }
                    if (is) v = (uint32_t)M::at(__ffs(is) - 1);
                    if (which < kEditRun && most == all) v = min(v, (uint32_t)which);
                    v += (uint32_t)v0;
                }
                v = __reduce_min_sync(0xFFFFFFFFu, v);
                best = (unsigned long long)top << 32 | (0xFFFFFFFFu - v);
                if (lane == 0) atomicMax(top_key + (b - b0), top);
            }
            if (lane == 0) warp_best[b - b0][warp] = best;
        } else {
            if (ok != M::kAll)
#pragma unroll
                for (int i = 0; i < kEach; ++i)
                    if (!(ok >> i & 1)) z.raw(i, M::kNone);
            z.store(dst, n, changed | ~ok);
            dst += e.out_stride * M::kSize;
        }
    }
    if (!kAccept) return;
    __syncthreads();
    if (tid < b1 - b0) {
        unsigned long long best = 0;
        for (int w = 0; w < kWarps; ++w) best = warp_best[tid][w] > best ? warp_best[tid][w] : best;
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

template <int kType, bool kWords, bool kAccept>
cudaError_t launch_edit(const moe::EditView& e, dim3 grid, size_t shared, cudaStream_t st) {
    static std::atomic<uint64_t> allowed{0};       // devices on which the kernel may have its shared memory
    int dev = 0;
    cudaError_t r = cudaGetDevice(&dev);
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (r == cudaSuccess && !(allowed.load(std::memory_order_acquire) & bit)) {
        r = cudaFuncSetAttribute(moe::edit_kernel<kType, kWords, kAccept>, cudaFuncAttributeMaxDynamicSharedMemorySize, moe::kEditShared);
        if (r == cudaSuccess) allowed.fetch_or(bit, std::memory_order_release);
    }
    return r != cudaSuccess ? r : moe::launch_dependent(moe::edit_kernel<kType, kWords, kAccept>, grid, dim3(moe::kEditThreads), shared, st, e);
}

template <bool kAccept>
int launch_edit(moe::EditView e, cudaStream_t st) {
    const dim3 grid((unsigned)((int64_t)e.a.streams * e.groups * e.runs));
    const int size = e.a.dtype == MOE_DTYPE_FP32 ? 4 : 2;
    const bool words = aligned(e.a.logits_dev, 16) && e.a.row_stride * size % 16 == 0 &&
                       (kAccept || (aligned(e.out, 16) && e.out_stride * size % 16 == 0));
    // the counts and lists, the biases if there are any, and as many rows of logits as there is room and positions for
    const int arrays = moe::kEditRun * (4 + 2 + (e.a.bias_begin_dev ? 4 : 0)), stage = moe::kEditRun * size;
    e.stages = (moe::kEditShared - arrays) / stage;
    if (e.stages > moe::kMostStages) e.stages = moe::kMostStages;
    if (e.stages > e.rows) e.stages = e.rows;
    if (!words) e.stages = 1;
    const size_t shared = arrays + (size_t)e.stages * stage;
    auto go = [&](auto launch) { return launch(e, grid, shared, st); };
    cudaError_t r;
    if (e.a.dtype == MOE_DTYPE_FP32)
        r = words ? go(launch_edit<MOE_DTYPE_FP32, true, kAccept>) : go(launch_edit<MOE_DTYPE_FP32, false, kAccept>);
    else if (e.a.dtype == MOE_DTYPE_BF16)
        r = words ? go(launch_edit<MOE_DTYPE_BF16, true, kAccept>) : go(launch_edit<MOE_DTYPE_BF16, false, kAccept>);
    else
        r = words ? go(launch_edit<MOE_DTYPE_FP16, true, kAccept>) : go(launch_edit<MOE_DTYPE_FP16, false, kAccept>);
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
