// Edits of a verify block's logits (moe_mxfp4_edit_logits) and acceptance of chains and trees of drafts with
// them (moe_mxfp4_accept_edited): penalties for tokens that a stream has said or was prompted with, biases and
// grammar masks.
//
// A vocabulary has few tokens that a stream has said, and the rest is copied, or compared, as it is.  How
// often a token was said is counted where it is needed: a CTA has a run of tokens of the vocabulary and counts
// those of the stream's history that lie in it in shared memory, once for some positions of the block, so
// nothing is kept from call to call.
#include <cuda_fp16.h>

#include <cmath>

#include "cache.cuh"

namespace moe {

constexpr int kEditThreads = 256;
constexpr int kEditRun = 4096;                     // tokens of the vocabulary of a CTA
constexpr int kParts = 4;                          // of a run, at most: a warp's work at a time
constexpr int kMostRows = 16;                      // positions of a CTA, at most
constexpr uint32_t kPrompted = 1u << 31;           // of a count: the prompt has the token, ...
constexpr uint32_t kInBlock = 1u << 30;            // ... and so has the block, at positions that not all of the CTA's see

struct EditView {
    moe_mxfp4_edit_args a;
    void* out;
    int64_t out_stride;
    unsigned long long* best;                      // acceptance: [rows, runs] largest (key, ~token) of a run, 0 = none
    int runs, rows, groups;                        // of a CTA's positions: how many, and groups of them in a block
    int parts;                                     // of a run: a power of two up to kParts
};

struct Penalty {
    float repetition, frequency, presence;
};

// What is taken off a token that was said c times.
__device__ __forceinline__ float penalty_of(uint32_t c, const Penalty& p) {
    return c ? __fmaf_rn(p.frequency, (float)c, p.presence) : 0.0f;
}
// The operations and their roundings are fixed: both entry points give the same value.  (A product with the rounded reciprocal
// is off by up to 1.5 steps instead of a half, and infinite below 2^-128.  It takes 12.1 us where this takes 12.9, for
// acceptance of 1 x 8 positions of 151936 behind 4000 tokens, and 53.4 where this takes 54.9, for 48 x 11.)
__device__ __forceinline__ float edited(float z, bool seen, float off, const Penalty& p) {
    if (seen && p.repetition != 1.0f) z = z > 0 ? __fdiv_rn(z, p.repetition) : __fmul_rn(z, p.repetition);
    return __fsub_rn(z, off);
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

// Logits as bits of their type.
template <int kType>
struct Bits {
    static constexpr int kSize = kType == MOE_DTYPE_FP32 ? 4 : 2;
    static constexpr uint32_t kNone = kType == MOE_DTYPE_FP32 ? 0xFF800000u : kType == MOE_DTYPE_BF16 ? 0xFF80u : 0xFC00u;   // -inf
    static __device__ __forceinline__ uint32_t read(const char* row, int v) {
        return kType == MOE_DTYPE_FP32 ? reinterpret_cast<const uint32_t*>(row)[v] : reinterpret_cast<const uint16_t*>(row)[v];
    }
    static __device__ __forceinline__ void write(char* row, int v, uint32_t bits) {
        if (kType == MOE_DTYPE_FP32) reinterpret_cast<uint32_t*>(row)[v] = bits;
        else reinterpret_cast<uint16_t*>(row)[v] = (uint16_t)bits;
    }
    static __device__ __forceinline__ float value(uint32_t bits) {
        return kType == MOE_DTYPE_FP32 ? __uint_as_float(bits) : to_f32<kType>((uint16_t)bits);
    }
    static __device__ __forceinline__ uint32_t of(float z) { return kType == MOE_DTYPE_FP32 ? __float_as_uint(z) : from_f32<kType>(z); }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        if (kType == MOE_DTYPE_BF16) asm("max.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
        else asm("max.f16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
        return a;
    }
    static __device__ __forceinline__ uint32_t add2(uint32_t a, uint32_t b) {
        if (kType == MOE_DTYPE_BF16) asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
        else asm("add.rn.f16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
        return a;
    }
};

// A warp's four loads of 512 bytes of a row, from a token that lies on 16 bytes: a lane has 4 words of kPer tokens, and a bit
// for each of its tokens (token i of word w: bit w kPer + i).  kShift: the first of them is any token of the run (rows that do not
// begin on 16 bytes), and its bits lie anywhere in the grammar's words.
template <int kType, bool kShift>
struct Batch {
    using B = Bits<kType>;
    static constexpr int kPer = 16 / B::kSize, kTokens = 4 * 32 * kPer, kLane = 4 * kPer;
    static constexpr uint32_t kAll = kLane == 32 ? 0xFFFFFFFFu : (1u << (kLane & 31)) - 1, kWord = (1u << kPer) - 1;
    uint4 x[4];
    uint32_t ok;                                   // allowed
    static __device__ __forceinline__ int token(int w, int lane) { return (w * 32 + lane) * kPer; }
    // The bits of the tokens from base on in a row of bits: the words' tokens lie a whole number of its words apart, kPer.
    static __device__ __forceinline__ uint32_t bits_from(const uint32_t* bits, int base, int w, int lane) {
        const int v = base + token(0, lane);
        if (!kShift) {                             // (a byte holds them)
            const uint32_t t = reinterpret_cast<const uint8_t*>(bits)[v / 8 + 4 * kPer * w];
            return kPer == 8 ? t : t >> (v & 7) & kWord;
        }
        const uint32_t lo = bits[(v >> 5) + kPer * w], hi = (v & 31) + kPer > 32 ? bits[(v >> 5) + kPer * w + 1] : 0;
        return __funnelshift_r(lo, hi, v & 31) & kWord;
    }
    // The run's row and grammar, tokens base .. last; words that reach beyond are left out.
    __device__ __forceinline__ void load(const char* row, const uint32_t* allowed, int base, int last, int lane) {
        const uint4* p = reinterpret_cast<const uint4*>(row + base * B::kSize) + lane;
        if (base + kTokens <= last) {
#pragma unroll
            for (int w = 0; w < 4; ++w) x[w] = __ldcs(p + 32 * w);
            ok = kAll;
            if (allowed) {
                ok = 0;
#pragma unroll
                for (int w = 0; w < 4; ++w) ok |= bits_from(allowed, base, w, lane) << (kPer * w);
            }
        } else {
            ok = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                x[w] = make_uint4(0, 0, 0, 0);
                if (base + token(w, lane) + kPer > last) continue;
                x[w] = __ldcs(p + 32 * w);
                ok |= (allowed ? bits_from(allowed, base, w, lane) : kWord) << (kPer * w);
            }
        }
    }
    // Those of the tokens that something is known of.
    static __device__ __forceinline__ uint32_t known_bits(const uint32_t* known, const uint32_t (*known_lane)[32], int base, int last, int lane) {
        if (!kShift) return known_lane[base / kTokens][lane];
        uint32_t t = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w)
            if (base + token(w, lane) + kPer <= last) t |= bits_from(known, base, w, lane) << (kPer * w);
        return t;
    }
    static __device__ __forceinline__ uint32_t part(const uint4& t, int i) { return i == 0 ? t.x : i == 1 ? t.y : i == 2 ? t.z : t.w; }
    __device__ __forceinline__ uint32_t get(int w, int i) const {
        if (kType == MOE_DTYPE_FP32) return part(x[w], i);
        const uint32_t t = part(x[w], i / 2);
        return i & 1 ? t >> 16 : t & 0xFFFFu;
    }
    // The largest of those with their bit (-inf: of none; NaN is not taken).  16-bit logits in pairs: -inf is added to those left out.
    __device__ __forceinline__ float most(uint32_t bits) const {
        const bool all = __all_sync(0xFFFFFFFFu, bits == kAll);
        if (kType == MOE_DTYPE_FP32) {
            float m = -INFINITY;
            if (all) {
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    m = fmaxf(m, fmaxf(fmaxf(B::value(x[w].x), B::value(x[w].y)), fmaxf(B::value(x[w].z), B::value(x[w].w))));
            } else {
#pragma unroll
                for (int w = 0; w < 4; ++w)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (bits >> (4 * w + i) & 1) m = fmaxf(m, B::value(part(x[w], i)));
            }
            return m;
        }
        uint32_t m = B::kNone * 0x10001u;
        if (all) {
#pragma unroll
            for (int w = 0; w < 4; ++w) m = B::max2(m, B::max2(B::max2(x[w].x, x[w].y), B::max2(x[w].z, x[w].w)));
        } else {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t out = (~bits >> (8 * w) & 0xFFu) * 0x8001u;       // bits 2 i and 2 i + 1, 16 apart
#pragma unroll
                for (int i = 0; i < 4; ++i) m = B::max2(m, B::add2(part(x[w], i), (out >> (2 * i) & 0x10001u) * B::kNone));
            }
        }
        return fmaxf(to_f32<kType>((uint16_t)m), to_f32<kType>((uint16_t)(m >> 16)));
    }
    // The first token with its bit and the value z; -1: none.
    __device__ __forceinline__ int find(uint32_t bits, float z, int lane) const {
        uint32_t is = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
            for (int i = 0; i < kPer; ++i) is |= (uint32_t)(B::value(get(w, i)) == z) << (w * kPer + i);
        is &= bits;
        const int k = __ffs(is) - 1;
        return k < 0 ? -1 : token(k / kPer, lane) + k % kPer;
    }
    // Those without their bit as -inf.
    __device__ __forceinline__ void hide() {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (kType == MOE_DTYPE_FP32) {
                if (!(ok >> (4 * w) & 1)) x[w].x = B::kNone;
                if (!(ok >> (4 * w + 1) & 1)) x[w].y = B::kNone;
                if (!(ok >> (4 * w + 2) & 1)) x[w].z = B::kNone;
                if (!(ok >> (4 * w + 3) & 1)) x[w].w = B::kNone;
            } else {
                const uint32_t out = (~ok >> (8 * w) & 0xFFu) * 0x8001u;
                auto masked = [&](uint32_t t, int i) {
                    const uint32_t m = (out >> (2 * i) & 0x10001u) * 0xFFFFu;
                    return (t & ~m) | (B::kNone * 0x10001u & m);
                };
                x[w] = make_uint4(masked(x[w].x, 0), masked(x[w].y, 1), masked(x[w].z, 2), masked(x[w].w, 3));
            }
        }
    }
};

// Calls f(token, whether the prompt has it) for the tokens of the history from place i0 on that fall to this thread.  (Many loads at
// once, before any of them is looked at: one after the other takes a round trip each.)
template <class F>
__device__ __forceinline__ void for_history(const int* h, int i0, int len, int prompt, F f) {
    const int tid = threadIdx.x;
    if (aligned_to_16(h))
        for (; i0 + 16 * kEditThreads <= len; i0 += 16 * kEditThreads) {
            int4 t[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) t[k] = reinterpret_cast<const int4*>(h + i0)[k * kEditThreads + tid];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = i0 + 4 * (k * kEditThreads + tid);
                f(t[k].x, i < prompt);
                f(t[k].y, i + 1 < prompt);
                f(t[k].z, i + 2 < prompt);
                f(t[k].w, i + 3 < prompt);
            }
        }
    for (; i0 < len; i0 += 8 * kEditThreads) {
        int t[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) t[k] = i0 + k * kEditThreads + tid < len ? h[i0 + k * kEditThreads + tid] : -1;
#pragma unroll
        for (int k = 0; k < 8; ++k) f(t[k], i0 + k * kEditThreads + tid < prompt);
    }
}
__device__ __forceinline__ void prefetch_run(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

__device__ __forceinline__ bool bit_at(const uint32_t* words, int v) { return words[v >> 5] >> (v & 31) & 1; }

// A CTA per run of the vocabulary, stream and group of positions.  It counts the run's tokens of the history once
// and lists those that something is known of, with what is taken off them: few of a vocabulary, so they are edited
// apart from the rest, a lane a token, and passing them over costs a bit each.  Then a warp takes a position's run, or
// a part of it, at a time: the rest is copied, or compared, as it is.  Low tokens are the common ones and have the
// longest lists, so their CTAs come first.
//
// Bound by HBM where rows are written: 32 x 8 positions of 151936 fp32 logits (311 MB read and written) in 56 us,
// 5.6 TB/s, 0.83 of the copy rate; in 16 bits 30 us, 0.77.  By instructions, half of them the masks', where 16-bit logits under a
// grammar are compared: 48 x 11 positions of 151936 in bf16 (171 MB) in 55 us, 3.1 TB/s, where 32 x 8 in fp32 without one take
// 34 us, 4.5 TB/s.  By its start (the look-ups, the history) where a CTA has one position, 96 x 1 of 32000 in 14 us, and behind
// a long history, which every CTA of the stream reads: 1 x 8 of 151936 behind 4000, 32768 and 131072 tokens in 10, 33 and 78 us,
// 32 x 8 in 60, 99 and 189.  128 and 512 threads took 66 and 62 us for those trees where 256 took 58.  Rows prefetched to L2 during the
// start: edits 58 -> 56, acceptance 58 -> 61 (left out there).
template <int kType, bool kShift, bool kAccept>
__global__ void __launch_bounds__(kEditThreads, kAccept ? 4 : 3) edit_kernel(EditView e) {
    using B = Bits<kType>;
    using X = Batch<kType, kShift>;
    constexpr int kWarps = kEditThreads / 32;
    constexpr uint32_t kListSeen = 1u << 15, kListInBlock = 1u << 14, kNoToken = 0xFFFFFFFFu;
    extern __shared__ uint4 dynamic[];
    __shared__ int block_token[64], block_at[64], n_block;       // tokens of the block that only some of the CTA's positions see
    __shared__ int listed[kParts];                               // tokens on the list, by parts of the run
    __shared__ uint32_t known[kEditRun / 32];                    // a bit for each of them,
    __shared__ uint32_t known_lane[kEditRun / X::kTokens][32];   // and as the lanes have them
    __shared__ unsigned long long part_best[kMostRows * kParts]; // acceptance: (key, ~token)
    const moe_mxfp4_edit_args& a = e.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sgs = a.streams * e.groups, run = blockIdx.x / sgs, sg = blockIdx.x - run * sgs, s = sg / e.groups, b0 = (sg - s * e.groups) * e.rows;
    const int64_t v0 = (int64_t)run * kEditRun, row0 = (int64_t)s * a.block;
    const int n = (int)min((int64_t)kEditRun, a.vocab - v0);
    uint32_t* const count = reinterpret_cast<uint32_t*>(dynamic);              // later, as fp32: what is taken off the token
    uint16_t* const list = reinterpret_cast<uint16_t*>(count + kEditRun);
    int* const entry = a.bias_begin_dev ? reinterpret_cast<int*>(list + kEditRun) : nullptr;
    float* const bias = reinterpret_cast<float*>(entry);         // 1 + the last entry of a token, then its bias
    grid_dependency_wait();
    const int b1 = min(min(b0 + e.rows, a.block), used_positions(a, s));
    if (b0 >= b1) return;
    // the rows are on their way to L2 meanwhile
    if (!kShift && !kAccept && tid < b1 - b0 && n * B::kSize >= 16)
        prefetch_run(static_cast<const char*>(a.logits_dev) + ((row0 + b0 + tid) * a.row_stride + v0) * B::kSize, (uint32_t)(n * B::kSize) & ~15u);
    // what the stream's part of the arguments says, all of it asked for at once
    const int parts = e.parts, span = kEditRun / parts, log_span = 31 - __clz(span);
    const int* const history = a.history_dev ? a.history_dev + s * a.history_stride : nullptr;
    const int len = history ? (int)min((int64_t)a.history_lengths_dev[s], a.history_room) : 0;
    const int prompt = history && a.prompt_lengths_dev ? a.prompt_lengths_dev[s] : 0;
    const int64_t bias_end = entry ? min((int64_t)a.bias_begin_dev[s + 1], a.bias_entries) : 0;
    const int64_t bias_begin = entry ? (int64_t)max(a.bias_begin_dev[s], 0) + tid : 0;
    const Penalty p{a.repetition_dev ? a.repetition_dev[s] : 1.0f, a.frequency_dev ? a.frequency_dev[s] : 0.0f,
                    a.presence_dev ? a.presence_dev[s] : 0.0f};
    const int token = a.tokens_dev && tid < b1 ? a.tokens_dev[row0 + tid] : -1;
    for (int i = tid; i < kEditRun / 4; i += kEditThreads) {
        reinterpret_cast<uint4*>(count)[i] = make_uint4(0, 0, 0, 0);
        if (entry) reinterpret_cast<uint4*>(entry)[i] = make_uint4(0, 0, 0, 0);
    }
    if (tid < kEditRun / 32) known[tid] = 0;
    for (int i = tid; i < kEditRun / X::kTokens * 32; i += kEditThreads) known_lane[0][i] = 0;
    if (tid < kParts) listed[tid] = 0;
    if (tid == 0) n_block = 0;
    __syncthreads();
    auto mark = [&](uint32_t v) {                  // puts a token on the list of its part, once
        const uint32_t bit = 1u << (v & 31);
        if (atomicOr(known + (v >> 5), bit) & bit) return;
        const int part = v >> log_span, in = v % X::kTokens, word = in / X::kPer;
        list[(part << log_span) + atomicAdd(listed + part, 1)] = (uint16_t)v;
        atomicOr(&known_lane[v / X::kTokens][word % 32], 1u << (word / 32 * X::kPer + in % X::kPer));
    };
    for_history(history, 0, len, prompt, [&](int t, bool prompted) {
        const uint32_t v = (uint32_t)t - (uint32_t)v0;
        if (v >= (uint32_t)n) return;
        const uint32_t was = prompted ? atomicOr(count + v, kPrompted) : atomicAdd(count + v, 1u);
        if (!was) mark(v);
    });
    if (a.tokens_dev)
        for (int j = tid; j < b1; j += kEditThreads) {
            const uint32_t v = (uint32_t)(j == tid ? token : a.tokens_dev[row0 + j]) - (uint32_t)v0;
            if (v >= (uint32_t)n) continue;
            if (!a.mask_dev && j <= b0) {
                atomicAdd(count + v, 1u);          // all positions here see it
            } else {
                atomicOr(count + v, kInBlock);
                const int k = atomicAdd(&n_block, 1);
                block_token[k] = (int)v;
                block_at[k] = j;
            }
            mark(v);
        }
    for (int64_t i = bias_begin; i < bias_end; i += kEditThreads) {
        const uint32_t v = (uint32_t)a.bias_ids_dev[i] - (uint32_t)v0;
        if (v < (uint32_t)n && !atomicMax(entry + v, (int)i + 1)) mark(v);
    }
    __syncthreads();
    for (int part = 0; part < parts; ++part)
        for (int k = tid; k < listed[part]; k += kEditThreads) {
            const int v = list[(part << log_span) + k];
            const uint32_t c = count[v];
            const float add = entry && entry[v] ? a.bias_dev[entry[v] - 1] : 0.0f;
            if (entry) bias[v] = add;
            list[(part << log_span) + k] = (uint16_t)(v | (c ? kListSeen : 0) | (c & kInBlock ? kListInBlock : 0));
            if (!(c & kInBlock)) reinterpret_cast<float*>(count)[v] = __fsub_rn(penalty_of(c & ~kPrompted, p), add);
        }
    __syncthreads();
    for (int item = warp; item < (b1 - b0) * parts; item += kWarps) {
        const int b = b0 + item / parts, part = item - (b - b0) * parts, first = part * span, last = min(first + span, n);
        const char* const row = static_cast<const char*>(a.logits_dev) + ((row0 + b) * a.row_stride + v0) * B::kSize;
        char* const out = static_cast<char*>(e.out) + ((row0 + b) * e.out_stride + v0) * B::kSize;
        const uint32_t* const allowed = a.allowed_dev ? a.allowed_dev + (row0 + b) * a.allowed_stride + (v0 >> 5) : nullptr;
        const uint16_t* const mine = list + first; // the first tokens on the list are asked for before the rest is looked at
        const int n_mine = listed[part];
        uint32_t token0 = lane < n_mine ? mine[lane] : kNoToken, x0 = 0;
        if (token0 != kNoToken) x0 = B::read(row, token0 & (kEditRun - 1));
        float most = -INFINITY;                    // of the rest,
        int where = -1;                            // and the first token of its batch, or (~) itself
        uint32_t some = 0;                         // whether the lane has a token that is allowed
        // the words of 16 bytes of first .. last, and the few tokens before and behind them
        const int lead = kShift ? (int)(-(reinterpret_cast<uintptr_t>(row + first * B::kSize) / B::kSize) & (X::kPer - 1)) : 0;
        const int begin = min(first + lead, last), end = begin + (last - begin) / X::kPer * X::kPer;
        const bool whole = !kShift || ((reinterpret_cast<uintptr_t>(out) - reinterpret_cast<uintptr_t>(row)) & 15) == 0;   // words of the output too
        auto single = [&](int v) {
            const uint32_t x = B::read(row, v);
            const bool ok = !allowed || bit_at(allowed, v);
            if (kAccept) {
                some |= ok;
                if (ok && !bit_at(known, v) && B::value(x) > most) {
                    most = B::value(x);
                    where = ~v;
                }
            } else if (!ok || e.out != a.logits_dev) {
                B::write(out, v, ok ? x : B::kNone);
            }
        };
        if (kShift && first + lane < begin) single(first + lane);
        if (begin < end) {
            X next;
            next.load(row, allowed, begin, end, lane);
            for (int base = begin; base < end; base += X::kTokens) {
                X x = next;
                if (base + X::kTokens < end) next.load(row, allowed, base + X::kTokens, end, lane);
                if (kAccept) {
                    some |= x.ok;
                    const float m = x.most(x.ok & ~X::known_bits(known, known_lane, base, end, lane));
                    if (m > most) {
                        most = m;
                        where = base;
                    }
                } else {
                    const bool all = x.ok == X::kAll;
                    if (!all) x.hide();
                    if (all && e.out == a.logits_dev) continue;
                    char* const to = out + (base + X::token(0, lane)) * B::kSize;
                    const bool full = base + X::kTokens <= end;
                    if (whole) {
#pragma unroll
                        for (int w = 0; w < 4; ++w)
                            if (full || base + X::token(w, lane) + X::kPer <= end) reinterpret_cast<uint4*>(to)[32 * w] = x.x[w];
                    } else {
#pragma unroll
                        for (int w = 0; w < 4; ++w)
#pragma unroll
                            for (int i = 0; i < X::kPer; ++i)
                                if (full || base + X::token(w, lane) + X::kPer <= end) B::write(to + 512 * w, i, x.get(w, i));
                    }
                }
            }
        }
        if (end + lane < last) single(end + lane);
        // the tokens on the list
        if (!kAccept) __syncwarp();
        float best = -INFINITY;
        int which = kEditRun;
        auto edit = [&](uint32_t token, uint32_t x) {
            const int v = token & (kEditRun - 1);
            if (allowed && !bit_at(allowed, v)) return;
            float off = reinterpret_cast<const float*>(count)[v];
            bool seen = token & kListSeen;
            if (token & kListInBlock) {
                uint32_t c = count[v] & ~kInBlock;
                const bool tree = a.mask_dev != nullptr;
                const unsigned long long sees = tree ? (a.mask_dev[row0 + b] & ((1ull << b) - 1)) | 1ull << b : 0;
                for (int j = 0; j < n_block; ++j)
                    if (block_token[j] == v && (tree ? sees >> block_at[j] & 1 : block_at[j] <= b)) ++c;
                seen = c != 0;
                off = __fsub_rn(penalty_of(c & ~kPrompted, p), entry ? bias[v] : 0.0f);
            }
            const float z = edited(B::value(x), seen, off, p);
            if (!kAccept) {
                B::write(out, v, B::of(z));
            } else if (z > best || (z == best && v < which)) {
                best = z;
                which = v;
            }
        };
        if (token0 != kNoToken) edit(token0, x0);
        for (int k0 = 32; k0 < n_mine; k0 += 128) {
            uint32_t tokens[4], x[4];              // (four at once: each comes from memory)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = k0 + 32 * i + lane;
                tokens[i] = k < n_mine ? mine[k] : kNoToken;
                x[i] = tokens[i] != kNoToken ? B::read(row, tokens[i] & (kEditRun - 1)) : 0;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (tokens[i] != kNoToken) edit(tokens[i], x[i]);
        }
        if (!kAccept) continue;
        const float all = fmaxf(most, best);
        const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, some || which < kEditRun ? logit_key(all) : 0);
        uint32_t v = 0xFFFFFFFFu;
        if (top == logit_key(-INFINITY)) {         // no numbers: the first that is allowed
            for (int i = (first >> 5) + lane; 32 * i < last; i += 32) {
                uint32_t word = allowed ? allowed[i] : 0xFFFFFFFFu;
                if (32 * i + 32 > n) word &= (1u << (n - 32 * i)) - 1;
                if (word && v == 0xFFFFFFFFu) v = 32 * i + __ffs(word) - 1;
            }
        } else if (top && logit_key(all) == top) { // the first of the largest (a lane without any has -inf here)
            if (best == all) v = which;
            if (most == all) {
                int at = ~where;
                if (where >= 0) {                  // its words once more
                    X x;
                    x.load(row, allowed, where, end, lane);
                    at = where + x.find(x.ok & ~X::known_bits(known, known_lane, where, end, lane), all, lane);
                }
                v = min(v, (uint32_t)at);
            }
        }
        v = __reduce_min_sync(0xFFFFFFFFu, v);
        if (lane == 0) part_best[item] = top ? (unsigned long long)top << 32 | (0xFFFFFFFFu - (uint32_t)(v0 + v)) : 0;
    }
    if (!kAccept) return;
    grid_dependency_launch();
    __syncthreads();
    if (tid < b1 - b0) {
        unsigned long long best = 0;
        for (int k = 0; k < parts; ++k) best = part_best[tid * parts + k] > best ? part_best[tid * parts + k] : best;
        e.best[(row0 + b0 + tid) * e.runs + run] = best;
    }
}

// A CTA per stream: the targets of its positions, and the path of accepted nodes; some 3 us of the launch and its look-ups.  It starts while the edits end (each of
// their CTAs has waited for what came before), and reads what they do not write before it waits for them.
__global__ void __launch_bounds__(256) accept_path_kernel(EditView e, int* __restrict__ target, int* __restrict__ accepted,
                                                          int* __restrict__ next_token, int* __restrict__ path) {
    __shared__ int s_target[1024], s_token[1024], s_parent[1024];
    const moe_mxfp4_edit_args& a = e.a;
    const int s = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    const int used = a.lengths_dev ? min(__ldcg(a.lengths_dev + s), a.block) : a.block;
    const int64_t row0 = (int64_t)s * a.block;
    for (int b = tid; b < a.block; b += 256) {
        s_token[b] = __ldcg(a.tokens_dev + row0 + b);
        s_parent[b] = a.mask_dev ? 63 - __clzll(__ldcg(reinterpret_cast<const unsigned long long*>(a.mask_dev) + row0 + b) & ((1ull << b) - 1)) : b - 1;
    }
    grid_dependency_wait();
    for (int b = tid >> 5; b < a.block; b += 8) {
        unsigned long long best = 0;
        if (b < used)
            for (int i = lane; i < e.runs; i += 32) {
                const unsigned long long x = __ldcg(e.best + (row0 + b) * e.runs + i);
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
    if (a->bias_begin_dev && (a->bias_entries < 0 || a->bias_entries >= 0x7FFFFFFF)) return MOE_ERR_INVALID_ARG;
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
    const int known = moe::current_sm_count(), sms = known ? known : 1;
    e->runs = edit_runs(e->a.vocab);
    const int64_t ctas = (int64_t)e->a.streams * e->a.block * e->runs, most = ctas / (4 * sms);
    e->rows = (int)(most < 1 ? 1 : most > moe::kMostRows ? moe::kMostRows : most);
    if (e->rows > e->a.block) e->rows = e->a.block;
    e->groups = (e->a.block + e->rows - 1) / e->rows;
    // parts of a run: the fewest that keep five eighths of the warps of all its rounds busy, up to kParts.  (Six and seven
    // eighths make more parts, each with a start and a reduction of its own.  Acceptance of 16 x 5 positions of 151936 in bf16 17 us, 22 with
    // either; of 16 x 9 and 16 x 10 28 and 27, 28 and 30 with six eighths, 34 and 35 with seven.  Edits differ by 3 % either way.)
    constexpr int warps = moe::kEditThreads / 32;
    for (e->parts = 1; e->parts < moe::kParts; e->parts *= 2) {
        const int items = e->rows * e->parts, rounds = (items + warps - 1) / warps;
        if (8 * items >= 5 * warps * rounds) break;
    }
}

template <bool kAccept>
int launch_edit(const moe::EditView& e, cudaStream_t st) {
    const dim3 grid((unsigned)((int64_t)e.a.streams * e.groups * e.runs));
    const int size = e.a.dtype == MOE_DTYPE_FP32 ? 4 : 2;
    const bool shift = !aligned(e.a.logits_dev, 16) || e.a.row_stride * size % 16 ||
                       (!kAccept && (!aligned(e.out, 16) || e.out_stride * size % 16));
    const size_t shared = moe::kEditRun * (4 + 2 + (e.a.bias_begin_dev ? 4 : 0));   // the counts and the list, the biases if there are any
    auto go = [&](auto kern) { return moe::launch_dependent(kern, grid, dim3(moe::kEditThreads), shared, st, e); };
    cudaError_t r;
    if (e.a.dtype == MOE_DTYPE_FP32)
        r = shift ? go(moe::edit_kernel<MOE_DTYPE_FP32, true, kAccept>) : go(moe::edit_kernel<MOE_DTYPE_FP32, false, kAccept>);
    else if (e.a.dtype == MOE_DTYPE_BF16)
        r = shift ? go(moe::edit_kernel<MOE_DTYPE_BF16, true, kAccept>) : go(moe::edit_kernel<MOE_DTYPE_BF16, false, kAccept>);
    else
        r = shift ? go(moe::edit_kernel<MOE_DTYPE_FP16, true, kAccept>) : go(moe::edit_kernel<MOE_DTYPE_FP16, false, kAccept>);
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
