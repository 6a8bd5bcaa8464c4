// Norms of query and key heads with the position rotation, in one pass: on their own (moe_mxfp4_rotate), and
// on the way into the paged cache (moe_mxfp4_cache_append_rotated).
//
// Mathematics.  A head x at position p: x_e <- x_e w_e / sqrt(mean(x^2) + eps), then each pair (a, b) turns by
// p f_i.  The angle is kept as a fraction of a turn in 64 bits, T_i = 2^64 f_i / 2 pi: p T_i modulo 2^64 is
// exact, and its upper 32 bits, as half turns in [-1, 1), are what the sine and cosine are taken of.  In fp32
// radians an angle of 10^5 would be off by up to 0.004.
#include <cuda_fp16.h>

#include <cmath>

#include "cache.cuh"

namespace moe {

struct RotaryView {
    const unsigned long long* turns;
    const uint16_t *q_norm, *k_norm;
    int R, norm, interleaved;
    float eps, gain;
};

// What a call reads and writes: rows of heads, `in` and `out` elements between rows.
struct HeadRows {
    const uint16_t* src;
    uint16_t* dst;
    int64_t in, out;
    int heads;
};

// Where the keys and values of a token go.
struct PagePlace {
    CacheView c;
    uint16_t *kp, *vp;
    const int* lengths;
    const unsigned long long* mask;
    int block;
};

// gain * (cos, sin) of position p's angle in pair i.
__device__ __forceinline__ float2 turn_of(unsigned long long turns, int p, float gain) {
    const unsigned long long phase = (unsigned long long)(long long)p * turns;
    float s, c;
    sincospif((float)(int)(phase >> 32) * 0x1p-31f, &s, &c);
    return make_float2(gain * c, gain * s);
}

// A token of a block on its way into the cache.  Its page and the page's count are asked for early and looked at
// late, when a key or a value is to be stored: the queries do not wait for them.
struct TokenPlace {
    int s, i, len;
    int position;          // of the rotation
    bool used;             // in use
    int page, holders;     // -1: not reserved
};
__device__ __forceinline__ TokenPlace token_place(const PagePlace& p, int tok) {
    TokenPlace t;
    t.s = tok / p.block;
    t.i = tok - t.s * p.block;
    t.len = p.c.length()[t.s];
    const int held = p.c.held()[t.s];
    const unsigned long long sees = p.mask ? p.mask[tok] : 0;
    t.used = !p.lengths || t.i < p.lengths[t.s];
    t.position = t.len + (p.mask ? __popcll(sees & ((1ull << t.i) - 1)) : t.i);
    const int64_t at = ((int64_t)t.len + t.i) >> p.c.page_shift;
    t.page = t.used && t.len >= 0 && at < min(held, p.c.L.M) ? p.c.table(t.s)[at] : -1;
    return t;
}
__device__ __forceinline__ void token_holders(const PagePlace& p, TokenPlace* t) {
    t->holders = (unsigned)t->page < (unsigned)p.c.L.P ? p.c.refcount()[t->page] : 2;
}
// The token's place in a pool (element of head 0), -1: its position is not reserved, or in a page that others hold too.
__device__ __forceinline__ int64_t token_at(const PagePlace& p, const TokenPlace& t) {
    if (t.holders > 1) {
        raise_status(p.c.state + kCacheStatus, MOE_ERR_CACHE_STATE, t.s);
        return -1;
    }
    return t.page * p.c.page_stride + ((t.len + t.i) & (p.c.page - 1)) * p.c.D;
}

// Two 16-bit values of a word as fp32, and back.
template <bool kBf16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
    if (kBf16) return make_float2(bf16_lo(v), bf16_hi(v));
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
template <bool kBf16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t v;
    if (kBf16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(hi), "f"(lo));
    return v;
}

__device__ __forceinline__ void copy_16(void* smem, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// How a head's pairs lie in its 16-byte words.
enum : int {
    kHalves,   // i and rotary_dim / 2 + i, rotary_dim a multiple of 16: word against word
    kPairs,    // side by side: within a word
    kAnywhere, // i and rotary_dim / 2 + i, any other rotary_dim
};

// A lane has 16 elements of a head in two words, D / 16 lanes a head, so a warp has 4 heads of 128 or 8 of 64 at a time.  The
// words are chosen so that they hold both sides of the lane's 8 pairs, with neighbours' words side by side in memory (with both words
// of a lane side by side each load touched half of every 32-byte sector: narrow heads took 92 us where this took 77, both before
// the steps that followed).  The lanes that share a token's 8 pairs each take the sine and cosine of some of them, two (heads of 64:
// one) where the warp has one token and up to eight (four) where it has kPack of them, and the others from their neighbours; they stay in
// registers for the token's heads.  kAnywhere: a warp takes a token's sines and cosines through shared memory, and the lanes
// exchange the normed elements there, laid out so that neither side has conflicts.  A warp takes `steps` rounds of a token's heads.
// Every lane copies its own words three rounds ahead (kAnywhere: two) into its own places of shared memory, across tokens, so
// memory is kept busy without registers and without barriers.
// Bound by HBM: 16381 tokens of 56 + 8 heads of 128 (537 MB read and written) in 86 us, 6.2 TB/s, 0.92 of the copy rate;
// 47976 tokens of 32 + 4 heads of 64 in 67 us, 0.97; 2 layers of those into the cache with their values in 156 us, 0.93.  Of few
// tokens by the launch and the chain of look-ups: 8 tokens of one layer in 2.5 us, 3.1 into the cache.
// Few heads: a round has the heads of kPack tokens, and a token's sines and cosines are shared by its lanes alone (two heads of
// 128, 300000 tokens: 96 us, 154 with a token a round; 46 are the bytes').
template <int D, bool kBf16, int kLayout, bool kCache, int kPack>
__global__ void __launch_bounds__(256, kLayout == kAnywhere ? 2 : 3) rotate_kernel(RotaryView r, HeadRows q, HeadRows k, const uint16_t* v,
                                                                                  const int* __restrict__ positions, int tokens, int parts,
                                                                                  int steps, PagePlace pages) {
    constexpr int kLanes = D / 16, kHeads = 32 / kLanes, kStages = kLayout == kAnywhere ? 3 : 4;
    constexpr int kColumn = D / 8, kHeadRow = D + kLanes;        // kAnywhere: element e of a head at place (e % 8) kColumn + e / 8
    constexpr int kTurns = kLayout == kAnywhere ? 16 : 8;
    __shared__ uint4 ring[8][kStages][2][32];
    __shared__ float normed[kLayout == kAnywhere ? 8 : 1][kHeads * kHeadRow];
    __shared__ float2 turned[kLayout == kAnywhere ? 8 : 1][D / 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = lane % kLanes, g = lane / kLanes;
    const int heads = q.heads + k.heads * (kCache ? 2 : 1), half = r.R / 2;
    // the lane's words: elements o0.. and o1..
    const bool across = kLayout == kHalves && 16 * j < r.R;
    const int o0 = kLayout != kHalves || across ? 8 * j : half + 8 * j, o1 = across ? half + 8 * j : D / 2 + 8 * j;
    // a token's lanes, and how many of them take the sines and cosines of eight pairs: pair i of the lane's eight is
    // taken by the (i % kSharers)-th of the lanes that share them, as its (i / kSharers)-th
    constexpr int kTokenLanes = 32 / kPack, kSharers = kTokenLanes / kLanes, kTaken = 8 / kSharers;
    const int member = lane / kTokenLanes;         // of the unit's tokens
    auto pair_of = [&](int j, int i) { return kLayout == kPairs ? 4 * j + (i < 4 ? i : D / 4 + i - 4) : 8 * j + i; };
    // which of its pairs (kAnywhere: elements) turn
    uint32_t turns = across ? 0xFF : 0;
    if (kLayout != kHalves) {
        turns = 0;
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const int e = kLayout == kPairs ? (i < 4 ? o0 + 2 * i : o1 + 2 * (i - 4)) : (i < 8 ? o0 + i : o1 + i - 8);
            turns |= (uint32_t)(e < r.R) << i;
        }
    }
    const int64_t units = kPack > 1 ? ((int64_t)tokens + kPack - 1) / kPack : (int64_t)tokens * parts, stride = (int64_t)gridDim.x * 8;
    const int64_t u0 = (int64_t)blockIdx.x * 8 + warp;
    // unit u: the lane's token, and the first of its heads that the warp takes (a 64-bit division costs as much as half a round)
    auto unit = [&](int64_t u, int* tok, int* head) {
        *tok = kPack > 1 ? (int)u * kPack + member : parts == 1 ? (int)u : (int)(u / parts);
        *head = kPack > 1 ? -member * (kHeads / kPack) : parts == 1 ? 0 : (int)(u - (int64_t)*tok * parts) * steps * kHeads;
    };
    int64_t ahead_u = u0;
    int ahead_step = 0, ahead_slot = 0, slot = 0, ahead_tok, ahead_head;
    unit(u0, &ahead_tok, &ahead_head);
    auto ahead = [&] {
        if (ahead_u < units) {
            const int h = ahead_head + ahead_step * kHeads + g;
            if (h < heads && (kPack == 1 || ahead_tok < tokens)) {
                const uint16_t* src;
                if (h < q.heads) {
                    src = q.src + ahead_tok * q.in + (int64_t)h * D;
                } else {
                    const bool is_v = h >= q.heads + k.heads;
                    src = (is_v ? v : k.src) + ahead_tok * k.in + (int64_t)(h - q.heads - (is_v ? k.heads : 0)) * D;
                }
                copy_16(&ring[warp][ahead_slot][0][lane], src + o0);
                copy_16(&ring[warp][ahead_slot][1][lane], src + o1);
            }
            if (++ahead_step == steps) {
                ahead_step = 0;
                ahead_u += stride;
                unit(ahead_u, &ahead_tok, &ahead_head);
            }
        }
        copies_commit();
        if (++ahead_slot == kStages) ahead_slot = 0;
    };
    grid_dependency_wait();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) ahead();
    for (int64_t u = u0; u < units; u += stride) {
        int tok, h0;
        unit(u, &tok, &h0);
        TokenPlace place{};
        const bool real = kPack == 1 || tok < tokens;            // (the last unit may have fewer tokens)
        if (kCache && real) place = token_place(pages, tok);
        const int p = kCache ? place.position : real ? positions[tok] : 0;
        float c[kTurns], s[kTurns];
        if (kLayout == kAnywhere) {
            __syncwarp();
            for (int i = lane; i < half; i += 32) turned[warp][i] = turn_of(r.turns[i], p, r.gain);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kTurns; ++i) {     // element e against e + half (the sine's sign with it) or e - half
                const int e = i < 8 ? o0 + i : o1 + i - 8;
                const float2 t = e < r.R ? turned[warp][e < half ? e : e - half] : make_float2(0, 0);
                c[i] = t.x;
                s[i] = e < half ? -t.y : t.y;
            }
        } else if (r.R) {
            float2 t[kTaken];
            const int in = lane % kTokenLanes;
#pragma unroll
            for (int i = 0; i < kTaken; ++i) {
                const int pair = pair_of(in / kSharers, i * kSharers + in % kSharers);
                t[i] = pair < half ? turn_of(r.turns[pair], p, r.gain) : make_float2(0, 0);
            }
#pragma unroll
            for (int i = 0; i < kTurns; ++i) {
                const int from = member * kTokenLanes + (kSharers * j + i % kSharers) % kTokenLanes;
                c[i] = __shfl_sync(0xFFFFFFFFu, t[i / kSharers % kTaken].x, from);
                s[i] = __shfl_sync(0xFFFFFFFFu, t[i / kSharers % kTaken].y, from);
            }
        }
        if (kCache && real) token_holders(pages, &place);
        for (int step = 0; step < steps; ++step) {
            ahead();
            copies_wait<kStages - 1>();
            uint4 w0 = ring[warp][slot][0][lane], w1 = ring[warp][slot][1][lane];
            if (++slot == kStages) slot = 0;
            const int h = h0 + step * kHeads + g;
            const bool is_q = h < q.heads, is_v = h >= q.heads + k.heads;
            float x[16];
            {
                const uint32_t in[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 f = unpack2<kBf16>(in[i]);
                    x[2 * i] = f.x;
                    x[2 * i + 1] = f.y;
                }
            }
            if (r.norm) {
                float sum = 0;
#pragma unroll
                for (int i = 0; i < 16; ++i) sum = fmaf(x[i], x[i], sum);
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                const float scale = rsqrtf(sum * (1.0f / D) + r.eps);
                const uint16_t* w = is_q ? r.q_norm : r.k_norm;
                if (w) {
                    const uint4 a = *reinterpret_cast<const uint4*>(w + o0), b = *reinterpret_cast<const uint4*>(w + o1);
                    const uint32_t in[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 f = unpack2<kBf16>(in[i]);
                        x[2 * i] *= scale * f.x;
                        x[2 * i + 1] *= scale * f.y;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] *= scale;
                }
            }
            if (kLayout == kAnywhere) {
                float* const head = normed[warp] + g * kHeadRow;
#pragma unroll
                for (int i = 0; i < 16; ++i) head[i % 8 * kColumn + (i < 8 ? o0 : o1) / 8] = x[i];
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int e = i < 8 ? o0 + i : o1 + i - 8, with = e < half ? e + half : e - half;
                    if (turns >> i & 1) x[i] = fmaf(head[with % 8 * kColumn + with / 8], s[i], x[i] * c[i]);
                }
                __syncwarp();
            }
            if (h >= heads || !real || (kCache && !place.used)) continue;
            if (!is_v) {
                if (kLayout != kAnywhere)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (kLayout == kHalves ? across : turns >> i & 1) {
                            float &a = x[kLayout == kPairs ? 2 * i : i], &b = x[kLayout == kPairs ? 2 * i + 1 : i + 8];
                            const float y = a * c[i] - b * s[i];
                            b = fmaf(a, s[i], b * c[i]);
                            a = y;
                        }
                w0 = make_uint4(pack2<kBf16>(x[0], x[1]), pack2<kBf16>(x[2], x[3]), pack2<kBf16>(x[4], x[5]), pack2<kBf16>(x[6], x[7]));
                w1 = make_uint4(pack2<kBf16>(x[8], x[9]), pack2<kBf16>(x[10], x[11]), pack2<kBf16>(x[12], x[13]), pack2<kBf16>(x[14], x[15]));
            }
            uint16_t* dst;
            if (is_q) {
                dst = q.dst + tok * q.out + (int64_t)h * D;
            } else {
                const int i = h - q.heads - (is_v ? k.heads : 0);
                dst = k.dst + tok * k.out + (int64_t)i * D;
                if (kCache) {
                    const int64_t at = token_at(pages, place);
                    if (at < 0) continue;
                    dst = (is_v ? pages.vp : pages.kp) + at + (int64_t)i * pages.c.page * D;
                }
            }
            *reinterpret_cast<uint4*>(dst + o0) = w0;
            *reinterpret_cast<uint4*>(dst + o1) = w1;
        }
    }
}

}  // namespace moe

namespace {

template <class T>
bool aligned(const void* p, T n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool good_rotary(const moe_mxfp4_rotary* r) {
    if (!r || (r->head_dim != 64 && r->head_dim != 128)) return false;
    if (r->rotary_dim < 0 || r->rotary_dim > r->head_dim || r->rotary_dim % 2) return false;
    if (r->dtype != MOE_DTYPE_BF16 && r->dtype != MOE_DTYPE_FP16) return false;
    if (r->flags & ~(MOE_ROTARY_INTERLEAVED | MOE_ROTARY_NORM)) return false;
    if (!(r->eps >= 0.0f) || !std::isfinite(r->eps) || !std::isfinite(r->gain)) return false;
    if (r->rotary_dim && !r->turns_dev) return false;
    return aligned(r->turns_dev, 8) && aligned(r->q_norm_dev, 16) && aligned(r->k_norm_dev, 16);
}

moe::RotaryView rotary_view(const moe_mxfp4_rotary* r) {
    moe::RotaryView v;
    v.turns = reinterpret_cast<const unsigned long long*>(r->turns_dev);
    v.q_norm = static_cast<const uint16_t*>(r->q_norm_dev);
    v.k_norm = static_cast<const uint16_t*>(r->k_norm_dev);
    v.R = r->rotary_dim;
    v.norm = (r->flags & MOE_ROTARY_NORM) != 0;
    v.interleaved = (r->flags & MOE_ROTARY_INTERLEAVED) != 0;
    v.eps = r->eps;
    v.gain = r->gain;
    return v;
}

// Resolves a stride of rows; false for one that is too short or not a multiple of 16 bytes.
bool good_stride(int64_t* stride, int64_t row) {
    if (*stride == 0) *stride = row;
    return *stride >= row && *stride % 8 == 0;
}

template <bool kCache, int D, bool kBf16>
cudaError_t launch_rotate(const moe::RotaryView& r, const moe::HeadRows& q, const moe::HeadRows& k, const uint16_t* v,
                          const int* positions, int tokens, const moe::PagePlace& pages, int sms, cudaStream_t st) {
    const int heads = q.heads + k.heads * (kCache ? 2 : 1), layout = r.interleaved ? moe::kPairs : r.R % 16 ? moe::kAnywhere : moe::kHalves;
    // Rounds of heads of a token, dealt out to warps in parts of `steps` each, by two or three CTAs on every SM: what gives
    // the busiest warps the least to do, a part's start (its page, its sines and cosines) taken for a round's work.  Where
    // both do as well two do better, whose loads and stores come in longer runs of memory (47976 tokens of 36 narrow heads: 67 us
    // with two, 76 with three); three serve where two leave warps idle (2560 tokens of 48 heads: 127 us for 8 layers, 140 with
    // two), and where a token has a round or two, and warps wait for its look-ups (two heads: 154 us, 195 with two).
    // Where two CTAs an SM have a warp for every round, that is the least, and is taken without a search: which finds the same up
    // to 64 rounds a token, and goes no further (8 tokens of 640 heads: 2.8 us, 3.6 in 64 parts; of 2100 heads of one token: 2.6
    // and 6.5).  Beyond, parts win over rounds of their own (200, 304 and 600 tokens of 64 heads: 3.6, 3.7 and 5.0 us, 4.0,
    // 4.5 and 7.3 with a round each).
    const int rounds = (heads * (D / 16) + 31) / 32;
    int parts = rounds, steps = 1, resident = 2;
    if (rounds <= 2 || (int64_t)tokens * rounds > 2 * 8 * (int64_t)sms) {
        int64_t least = INT64_MAX;
        for (int ctas = rounds <= 2 && layout != moe::kAnywhere ? 3 : 2; ctas <= (layout == moe::kAnywhere ? 2 : 3); ++ctas)
            for (int n = 1; n <= rounds && n <= 64; ++n) {
                const int each = (rounds + n - 1) / n, made = (rounds + each - 1) / each;
                const int64_t warps = 8 * (int64_t)ctas * sms, cost = ((int64_t)tokens * made + warps - 1) / warps * (each + 1) * ctas;
                if (cost < least) {
                    least = cost;
                    parts = made;
                    steps = each;
                    resident = ctas;
                }
            }
    }
    // few heads: as many tokens a round as it has room for, up to four
    const int pack = layout == moe::kAnywhere || heads * (D / 16) > 16 ? 1 : heads * (D / 16) > 8 ? 2 : 4;
    if (pack > 1) resident = 3;
    const int64_t want = (pack > 1 ? ((int64_t)tokens + pack - 1) / pack + 7 : (int64_t)tokens * parts + 7) / 8;
    auto kern = moe::rotate_kernel<D, kBf16, moe::kAnywhere, kCache, 1>;
    if (layout == moe::kHalves)
        kern = pack == 4 ? moe::rotate_kernel<D, kBf16, moe::kHalves, kCache, 4> : pack == 2 ? moe::rotate_kernel<D, kBf16, moe::kHalves, kCache, 2>
                                                                                            : moe::rotate_kernel<D, kBf16, moe::kHalves, kCache, 1>;
    if (layout == moe::kPairs)
        kern = pack == 4 ? moe::rotate_kernel<D, kBf16, moe::kPairs, kCache, 4> : pack == 2 ? moe::rotate_kernel<D, kBf16, moe::kPairs, kCache, 2>
                                                                                           : moe::rotate_kernel<D, kBf16, moe::kPairs, kCache, 1>;
    return moe::launch_dependent(kern, dim3((unsigned)(want < (int64_t)resident * sms ? want : (int64_t)resident * sms)), dim3(256), 0, st, r, q, k, v, positions, tokens,
                                 parts, steps, pages);
}

template <bool kCache>
int launch_rotate(const moe_mxfp4_rotary* r, const moe::HeadRows& q, const moe::HeadRows& k, const uint16_t* v,
                  const int* positions, int tokens, const moe::PagePlace& pages, int sms, cudaStream_t st) {
    const moe::RotaryView view = rotary_view(r);
    const bool bf16 = r->dtype == MOE_DTYPE_BF16;
    auto go = [&](auto launch) { return launch(view, q, k, v, positions, tokens, pages, sms, st); };
    const cudaError_t e = r->head_dim == 64 ? (bf16 ? go(launch_rotate<kCache, 64, true>) : go(launch_rotate<kCache, 64, false>))
                                            : (bf16 ? go(launch_rotate<kCache, 128, true>) : go(launch_rotate<kCache, 128, false>));
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// 2^64 f / 2 pi, |f| <= 2 pi, modulo 2^64: the product with 1 / 2 pi in two doubles.
bool turns_of(double f, uint64_t* turns) {
    if (!(std::fabs(f) <= 6.283185307179587)) return false;
    const double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;   // 1 / 2 pi
    const double x = std::fabs(f), t = x * hi, rest = std::fma(x, hi, -t) + x * lo;
    const double a = std::ldexp(t, 64), whole = std::floor(a);
    const uint64_t n = whole >= 0x1p64 ? 0 : (uint64_t)whole;
    const uint64_t v = n + (uint64_t)(int64_t)std::llround((a - whole) + std::ldexp(rest, 64));
    *turns = f < 0 ? 0 - v : v;
    return true;
}

}  // namespace

extern "C" {

int moe_mxfp4_rotary_from(const double* frequencies, int32_t n, uint64_t* turns) {
    if (n < 0 || (n && (!frequencies || !turns))) return MOE_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i)
        if (!turns_of(frequencies[i], turns + i)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

int moe_mxfp4_rotary_turns(int32_t rotary_dim, double base, const moe_mxfp4_rotary_scaling* scaling, uint64_t* turns) {
    if (rotary_dim < 0 || rotary_dim % 2 || !(base > 0) || !std::isfinite(base) || (rotary_dim && !turns)) return MOE_ERR_INVALID_ARG;
    const int kind = scaling ? scaling->kind : MOE_ROTARY_NONE;
    if (kind < MOE_ROTARY_NONE || kind > MOE_ROTARY_PARTS) return MOE_ERR_INVALID_ARG;
    const double factor = kind == MOE_ROTARY_NONE ? 1 : scaling->factor;
    if (!(factor > 0) || !std::isfinite(factor)) return MOE_ERR_INVALID_ARG;
    if (kind == MOE_ROTARY_PARTS && (!(scaling->original > 0) || !std::isfinite(scaling->original) || !std::isfinite(scaling->low) ||
                                     !std::isfinite(scaling->high) || scaling->high <= scaling->low))
        return MOE_ERR_INVALID_ARG;
    if (kind == MOE_ROTARY_NTK && rotary_dim > 2) base *= std::pow(factor, (double)rotary_dim / (rotary_dim - 2));
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rotary_dim);
        if (kind == MOE_ROTARY_LINEAR) f /= factor;
        if (kind == MOE_ROTARY_PARTS) {
            const double turned = scaling->original * f / 6.283185307179586;
            const double g = std::fmin(std::fmax((turned - scaling->low) / (scaling->high - scaling->low), 0.0), 1.0);
            f = g * f + (1 - g) * f / factor;
        }
        if (!turns_of(f, turns + i)) return MOE_ERR_INVALID_ARG;
    }
    return MOE_OK;
}

int moe_mxfp4_rotate(const moe_mxfp4_rotary* r, const moe_mxfp4_rotate_args* args, void* stream) {
    if (!good_rotary(r) || !args) return MOE_ERR_INVALID_ARG;
    const moe_mxfp4_rotate_args& a = *args;
    if (a.tokens < 0 || a.q_heads < 0 || a.q_heads > 65536 || a.kv_heads < 0 || a.kv_heads > 65536) return MOE_ERR_INVALID_ARG;
    moe::HeadRows q{static_cast<const uint16_t*>(a.q_dev), static_cast<uint16_t*>(a.q_out_dev), a.q_stride, a.q_out_stride, a.q_heads};
    moe::HeadRows k{static_cast<const uint16_t*>(a.k_dev), static_cast<uint16_t*>(a.k_out_dev), a.k_stride, a.k_out_stride, a.kv_heads};
    for (moe::HeadRows* x : {&q, &k}) {
        const int64_t row = (int64_t)x->heads * r->head_dim;
        if (!good_stride(&x->in, row) || !good_stride(&x->out, row)) return MOE_ERR_INVALID_ARG;
        if (a.tokens && x->heads && (!x->src || !x->dst || !aligned(x->src, 16) || !aligned(x->dst, 16))) return MOE_ERR_INVALID_ARG;
    }
    if (a.tokens == 0 || a.q_heads + a.kv_heads == 0) return MOE_OK;
    if (!a.positions_dev || !aligned(a.positions_dev, 4)) return MOE_ERR_INVALID_ARG;
    const int sms = moe::current_sm_count();
    if (!sms) return MOE_ERR_CUDA;
    return launch_rotate<false>(r, q, k, nullptr, a.positions_dev, a.tokens, moe::PagePlace{}, sms, static_cast<cudaStream_t>(stream));
}

int moe_mxfp4_cache_append_rotated(moe_mxfp4_cache* c, void* state_dev, int32_t layer, const moe_mxfp4_rotary* r,
                                   const moe_mxfp4_append_args* args, void* stream) {
    if (!c || !state_dev || !aligned(state_dev, 16) || layer < 0 || layer >= c->cfg.num_layers) return MOE_ERR_INVALID_ARG;
    if (!good_rotary(r) || r->head_dim != c->cfg.head_dim || r->dtype != c->cfg.dtype || !args) return MOE_ERR_INVALID_ARG;
    const moe_mxfp4_append_args& a = *args;
    if (a.streams < 0 || a.streams > c->cfg.num_streams || a.block < 0 || (int64_t)a.streams * a.block > 0x7FFFFFFF) return MOE_ERR_INVALID_ARG;
    if (a.q_heads < 0 || a.q_heads > 65536 || !aligned(a.lengths_dev, 4) || !aligned(a.mask_dev, 8)) return MOE_ERR_INVALID_ARG;
    if (a.mask_dev && a.block > 64) return MOE_ERR_INVALID_ARG;
    const int64_t D = c->cfg.head_dim;
    moe::HeadRows q{static_cast<const uint16_t*>(a.q_dev), static_cast<uint16_t*>(a.q_out_dev), a.q_stride, a.q_heads * D, a.q_heads};
    moe::HeadRows k{static_cast<const uint16_t*>(a.k_dev), nullptr, a.row_stride, 0, c->cfg.kv_heads};
    if (!good_stride(&q.in, q.heads * D) || !good_stride(&k.in, k.heads * D)) return MOE_ERR_INVALID_ARG;
    if (a.streams == 0 || a.block == 0) return MOE_OK;
    if (!a.k_dev || !a.v_dev || !aligned(a.k_dev, 16) || !aligned(a.v_dev, 16)) return MOE_ERR_INVALID_ARG;
    if (a.q_heads && (!a.q_dev || !a.q_out_dev || !aligned(a.q_dev, 16) || !aligned(a.q_out_dev, 16))) return MOE_ERR_INVALID_ARG;
    const moe::DeviceScope on(c->device);
    if (!on.ok()) return MOE_ERR_CUDA;
    moe::PagePlace pages;
    pages.c = moe::cache_view(c, state_dev);
    pages.kp = static_cast<uint16_t*>(c->layers[layer].k_dev);
    pages.vp = static_cast<uint16_t*>(c->layers[layer].v_dev);
    pages.lengths = a.lengths_dev;
    pages.mask = reinterpret_cast<const unsigned long long*>(a.mask_dev);
    pages.block = a.block;
    return launch_rotate<true>(r, q, k, static_cast<const uint16_t*>(a.v_dev), nullptr, a.streams * a.block, pages, c->sm_count,
                               static_cast<cudaStream_t>(stream));
}

}  // extern "C"
