// moe.cuh -- the operators of a routed expert layer around the grouped GEMMs: routing, the expert
// order of the rows (plan), dispatch into quantised rows, combine back to tokens, and the SwiGLU
// between the experts' two GEMMs with its 8-bit checkpoint.  Everything here streams through HBM
// (routing and the plan excepted: their data is small and latency counts), so the design rule is
// one pass: quantised outputs leave from registers, gathers replace copies.
#pragma once

#include <float.h>
#include <math_constants.h>
#include <stdint.h>

#include <type_traits>

#include "ptx.cuh"
#include "quant.cuh"

namespace fp8q {

constexpr int kDevBadOffsets = 2;   // FP8Q_DEV_BAD_OFFSETS
constexpr int kDevBadIndex = 4;     // FP8Q_DEV_BAD_INDEX
constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxTopK = 32;
constexpr int kMoeMaxGroups = 32;
constexpr unsigned kFull = 0xFFFFFFFFu;

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

__device__ __forceinline__ uint32_t bf16_rn(float x)
{
    uint16_t r;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) { *p = (uint16_t)bf16_rn(v); }

// ------------------------------------------------------------------------------------------
// Arithmetic shared by the kernels below
// ------------------------------------------------------------------------------------------
// max(m, |a|, |b|), a NaN losing (max.f32 with three inputs).
__device__ __forceinline__ float max_abs(float m, float a, float b)
{
    float r;
    asm("{.reg .f32 a, b;\n\t"
        "abs.f32 a, %2;\n\t"
        "abs.f32 b, %3;\n\t"
        "max.f32 %0, %1, a, b;}"
        : "=f"(r)
        : "f"(m), "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float amax16f(const float (&f)[16])
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i += 2) m = max_abs(m, f[i], f[i + 1]);
    return m;
}
// Four codes of four values, the first in the low byte.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d)
{
    uint32_t r;
    asm("{.reg .b16 l, h;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d, float inv)
{
    return codes4(__fmul_rn(a, inv), __fmul_rn(b, inv), __fmul_rn(c, inv), __fmul_rn(d, inv));
}
__device__ __forceinline__ uint4 quant16f(const float (&f)[16], float inv)
{
    return make_uint4(e4m3x4(f[0], f[1], f[2], f[3], inv), e4m3x4(f[4], f[5], f[6], f[7], inv),
                      e4m3x4(f[8], f[9], f[10], f[11], inv), e4m3x4(f[12], f[13], f[14], f[15], inv));
}
// The largest of 8 neighbouring lanes (all 32 take part).
__device__ __forceinline__ float max8(float v)
{
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}

// Two FP32 products at once (mul.rn.f32x2: each rounded to nearest, as __fmul_rn).
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 r;
    asm("{.reg .b64 a, b, c;\n\t"
        "mov.b64 a, {%2, %3};\n\t"
        "mov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 c, a, b;\n\t"
        "mov.b64 {%0, %1}, c;}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 r;
    asm("{.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\t"
        "mov.b64 b, {%4, %5};\n\t"
        "mov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\t"
        "mov.b64 {%0, %1}, d;}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 r;
    asm("{.reg .b64 a, b, c;\n\t"
        "mov.b64 a, {%2, %3};\n\t"
        "mov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 c, a, b;\n\t"
        "mov.b64 {%0, %1}, c;}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
// Two bf16 values as FP32, by a mixed-precision x + (-0), which is x: it runs on the FMA pipe, whereas
// shifting and masking take the ALU, which the conversions to E4M3 and the maxima already fill.
__device__ __forceinline__ float2 widen(uint32_t w)
{
    float2 r;
    asm("{.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "add.f32.bf16 %0, l, %3;\n\t"
        "add.f32.bf16 %1, h, %3;}"
        : "=f"(r.x), "=f"(r.y)
        : "r"(w), "f"(-0.0f));
    return r;
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
template <typename T>
__device__ __forceinline__ T warp_sum(T v)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// ------------------------------------------------------------------------------------------
// Routing.  One warp per token; lane l holds the NV consecutive experts l NV ..  The order of the
// experts is that of key = score + bias in binary64 (without a bias that of the logits themselves,
// which is the same order and needs no arithmetic); equal keys go to the lower index.  A masked
// expert (logit or bias -inf, NaN or +inf) has the key -inf.
//
// Keys are first formed in binary32 and truncated, with an error that is bounded below.  Where two
// neighbours in the order found that way are nearer than the bound, the candidates are put in order by
// whole keys, in binary64 where there is a bias; where two groups at the border are, the token is done
// again with whole keys throughout.  Both are rare (binary64 for every token: 65 us instead of 16 below).
// Bound by instruction issue while the SMs are busy (0.71 of the slots; the ALU 0.63), and by the latency of one
// token's rounds at either end of the launch: 8192 tokens of 256 experts in 8 groups with a bias take 16 us,
// without groups and bias 8.2 us (their 8 MB of logits 1.3 us); one token 3.3 us.  Where all logits and biases are equal,
// as in a router at its start, 20 and 12.5 us (51 and 33 where equal inputs counted as doubt).
// ------------------------------------------------------------------------------------------
// Keys as unsigned integers of the same order, above 1.  0: not to be chosen (again); 1: masked.
__device__ __forceinline__ uint32_t rank_of(float f)
{
    const uint32_t u = __float_as_uint(f + 0.0f);   // -0 is 0
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ unsigned long long rank_of(double f)
{
    const unsigned long long u = (unsigned long long)__double_as_longlong(f + 0.0);
    return u ^ ((u >> 63) ? ~0ull : 0x8000000000000000ull);
}
__device__ __forceinline__ uint32_t warp_top(uint32_t v) { return __reduce_max_sync(kFull, v); }
__device__ __forceinline__ unsigned long long warp_top(unsigned long long v)
{
    const uint32_t hi = __reduce_max_sync(kFull, (uint32_t)(v >> 32));
    const uint32_t lo = __reduce_max_sync(kFull, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return ((unsigned long long)hi << 32) | lo;
}
template <typename F> struct Rank { typedef uint32_t type; };
template <> struct Rank<double> { typedef unsigned long long type; };
template <typename F> __device__ __forceinline__ F lowest() { return (F)-CUDART_INF_F; }

// (a, b) <- the two largest of a, b, c, d with a >= b, c >= d.
template <typename F>
__device__ __forceinline__ void merge_two(F& a, F& b, F c, F d)
{
    b = a > c ? (b > c ? b : c) : (a > d ? a : d);
    a = a > c ? a : c;
}

struct RouteShape {
    int E, k, n_group, topk_group;
    int per;     // experts of a group
    int shift;   // a group is 2^shift whole lanes; -1: it is not
};

// Lane j: the j-th expert by key[i] (of expert lane * NV + i; -inf: masked).  `pair`: a group's score is
// the sum of its two largest keys, not its largest.
template <typename F, int NV>
__device__ __forceinline__ int choose(const F (&key)[NV], const RouteShape& sh, bool pair)
{
    typedef typename Rank<F>::type R;
    const int lane = threadIdx.x & 31, e0 = lane * NV, per = sh.per;
    uint32_t allowed = kFull;   // bit g: experts of group g may be chosen
    if (sh.n_group > sh.topk_group) {
        F mine = lowest<F>();   // lane g: the score of group g
        if (sh.shift >= 0) {
            // A group is a power of two of whole lanes: the two largest by a butterfly in each.
            F a = lowest<F>(), b = lowest<F>();
#pragma unroll
            for (int i = 0; i < NV; ++i) merge_two(a, b, key[i], lowest<F>());
            for (int o = 1; o >> sh.shift == 0; o <<= 1)
                merge_two(a, b, __shfl_xor_sync(kFull, a, o), __shfl_xor_sync(kFull, b, o));
            mine = __shfl_sync(kFull, pair && b > lowest<F>() ? a + b : a, (lane << sh.shift) & 31);
        } else {
            for (int g = 0; g < sh.n_group; ++g) {
                F a = lowest<F>(), b = lowest<F>();
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (e0 + i >= g * per && e0 + i < (g + 1) * per) merge_two(a, b, key[i], lowest<F>());
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1)
                    merge_two(a, b, __shfl_xor_sync(kFull, a, o), __shfl_xor_sync(kFull, b, o));
                if (lane == g) mine = pair && b > lowest<F>() ? a + b : a;
            }
        }
        int rank = 0;
        for (int g = 0; g < sh.n_group; ++g) {
            const F other = __shfl_sync(kFull, mine, g);
            if (other > mine || (other == mine && g < lane)) ++rank;
        }
        if (lane >= sh.n_group) rank = 32;
        allowed = __ballot_sync(kFull, rank < sh.topk_group);
    }
    R rank[NV];
    int g = e0 / per, left = per - (e0 - g * per);   // the group at hand, and its experts from here on
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (left == 0) {
            left = per;
            ++g;
        }
        --left;
        rank[i] = key[i] > lowest<F>() ? rank_of(key[i]) : (R)1;
        if (e0 + i >= sh.E || !((allowed >> (g & 31)) & 1u)) rank[i] = 0;
    }
    R best = 0;   // of this lane
#pragma unroll
    for (int i = 0; i < NV; ++i) best = best > rank[i] ? best : rank[i];
    int chosen = 0;
    for (int j = 0; j < sh.k; ++j) {
        const R top = warp_top(best);
        const int who = __ffs(__ballot_sync(kFull, best == top)) - 1;   // the lowest lane has the lowest index
        int at = 0;
        if (lane == who) {
#pragma unroll
            for (int i = NV - 1; i >= 0; --i)
                if (rank[i] == top) at = i;
            best = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (i == at) rank[i] = 0;
                best = best > rank[i] ? best : rank[i];
            }
        }
        const int e = __shfl_sync(kFull, e0 + at, who);
        if (lane == j) chosen = e;
    }
    return chosen;
}

// Batcher's odd-even merge sort, descending.
template <int N>
__device__ __forceinline__ void sort_down(uint32_t (&r)[N])
{
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const uint32_t hi = max(r[i + j], r[i + j + q]), lo = min(r[i + j], r[i + j + q]);
                        r[i + j] = hi;
                        r[i + j + q] = lo;
                    }
}

__device__ __forceinline__ float key_of(uint32_t rank)   // of a rank above 1
{
    return __uint_as_float(rank ^ ((rank >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// A group's score from its two largest keys.  A sum that leaves fp32 stays finite: an infinite one would be a
// masked group's.
__device__ __forceinline__ float pair_score(float a, float b) { return fminf(fmaxf(a + b, -FLT_MAX), FLT_MAX); }

// The same choice from truncated keys, in about half the instructions: the low bits of a key's rank
// hold its place in the lane (the lowest index the highest), so a lane's keys sort as plain integers
// and the winner carries its index.  Ties of truncated keys go to the lower index.  Two keys p, q are near where
// they are not more than fixed + rel max(|p|, |q|) apart: a bound that grows with the keys at hand, not with the
// row's largest, because a mask of the type's lowest number is such a key (8192 tokens of 256 experts, a fifth
// of the biases so masked: 15.9 us, 54 with the row's largest; 15.8 and 16.7 where none is).  Where two neighbours in this order are near
// and have not the same inputs, the k and all that are near the k-th are put in order by their whole keys, one a
// lane.  (If a key is not near the k-th, none behind it is: rel < 1.)  *unsure is set where that is not enough: a group that is kept and
// one that is left out whose scores may be in the other order, or more than 32 candidates (with k = 32, one key
// near the 32nd is enough).
// exact: truncation loses nothing (bf16 logits without a bias), so that ties are ties.
// same(p, q): experts p and q have the same logit and bias.  exactly(e): the whole key of expert e, asked
// by the whole warp.
template <int NV, typename Same, typename Exactly>
__device__ __forceinline__ int choose_fast(const float (&key)[NV], const RouteShape& sh, bool pair, bool exact,
                                           float fixed, float rel, Same same, Exactly exactly, bool* unsure)
{
    constexpr uint32_t kPlace = NV - 1;   // NV is a power of two
    const int lane = threadIdx.x & 31, e0 = lane * NV, per = sh.per;
    // Masked: the lowest ranks there are, in the order of the index; an expert that is not there: 0.
    uint32_t rank[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const uint32_t r = key[i] > -CUDART_INF_F ? rank_of(key[i]) & ~kPlace : NV;   // a finite key's is above 2^23
        rank[i] = e0 + i < sh.E ? r | (kPlace - (uint32_t)i) : 0u;
    }
    const auto value_of = [](uint32_t r) { return r >= 2u * NV ? key_of(r & ~kPlace) : -CUDART_INF_F; };

    const bool whole = sh.shift >= 0;
    const bool grouped = sh.n_group > sh.topk_group;
    // Up to eight keys are sorted; longer lists cost more to sort than to search.
    if (NV <= 8 && (whole || !grouped)) sort_down<NV>(rank);
    if (grouped) {
        float mine = -CUDART_INF_F, off = 0.0f;   // lane g: the score of group g, and what it may be off by
        // Twice what the two keys' errors, their truncation and the sum's rounding come to.
        const auto off_by = [&](float a, float b) {
            return fixed + rel * fabsf(a) + (pair && b > -CUDART_INF_F ? rel * fabsf(b) : 0.0f);
        };
        if (whole) {
            float a = -CUDART_INF_F, b = -CUDART_INF_F;
            if (NV <= 8) {
                a = value_of(rank[0]);
                if (NV > 1) b = value_of(rank[NV > 1 ? 1 : 0]);
            } else {
#pragma unroll
                for (int i = 0; i < NV; ++i) merge_two(a, b, key[i], -CUDART_INF_F);
            }
            for (int o = 1; o >> sh.shift == 0; o <<= 1)
                merge_two(a, b, __shfl_xor_sync(kFull, a, o), __shfl_xor_sync(kFull, b, o));
            mine = __shfl_sync(kFull, pair && b > -CUDART_INF_F ? pair_score(a, b) : a, (lane << sh.shift) & 31);
            if (!exact) off = __shfl_sync(kFull, off_by(a, b), (lane << sh.shift) & 31);
        } else {
            for (int g = 0; g < sh.n_group; ++g) {
                float a = -CUDART_INF_F, b = -CUDART_INF_F;
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (e0 + i >= g * per && e0 + i < (g + 1) * per) merge_two(a, b, key[i], -CUDART_INF_F);
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1)
                    merge_two(a, b, __shfl_xor_sync(kFull, a, o), __shfl_xor_sync(kFull, b, o));
                if (lane == g) {
                    mine = pair && b > -CUDART_INF_F ? pair_score(a, b) : a;
                    off = off_by(a, b);
                }
            }
        }
        // The best groups one after another.
        uint32_t allowed = 0u, standing = lane < sh.n_group ? rank_of(mine) : 0u;
        for (int j = 0; j < sh.topk_group; ++j) {
            const uint32_t top = __reduce_max_sync(kFull, standing);
            const int g = __ffs(__ballot_sync(kFull, standing == top)) - 1;
            allowed |= 1u << g;
            if (lane == g) standing = 0u;
        }
        if (!exact) {
            // The least that one that is kept can have, and the most that one that is left out can have.  Masked
            // groups are not off; if one is kept, all that are left out are masked.
            const bool live = lane < sh.n_group && mine > -CUDART_INF_F, kept = (allowed >> lane) & 1u;
            const uint32_t least = __reduce_min_sync(kFull, live && kept ? rank_of(mine - off) : 0xFFFFFFFFu);
            const uint32_t most = __reduce_max_sync(kFull, live && !kept ? rank_of(mine + off) : 0u);
            if (most >= least) *unsure = true;
        }
        // Experts of the other groups are out.  (A rank holds its place, wherever sorting took it.)
        if (whole) {
            if (!((allowed >> (lane >> sh.shift)) & 1u)) {
#pragma unroll
                for (int i = 0; i < NV; ++i) rank[i] = 0u;
            }
        } else {
            int g = e0 / per, left = per - (e0 - g * per);   // rank is not sorted yet
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (left == 0) {
                    left = per;
                    ++g;
                }
                --left;
                if (!((allowed >> (g & 31)) & 1u)) rank[i] = 0u;
            }
        }
        if (NV <= 8 && !whole) sort_down<NV>(rank);
    }
    uint32_t head = rank[0];
    if (NV > 8) {
#pragma unroll
        for (int i = 1; i < NV; ++i) head = max(head, rank[i]);
    }
    // The best one left, whose truncated rank is `top`, is taken out.
    const auto take = [&](uint32_t top) {
        const int who = __ffs(__ballot_sync(kFull, (head & ~kPlace) == top)) - 1;   // the lowest lane: the lowest index
        const int e = __shfl_sync(kFull, e0 + (int)(kPlace - (head & kPlace)), who);
        if (NV <= 8) {
            if (lane == who) {
#pragma unroll
                for (int i = 0; i + 1 < NV; ++i) rank[i] = rank[i + 1];
                rank[NV - 1] = 0u;
            }
            head = rank[0];
        } else if (lane == who) {
            uint32_t best = 0u;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (rank[i] == head) rank[i] = 0u;
                best = max(best, rank[i]);
            }
            head = best;
        }
        return e;
    };
    const auto near = [&](float above, float below) {
        return !(above - below > fixed + rel * fmaxf(fabsf(above), fabsf(below)));
    };
    // The k best one after another.
    int chosen = 0, last_e = 0, n = 0;
    float last = 0.0f;
    bool doubt = false;
    for (; n < sh.k; ++n) {
        const uint32_t top = __reduce_max_sync(kFull, head & ~kPlace);
        const float value = value_of(top);
        const int e = take(top);
        if (!exact) {   // equal inputs have equal keys
            if (value > -CUDART_INF_F && n > 0 && near(last, value) && !same(last_e, e)) doubt = true;
            last = value;
            last_e = e;
        }
        if (lane == n) chosen = e;
    }
    const float next = exact ? -CUDART_INF_F : value_of(__reduce_max_sync(kFull, head & ~kPlace));
    if (next > -CUDART_INF_F && near(last, next)) {
        // Equal inputs stand in the order of the index: no doubt about the border if all that are near the k-th have
        // its inputs.  (Those before it have, unless there is doubt among them.)
        bool differ = doubt;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float v = value_of(rank[i]);
            if (v > -CUDART_INF_F && near(last, v)) differ |= !same(last_e, e0 + (int)(kPlace - (rank[i] & kPlace)));
        }
        if (__any_sync(kFull, differ)) {
            doubt = true;
            for (;; ++n) {   // all that are too near the k-th to be left out for certain
                const uint32_t top = __reduce_max_sync(kFull, head & ~kPlace);
                const float value = value_of(top);
                if (value == -CUDART_INF_F || !near(last, value)) break;
                if (n == 32) {   // no lane is left for it
                    *unsure = true;
                    break;
                }
                const int e = take(top);
                if (lane == n) chosen = e;
            }
        }
    }
    if (doubt) {
        // Lane i: candidate i's whole key, and how many come before it.
        const double whole_key = exactly(chosen);
        int before = 0;
        for (int i = 0; i < n; ++i) {
            const double other = __shfl_sync(kFull, whole_key, i);
            const int other_e = __shfl_sync(kFull, chosen, i);
            if (other > whole_key || (other == whole_key && other_e < chosen)) ++before;
        }
        int ordered = 0;
        for (int j = 0; j < sh.k; ++j) {
            const int e = __shfl_sync(kFull, chosen, __ffs(__ballot_sync(kFull, lane < n && before == j)) - 1);
            if (lane == j) ordered = e;
        }
        chosen = ordered;
    }
    return chosen;
}

template <typename L, int NV>
struct RouteRow {
    float l[NV];   // usable logits; -inf for the others
    float b[NV];   // usable biases; -inf for the others
    float top;     // the largest usable logit
    bool bad;      // a NaN or +inf somewhere in the row or the bias
};

// NV consecutive values from p, whole 16-byte loads where `wide`.
template <int NV>
__device__ __forceinline__ void load_some(const float* p, int n, bool wide, float (&v)[NV])
{
    if (NV % 4 == 0 && wide) {
#pragma unroll
        for (int i = 0; i < NV; i += 4) {
            float4 f = make_float4(-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F);
            if (i < n) f = __ldg(reinterpret_cast<const float4*>(p + i));
            v[i] = f.x;
            v[(i + 1) % NV] = f.y;
            v[(i + 2) % NV] = f.z;
            v[(i + 3) % NV] = f.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = i < n ? __ldg(p + i) : -CUDART_INF_F;
    }
}
template <int NV>
__device__ __forceinline__ void load_some(const uint16_t* p, int n, bool wide, float (&v)[NV])
{
    if (NV % 8 == 0 && wide) {
#pragma unroll
        for (int i = 0; i < NV; i += 8) {
            uint4 f = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);   // -inf
            if (i < n) f = __ldg(reinterpret_cast<const uint4*>(p + i));
            const uint32_t u[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[(i + 2 * j) % NV] = __uint_as_float(u[j] << 16);
                v[(i + 2 * j + 1) % NV] = __uint_as_float(u[j] & 0xFFFF0000u);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = i < n ? __uint_as_float((uint32_t)__ldg(p + i) << 16) : -CUDART_INF_F;
    }
}

// wide: E is a multiple of 8 and the rows are 16-byte aligned (then a lane's experts are too, and
// each 16-byte piece lies inside the row or outside it).
template <typename L, int NV>
__device__ __forceinline__ void load_route(RouteRow<L, NV>& r, const L* row, const float* bias, int E, bool wide)
{
    const int e0 = (threadIdx.x & 31) * NV;
    load_some<NV>(row + e0, E - e0, wide, r.l);
    if (bias) {
        load_some<NV>(bias + e0, E - e0, wide, r.b);
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) r.b[i] = 0.0f;
    }
    bool bad = false;
    float top = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        bad |= !(r.l[i] < CUDART_INF_F) || !(r.b[i] < CUDART_INF_F);
        if (!(r.l[i] < CUDART_INF_F)) r.l[i] = -CUDART_INF_F;
        if (!(r.b[i] < CUDART_INF_F)) r.b[i] = -CUDART_INF_F;
        top = fmaxf(top, r.l[i]);
    }
    r.bad = __any_sync(kFull, bad);
    r.top = warp_max(top);
}

// Whether all usable experts of the row have the same logit and the same bias, and (`pair`) as many of them count
// for the score of every group that has any: one, or two.  Their keys, and those groups' scores, are then equal.
template <typename L, int NV>
__device__ __forceinline__ bool uniform_row(const RouteRow<L, NV>& r, const RouteShape& sh, bool pair)
{
    const int e0 = (threadIdx.x & 31) * NV;
    float top_l = -CUDART_INF_F, low_l = CUDART_INF_F, top_b = -CUDART_INF_F, low_b = CUDART_INF_F;
    bool masked = false;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (r.l[i] > -CUDART_INF_F && r.b[i] > -CUDART_INF_F) {
            top_l = fmaxf(top_l, r.l[i]);
            low_l = fminf(low_l, r.l[i]);
            top_b = fmaxf(top_b, r.b[i]);
            low_b = fminf(low_b, r.b[i]);
        } else {
            masked |= e0 + i < sh.E;
        }
    }
    if (warp_max(top_l) != -warp_max(-low_l) || warp_max(top_b) != -warp_max(-low_b)) return false;
    if (!pair || !__any_sync(kFull, masked)) return true;
    int kinds = 0;   // 1: a group of one usable expert, 2: of more
    for (int g = 0; g < sh.n_group; ++g) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (e0 + i >= g * sh.per && e0 + i < (g + 1) * sh.per && r.l[i] > -CUDART_INF_F && r.b[i] > -CUDART_INF_F) ++n;
        n = warp_sum(n);
        if (n > 0) kinds |= n > 1 ? 2 : 1;
    }
    return kinds != 3;
}

// The choice from whole keys: the logits, or with a bias binary64 sums.  `fast`: what choose_fast made of it, which
// has the order of the index where nothing else orders the experts.
template <typename L, int NV, bool SOFTMAX>
__device__ __noinline__ int choose_exactly(const L* row, const float* bias, RouteShape sh, bool wide, int fast)
{
    RouteRow<L, NV> r;
    load_route<L, NV>(r, row, bias, sh.E, wide);
    if (uniform_row<L, NV>(r, sh, bias != nullptr && sh.n_group > sh.topk_group)) return fast;
    if (!bias) return choose<float, NV>(r.l, sh, false);
    double key[NV], total = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        key[i] = 0.0;
        if (r.l[i] > -CUDART_INF_F) key[i] = SOFTMAX ? exp((double)r.l[i] - (double)r.top) : 1.0 / (1.0 + exp(-(double)r.l[i]));
        total += key[i];
    }
    if (SOFTMAX) total = warp_sum(total);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (SOFTMAX) key[i] = key[i] / total;
        key[i] = r.l[i] > -CUDART_INF_F && r.b[i] > -CUDART_INF_F ? key[i] + (double)r.b[i] : -CUDART_INF;
    }
    return choose<double, NV>(key, sh, true);
}

template <typename L, int NV, bool SOFTMAX>
__global__ void __launch_bounds__(128) moe_route_kernel(const L* __restrict__ logits, const float* __restrict__ bias,
                                                        int64_t T, RouteShape sh, bool wide, int renorm, float scale,
                                                        int32_t* __restrict__ idx, float* __restrict__ w)
{
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (t >= T) return;
    const L* row = logits + t * sh.E;
    RouteRow<L, NV> r;
    load_route<L, NV>(r, row, bias, sh.E, wide);

    // Scores.  e^x by __expf is off by (2 + 1.2 |x|) 2^-23 of itself, so sigmoid by less than 2^-22 in all
    // (s (1 - s) (2 + 1.2 |l|) < 0.65), and softmax, whose sum of up to 1024 terms adds 37 roundings, by
    // less than 2^-18.  A key's own rounding is 2^-24 of it.  The bound of choose_fast
    // is twice the sum of two such errors.
    float total = 0.0f, key[NV];
    if (SOFTMAX || bias) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            key[i] = 0.0f;
            if (r.l[i] > -CUDART_INF_F)
                key[i] = SOFTMAX ? __expf(r.l[i] - r.top) : __fdividef(1.0f, 1.0f + __expf(-r.l[i]));
            total += key[i];
        }
        if (SOFTMAX) total = warp_sum(total);
    }
    // Truncation takes less than NV steps off a key, each at most 2^-23 of the key, or 2^-149.
    constexpr float kCut = NV * 0x1p-23f;
    const bool exact = !bias && sizeof(L) == 2;
    const float fixed = (bias ? (SOFTMAX ? 0x1p-16f : 0x1p-20f) : 0.0f) + 4 * NV * 0x1p-149f;
    const float rel = (bias ? 0x1p-22f : 0.0f) + 2.0f * kCut;
    const float inv = SOFTMAX ? __fdividef(1.0f, total) : 1.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (bias)
            key[i] = r.l[i] > -CUDART_INF_F && r.b[i] > -CUDART_INF_F ? (SOFTMAX ? key[i] * inv : key[i]) + r.b[i] : -CUDART_INF_F;
        else
            key[i] = r.l[i];
    }
    bool unsure = false;
    const auto same = [&](int p, int q) {
        return load_logit(row + p) == load_logit(row + q) && (!bias || bias[p] == bias[q]);
    };
    const auto exactly = [&](int e) {
        const double x = load_logit(row + e);
        if (!bias) return x < CUDART_INF ? x : -CUDART_INF;
        double sum = 0.0;
        if (SOFTMAX) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (r.l[i] > -CUDART_INF_F) sum += exp((double)r.l[i] - (double)r.top);
            sum = warp_sum(sum);
        }
        const double b = bias[e];
        if (!(x > -CUDART_INF && x < CUDART_INF && b > -CUDART_INF && b < CUDART_INF)) return -CUDART_INF;
        return (SOFTMAX ? exp(x - (double)r.top) / sum : 1.0 / (1.0 + exp(-x))) + b;
    };
    int chosen = choose_fast<NV>(key, sh, bias != nullptr, exact, fixed, rel, same, exactly, &unsure);
    if (unsure) chosen = choose_exactly<L, NV, SOFTMAX>(row, bias, sh, wide, chosen);   // the same for the whole warp

    // Weights, in fp32: only the order needs more.  The renormalised ones divide scores by their sum, so scores that would underflow are
    // first scaled by exp(-m), m = min(largest chosen logit, 0): sigmoid(l) e^-m = e^(l-m) / (1 + e^l).
    bool usable = false;
    float x = -CUDART_INF_F;
    if (lane < sh.k) {
        x = load_logit(row + chosen);
        const float b = bias ? bias[chosen] : 0.0f;
        usable = x > -CUDART_INF_F && x < CUDART_INF_F && b > -CUDART_INF_F && b < CUDART_INF_F;
    }
    const float best = warp_max(usable ? x : -CUDART_INF_F);
    float s = 0.0f;
    if (SOFTMAX) {
        if (usable) s = renorm ? expf(x - best) : expf(x - r.top) / total;
    } else {
        const float m = renorm ? fminf(best, 0.0f) : 0.0f;   // the same for the whole warp
        const float z = expf(-fabsf(x));
        float num = x > 0.0f ? 1.0f : z;
        if (m < 0.0f) num = expf(x - m);
        if (usable) s = num / (1.0f + z);
    }
    if (renorm) {
        const float sum = warp_sum(s);
        s = sum > 0.0f ? s / sum : 0.0f;
    }
    if (lane < sh.k) {
        idx[t * sh.k + lane] = chosen;
        w[t * sh.k + lane] = r.bad ? CUDART_NAN_F : s * scale;
    }
}

// Gradient of the weights with respect to the logits, g = dL/dw, p_j = w_j / scale:
//   renormalised:  sigmoid  dl_j = w_j (1 - s_j) sum_i p_i (g_j - g_i)     softmax the same without (1 - s_j)
//   as they are:   sigmoid  dl_j = w_j (1 - s_j) g_j                       softmax dl_e = [chosen] w_e g_e - p_e sum_i w_i g_i
// (sum_i p_i = 1 turns g_j - sum_i p_i g_i into differences, which do not cancel.)  A slot of
// weight zero takes no part; every other expert's gradient is zero and is written.
// One warp per token: the row without the choice is written whole (zeros; DENSE, for softmax as it is,
// -p_e sum), then lane j its expert's value over it.
template <int NV>
__device__ __forceinline__ void store_some(float* p, int n, bool wide, const float (&v)[NV])
{
    if (NV % 4 == 0 && wide) {
#pragma unroll
        for (int i = 0; i < NV; i += 4)
            if (i < n)
                *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[(i + 1) % NV], v[(i + 2) % NV], v[(i + 3) % NV]);
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i < n) p[i] = v[i];
    }
}
template <int NV>
__device__ __forceinline__ void store_some(uint16_t* p, int n, bool wide, const float (&v)[NV])
{
    if (NV % 8 == 0 && wide) {
#pragma unroll
        for (int i = 0; i < NV; i += 8)
            if (i < n)
                *reinterpret_cast<uint4*>(p + i) =
                    make_uint4(bf16_rn(v[i]) | (bf16_rn(v[(i + 1) % NV]) << 16), bf16_rn(v[(i + 2) % NV]) | (bf16_rn(v[(i + 3) % NV]) << 16),
                               bf16_rn(v[(i + 4) % NV]) | (bf16_rn(v[(i + 5) % NV]) << 16), bf16_rn(v[(i + 6) % NV]) | (bf16_rn(v[(i + 7) % NV]) << 16));
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i < n) store_logit(p + i, v[i]);
    }
}

template <typename L, int NV, bool DENSE>
__global__ void __launch_bounds__(128) moe_route_backward_kernel(const float* __restrict__ dw,
                                                                 const float* __restrict__ w,
                                                                 const int32_t* __restrict__ idx,
                                                                 const L* __restrict__ logits, int64_t T, int E,
                                                                 int k, bool wide, int sigmoid, int renorm,
                                                                 float scale, L* dlogits)
{
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (t >= T) return;
    const L* row = logits + t * E;
    int e = -1;
    float g = 0.0f, wt = 0.0f;
    if (lane < k) {
        e = idx[t * k + lane];
        wt = w[t * k + lane];
        g = dw[t * k + lane];
        if (e < 0 || e >= E) {
            latch_status(kDevBadIndex);
            e = -1;
        }
    }
    float x = 0.0f;
    if ((DENSE || sigmoid) && e >= 0) x = load_logit(row + e);
    float v[NV];
    float top = -CUDART_INF_F, inv = 0.0f;
    if (DENSE) {
        load_some<NV>(row + lane * NV, E - lane * NV, wide, v);
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!(v[i] < CUDART_INF_F)) v[i] = -CUDART_INF_F;
            top = fmaxf(top, v[i]);
        }
        top = warp_max(top);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            v[i] = v[i] > -CUDART_INF_F ? expf(v[i] - top) : 0.0f;
            total += v[i];
        }
        total = warp_sum(total);
        inv = total > 0.0f ? 1.0f / total : 0.0f;
    }
    const bool live = e >= 0 && wt != 0.0f;
    const float p = live ? wt / scale : 0.0f;
    if (!live) g = 0.0f;
    float d = 0.0f;
    if (renorm) {
        for (int i = 0; i < k; ++i) d += __shfl_sync(kFull, p, i) * (g - __shfl_sync(kFull, g, i));
    } else {
        d = g;
    }
    if (sigmoid && live) d *= 1.0f / (1.0f + expf(x));   // 1 - sigmoid(x)
    d = live ? d * wt : 0.0f;
    const float sum = DENSE ? warp_sum(d) : 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = DENSE ? -sum * (v[i] * inv) : 0.0f;
    store_some<NV>(dlogits + t * E + lane * NV, E - lane * NV, wide, v);
    // The same expert twice: each of its lanes writes the sum.
    float mine = DENSE && x < CUDART_INF_F && x > -CUDART_INF_F ? -sum * (expf(x - top) * inv) : 0.0f;
    for (int i = 0; i < k; ++i) {
        const float di = __shfl_sync(kFull, d, i);
        if (__shfl_sync(kFull, e, i) == e) mine += di;
    }
    __syncwarp();   // behind the row's stores by other lanes
    if (e >= 0) store_logit(dlogits + t * E + e, mine);
}

// ------------------------------------------------------------------------------------------
// The plan: a stable counting sort of the M = T k slots by expert, in one launch of one cluster.  Warp w
// of CTA c owns a contiguous run of slots; it counts its experts 32 at a time, a slot's rank among the
// 32 coming from one ballot per bit of the expert (with match.any, which loops over the distinct values,
// 65536 slots took 22 us instead of 15).  The counts become starting rows by a scan over (expert, CTA, warp) through
// distributed shared memory, and a second walk over the same slots places them.  No atomics on the rows,
// so the order is a function of the input alone.  Bound by latency: 65536 slots of 256 experts take 15 us.
// ------------------------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanCtas = 8;    // the portable cluster size
constexpr int kPlanAhead = 8;   // blocks of 32 slots whose loads are in flight together

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A word of another CTA's shared memory, at the address that it has in this one.
__device__ __forceinline__ int32_t peer_word(const int32_t* p, uint32_t cta)
{
    uint32_t a;
    int32_t v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(cta));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

// The lanes with the same value of `bits` bits as this one.
__device__ __forceinline__ unsigned same_lanes(int e, int bits)
{
    unsigned m = kFull;
#pragma unroll
    for (int b = 0; b < 10; ++b) {   // kMoeMaxExperts = 2^10
        if (b >= bits) break;
        const bool one = (e >> b) & 1;
        const unsigned v = __ballot_sync(kFull, one);
        m &= one ? v : ~v;
    }
    return m;
}

// Shared memory: counts [kPlanWarps][E] (16 bits would do for the counts, not for the rows), totals [E],
// starts [E].
constexpr int plan_smem(int E) { return (kPlanWarps + 2) * E * (int)sizeof(int32_t); }

template <int CTAS>
__global__ void __launch_bounds__(kPlanThreads) moe_plan_kernel(const int32_t* __restrict__ idx, int64_t M, int E,
                                                                int32_t* __restrict__ offsets,
                                                                int32_t* __restrict__ slots,
                                                                int32_t* __restrict__ rows)
{
    griddep_launch_dependents();
    griddep_wait();
    extern __shared__ int32_t counts[];
    __shared__ int32_t part[kPlanWarps];
    __shared__ int32_t s_bad;
    int32_t* totals = counts + kPlanWarps * E;   // this CTA's slots of each expert
    int32_t* starts = totals + E;                // the first row of this CTA's slots of each expert
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const uint32_t cta = CTAS > 1 ? cluster_rank() : 0;
    for (int i = tid; i < kPlanWarps * E; i += kPlanThreads) counts[i] = 0;
    if (tid == 0) s_bad = 0;
    __syncthreads();
    // Whole blocks of 32 slots, dealt out evenly to the CTAS x 32 warps in order.
    const int64_t blocks = (M + 31) >> 5;
    const int64_t who = (int64_t)cta * kPlanWarps + w, all = CTAS * kPlanWarps;
    const int64_t lo = 32 * (blocks * who / all), hi = min(M, 32 * (blocks * (who + 1) / all));
    int32_t* mine = counts + w * E;
    const int bits = 32 - __clz(E - 1);   // 0 for one expert
    bool bad = false;
    int32_t expert[kPlanAhead];   // of this lane's slots in the blocks at hand, -1 for none
    int32_t place[kPlanAhead];    // of a slot with an expert: 64 * (slots of that expert in the block) + (those before this one)
    auto load = [&](int64_t at) {
#pragma unroll
        for (int u = 0; u < kPlanAhead; ++u) {
            const int64_t i = at + 32 * u + lane;
            expert[u] = i < hi ? __ldg(idx + i) : -1;
            if (expert[u] < 0 || expert[u] >= E) {
                bad |= i < hi;
                expert[u] = -1;
            }
        }
#pragma unroll
        for (int u = 0; u < kPlanAhead; ++u) {
            if (at + 32 * u >= hi) break;
            const unsigned peers = same_lanes(expert[u], bits) & __ballot_sync(kFull, expert[u] >= 0);
            place[u] = 64 * __popc(peers) + __popc(peers & ((1u << lane) - 1u));
        }
    };
    for (int64_t b = lo; b < hi; b += 32 * kPlanAhead) {
        load(b);
#pragma unroll
        for (int u = 0; u < kPlanAhead; ++u) {
            if (b + 32 * u >= hi) break;
            if (expert[u] >= 0 && (place[u] & 63) == 0) mine[expert[u]] += place[u] >> 6;
            __syncwarp();
        }
    }
    if (bad) s_bad = 1;
    __syncthreads();
    // Per expert: the counts of the warps become their exclusive sums, and the CTA's total.
    for (int e = tid; e < E; e += kPlanThreads) {
        int32_t sum = 0;
#pragma unroll 8
        for (int v = 0; v < kPlanWarps; ++v) {
            const int32_t c = counts[v * E + e];
            counts[v * E + e] = sum;
            sum += c;
        }
        totals[e] = sum;
    }
    if (CTAS > 1) cluster_sync(); else __syncthreads();
    // Every CTA scans the experts' totals over all CTAs; E <= kPlanThreads, one expert a thread.
    int32_t before = 0, total = 0;
    if (tid < E) {
#pragma unroll
        for (uint32_t c = 0; c < CTAS; ++c) {
            const int32_t n = CTAS > 1 ? peer_word(totals + tid, c) : totals[tid];
            if (c < cta) before += n;
            total += n;
        }
    }
    int32_t any_bad = 0;
#pragma unroll
    for (uint32_t c = 0; c < CTAS; ++c) any_bad |= CTAS > 1 ? peer_word(&s_bad, c) : s_bad;
    int32_t incl = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) part[w] = incl;
    if (CTAS > 1) cluster_sync(); else __syncthreads();   // and no CTA leaves while another reads its words
    if (w == 0) {
        const int32_t v = part[lane];
        int32_t c = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t y = __shfl_up_sync(kFull, c, o);
            if (lane >= o) c += y;
        }
        part[lane] = c - v;
    }
    __syncthreads();
    if (any_bad) {   // an expert outside [0, E): an empty plan, which every reader refuses
        if (cta == 0 && tid == 0) latch_status(kDevBadIndex);
        if (cta == 0)
            for (int i = tid; i <= E; i += kPlanThreads) offsets[i] = 0;
        for (int64_t i = lo + lane; i < hi; i += 32) {
            slots[i] = -1;
            rows[i] = -1;
        }
        return;
    }
    if (tid < E) {
        const int32_t first = part[w] + incl - total;
        starts[tid] = first + before;
        if (cta == 0) offsets[tid] = first;
    }
    if (cta == 0 && tid == 0) offsets[E] = (int32_t)M;
    __syncthreads();
    for (int64_t b = lo; b < hi; b += 32 * kPlanAhead) {
        if (hi - lo > 32 * kPlanAhead) load(b);   // else they are still at hand
#pragma unroll
        for (int u = 0; u < kPlanAhead; ++u) {
            if (b + 32 * u >= hi) break;
            const int e = expert[u];
            int32_t base = 0;
            if (e >= 0) base = mine[e];
            __syncwarp();
            if (e >= 0) {
                const int32_t r = starts[e] + base + (place[u] & 63);
                slots[r] = (int32_t)(b + 32 * u + lane);
                rows[b + 32 * u + lane] = r;
                if ((place[u] & 63) == 0) mine[e] = base + (place[u] >> 6);
            }
            __syncwarp();
        }
    }
}

// The padded 128-row groups of expert-ordered rows (as act_128x1_t_ragged_kernel counts them), in
// shared memory of group_table_bytes(E): E + 1 offsets, E + 1 counts of the groups before an expert,
// one flag.
constexpr int group_table_bytes(int E) { return ((2 * (E + 1) + 1) * 4 + 15) & ~15; }
struct GroupTable {
    int* off;
    int* pre;
    int* bad;
    __device__ GroupTable(void* smem, int E)
        : off(static_cast<int*>(smem)), pre(off + E + 1), bad(pre + E + 1) {}
};

// Fills the table (whole CTA; `offsets` null: one sequence of M rows).  False if the offsets are
// malformed; FP8Q_DEV_BAD_OFFSETS is then latched.
__device__ __forceinline__ bool group_table(const GroupTable& t, const int32_t* __restrict__ offsets, int E, int64_t M,
                                            int64_t Kcap)
{
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (w == 0) {
        if (offsets) {
            for (int i = lane; i <= E; i += 32) t.off[i] = __ldg(offsets + i);
        } else if (lane < 2) {
            t.off[lane] = lane ? (int)M : 0;
        }
        __syncwarp();
        const int per = (E + 31) >> 5;
        const int lo = min(E, lane * per), hi = min(E, lo + per);
        int local = 0;
        bool bad = false;
        for (int e = lo; e < hi; ++e) {
            const int64_t cnt = (int64_t)t.off[e + 1] - t.off[e];
            bad |= cnt < 0 || cnt > M;
            local += cnt > 0 && cnt <= M ? (int)((cnt + 127) >> 7) : 0;
        }
        int incl = local;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += y;
        }
        int run = incl - local;
        for (int e = lo; e < hi; ++e) {
            t.pre[e] = run;
            const int64_t cnt = (int64_t)t.off[e + 1] - t.off[e];
            run += cnt > 0 && cnt <= M ? (int)((cnt + 127) >> 7) : 0;
        }
        if (lane == 31) {
            t.pre[E] = incl;
            bad |= t.off[0] != 0 || (int64_t)t.off[E] != M || (int64_t)incl * 128 > Kcap;
        }
        bad = __any_sync(kFull, bad);
        if (lane == 0) *t.bad = bad ? 1 : 0;
    }
    __syncthreads();
    if (*t.bad && threadIdx.x == 0) latch_status(kDevBadOffsets);
    return !*t.bad;
}

// First row and number of rows of padded group g < pre[E].
__device__ __forceinline__ void group_rows(const GroupTable& t, int E, int g, int64_t& r0, int& nvalid)
{
    int lo = 0, hi = E;   // pre[lo] <= g < pre[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.pre[mid] <= g) lo = mid; else hi = mid;
    }
    r0 = (int64_t)t.off[lo] + 128ll * (g - t.pre[lo]);
    nvalid = (int)min((int64_t)128, (int64_t)t.off[lo + 1] - r0);
}

// ------------------------------------------------------------------------------------------
// Dispatch, 1x128 codes: row rows[t,j] holds (weight of the slot) * x[t].  A warp takes four 128-element
// tiles of one token (eight lanes each), reads them once and writes them to the token's k rows.  Without
// weights the k rows hold the same codes, which are formed once.
// Bound by the writes: 8192 tokens x 8 of 7168 channels take 130 us (4.6 TB/s), 100 without the scales,
// whose neighbours in memory belong to other tokens and so leave 4 bytes at a time.
// ------------------------------------------------------------------------------------------
template <bool WEIGHTED>
__global__ void __launch_bounds__(256) moe_dispatch_rows_kernel(const uint16_t* __restrict__ x,
                                                                const int32_t* __restrict__ rows,
                                                                const float* __restrict__ weights, uint32_t T,
                                                                uint32_t k, uint32_t C, uint8_t* __restrict__ q,
                                                                float* __restrict__ s,
                                                                const int32_t* __restrict__ offsets, int E,
                                                                int64_t Kcap)
{
    griddep_launch_dependents();
    griddep_wait();
    if (offsets) {   // the 128x1 form follows: write neither if it will refuse the offsets
        extern __shared__ __align__(16) uint8_t smem[];
        if (!group_table(GroupTable(smem, E), offsets, E, (int64_t)T * k, Kcap)) return;
    }
    const uint32_t M = T * k, CB = C >> 7, quads = (CB + 3) >> 2, items = T * quads;
    const int lane = threadIdx.x & 31, sub = lane & 7;
    const uint32_t warps = (gridDim.x * blockDim.x) >> 5;
    // An item's loads are issued before the item ahead of it is written: behind those writes they take
    // several microseconds.
    uint4 a, b;
    int32_t row;
    float wt;
    auto load = [&](uint32_t it, uint4& a, uint4& b, int32_t& row, float& wt) {
        const uint32_t t = it / quads, kb = (it - t * quads) * 4 + (lane >> 3);
        row = -1;
        wt = 1.0f;
        if (lane < k && it < items) {
            row = __ldg(rows + t * k + lane);
            if (WEIGHTED) wt = __ldg(weights + t * k + lane);
        }
        a = make_uint4(0u, 0u, 0u, 0u);
        b = a;
        if (kb < CB && it < items) {
            const uint4* p = reinterpret_cast<const uint4*>(x + (size_t)t * C + kb * 128) + 2 * sub;
            a = __ldg(p);
            b = __ldg(p + 1);
        }
    };
    uint32_t it = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (it < items) load(it, a, b, row, wt);
    uint4 next_a, next_b;
    int32_t next_row;
    float next_wt;
    for (; it < items; it += warps, a = next_a, b = next_b, row = next_row, wt = next_wt) {
        load(it + warps, next_a, next_b, next_row, next_wt);
        const uint32_t t = it / quads, kb = (it - t * quads) * 4 + (lane >> 3);
        const bool live = kb < CB;
        if (lane < k && (row < 0 || row >= (int32_t)M)) {
            latch_status(kDevBadIndex);
            row = -1;
        }
        const float amax = max8(amax16(a, b));
        uint8_t* qb = q + kb * 128 + 16 * sub;
        float* sb = s + (size_t)kb * M;
        if (!WEIGHTED) {
            float sc, inv;
            group_scale<false>(amax, sc, inv);
            const uint2 lo = quant8(a, inv), hi = quant8(b, inv);
            for (uint32_t j = 0; j < k; ++j) {
                const int32_t r = __shfl_sync(kFull, row, j);
                if (r < 0 || !live) continue;
                *reinterpret_cast<uint4*>(qb + (size_t)r * C) = make_uint4(lo.x, lo.y, hi.x, hi.y);
                if (sub == 0) sb[r] = sc;
            }
        } else {
            const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            float sc8 = 0.0f, inv8 = 0.0f;   // lane sub: of copy (j & ~7) + sub
            for (uint32_t j = 0; j < k; ++j) {
                const int32_t r = __shfl_sync(kFull, row, j);
                const float wj = __shfl_sync(kFull, wt, j);
                // |w| max|x| is the largest |w x|: rounding keeps the order.
                if ((j & 7) == 0) {
                    const float w8 = __shfl_sync(kFull, wt, j + sub);
                    group_scale<false>(__fmul_rn(fabsf(w8), amax), sc8, inv8);
                }
                const float sc = __shfl_sync(kFull, sc8, j & 7, 8), inv = __shfl_sync(kFull, inv8, j & 7, 8);
                if (r < 0 || !live) continue;
                uint32_t c[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 w2 = make_float2(wj, wj), i2 = make_float2(inv, inv);
                    const float2 lo = mul2(mul2(widen(u[2 * i]), w2), i2), hi = mul2(mul2(widen(u[2 * i + 1]), w2), i2);
                    c[i] = codes4(lo.x, lo.y, hi.x, hi.y);
                }
                *reinterpret_cast<uint4*>(qb + (size_t)r * C) = make_uint4(c[0], c[1], c[2], c[3]);
                if (sub == 0) sb[r] = sc;
            }
        }
    }
}

// ------------------------------------------------------------------------------------------
// Dispatch, ragged 128x1 codes.  A CTA takes tiles of one padded group (128 rows) x 128 channels; the
// gathered rows come into shared memory by asynchronous copies, 256 bytes of a row at a time, while the
// previous tile is quantised.  Warp w quantises channels 16w .. 16w+15: lane (r, h) = (lane >> 1,
// lane & 1) holds consecutive rows of channels 8h .. 8h+7, so the column maxima need shuffles only, and a
// channel's 128 codes leave as one line, 8 bytes from each r.  One barrier a tile.
// Tiles are ordered by channel block first: at any time the whole grid gathers from a few channel blocks
// of x (2 MB per 128 channels of 8192 tokens), so a token's k reads find it in L2 although x as a whole need
// not fit.  65536 rows of 7168 channels in 645 groups take 207 us: the copies (through L2) and stores
// alone 154 us, the arithmetic and stores alone 194 us.
// ------------------------------------------------------------------------------------------
// 16-byte piece c of row r of a staged tile (256 bytes a row) lies at piece c ^ 2 ((r >> 3) & 3) of the
// row: the four r of a quarter-warp then read different banks.
__device__ __forceinline__ uint32_t stage_at(int r, int c) { return r * 256 + ((c ^ (((r >> 3) & 3) << 1)) << 4); }

constexpr int kStageBytes = 128 * 256;
struct GatherSmem {   // byte offsets
    static constexpr int token = 2 * kStageBytes;          // [3 items][128], -1: no row
    static constexpr int weight = token + 3 * 128 * 4;     // [3 items][128]
    static constexpr int rows = weight + 3 * 128 * 4;      // [3 items]: the rows of its group
    static constexpr int table = rows + 16;
};
constexpr int gather_smem(int E) { return GatherSmem::table + group_table_bytes(E); }

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live)   // zeros unless live
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

// Larger magnitude of each of two bf16 pairs, its sign unspecified; a NaN loses.
__device__ __forceinline__ uint32_t maxabs2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int j) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; }

// Scales of a warp's 16 columns from m[j], the largest magnitude in this lane's rows of column 8h + j:
// stores them (lanes r < 8: column 8h + r) and returns in m the factors 1 / scale of columns 8h + j.
__device__ __forceinline__ void column_scales(float (&m)[8], int lane, float* __restrict__ st)
{
    const bool b0 = lane & 2, b1 = lane & 4, b2 = lane & 8;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float send = b2 ? m[j] : m[j + 4], keep = b2 ? m[j + 4] : m[j];
        m[j] = fmaxf(keep, __shfl_xor_sync(kFull, send, 8));
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float send = b1 ? m[j] : m[j + 2], keep = b1 ? m[j + 2] : m[j];
        m[j] = fmaxf(keep, __shfl_xor_sync(kFull, send, 4));
    }
    const float send = b0 ? m[0] : m[1], keep = b0 ? m[1] : m[0];
    float a = fmaxf(keep, __shfl_xor_sync(kFull, send, 2));
    a = fmaxf(a, __shfl_xor_sync(kFull, a, 16));
    float sc, inv;
    group_scale<false>(a, sc, inv);
    if (lane < 16) st[8 * (lane & 1) + (lane >> 1)] = sc;
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = __shfl_sync(kFull, inv, 2 * j + (lane & 1));
}

// n / d for n < 2^31 and the d that (mul, shift) were made for.
struct FastDiv {
    uint32_t mul, shift;
};
__device__ __forceinline__ uint32_t div_by(uint32_t n, FastDiv d) { return (__umulhi(n, d.mul) + n) >> d.shift; }

// A CTA's tiles, one after another: items of kColBlocks channel blocks of one group, every gridDim.x-th
// in the order of the channel blocks, then the groups; `slot` counts the items modulo 3.
constexpr uint32_t kColBlocks = 4;
struct TileWalk {
    uint32_t cb, first, g, slot, groups, CB, dcb, dg;
    __device__ TileWalk(uint32_t n, uint32_t blocks)
        : first(blockIdx.x / n * kColBlocks), g(blockIdx.x % n), slot(0), groups(n), CB(blocks),
          dcb(gridDim.x / n * kColBlocks), dg(gridDim.x % n)
    {
        cb = first;
    }
    __device__ bool live() const { return cb < CB; }
    __device__ bool at_first() const { return cb == first; }
    __device__ void next_item()
    {
        first += dcb;
        g += dg;
        if (g >= groups) {
            g -= groups;
            first += kColBlocks;
        }
        cb = first;
        slot = slot == 2 ? 0 : slot + 1;
    }
    __device__ void next()
    {
        if (++cb == first + kColBlocks || cb == CB) next_item();
    }
};

// One warp's 16 channels of a tile: lane (r, h) has rows R r .. of channels 8h .. 8h+7.  R = 8, or 4 where the
// group has at most 64 rows; the other half of each line is then written as it is, zero.  (The whole dispatch
// of 250 tokens to 8 of 256 experts: 76 us instead of 89, of 8192 tokens 352 instead of 355.)
template <bool WEIGHTED, int R>
__device__ __forceinline__ void quantise_columns(const uint8_t* tile, const float* weight, int w, int lane,
                                                 float* __restrict__ st, uint8_t* __restrict__ out, int64_t Kcap)
{
    const int r = lane >> 1, h = lane & 1;
    uint4 v[R];
    float wt[R];
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] = *reinterpret_cast<const uint4*>(tile + stage_at(R * r + i, 2 * w + h));
    if (WEIGHTED) {
#pragma unroll
        for (int i = 0; i < R; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(weight + R * r + i);
            wt[i] = f.x;
            wt[i + 1] = f.y;
            wt[i + 2] = f.z;
            wt[i + 3] = f.w;
        }
    }
    float m[8];
    if (WEIGHTED) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            m[2 * j] = m[2 * j + 1] = 0.0f;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float2 f = mul2(widen(word(v[i], j)), both(wt[i]));
                m[2 * j] = fmaxf(m[2 * j], fabsf(f.x));
                m[2 * j + 1] = fmaxf(m[2 * j + 1], fabsf(f.y));
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t p = 0u;
#pragma unroll
            for (int i = 0; i < R; ++i) p = maxabs2(p, word(v[i], j));
            m[2 * j] = fabsf(bf16_lo(p));
            m[2 * j + 1] = fabsf(bf16_hi(p));
        }
    }
    column_scales(m, lane, st);
    out += 8 * h * Kcap + R * r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {   // channels 8h + 2j, + 1
        const float2 inv = make_float2(m[2 * j], m[2 * j + 1]);
        float2 y[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            y[i] = widen(word(v[i], j));
            if (WEIGHTED) y[i] = mul2(y[i], both(wt[i]));
            y[i] = mul2(y[i], inv);
        }
        const uint32_t lo0 = codes4(y[0].x, y[1].x, y[2].x, y[3].x), lo1 = codes4(y[0].y, y[1].y, y[2].y, y[3].y);
        if (R == 8) {
            *reinterpret_cast<uint2*>(out) = make_uint2(lo0, codes4(y[R - 4].x, y[R - 3].x, y[R - 2].x, y[R - 1].x));
            out += Kcap;
            *reinterpret_cast<uint2*>(out) = make_uint2(lo1, codes4(y[R - 4].y, y[R - 3].y, y[R - 2].y, y[R - 1].y));
        } else {
            *reinterpret_cast<uint32_t*>(out) = lo0;
            *reinterpret_cast<uint32_t*>(out + 64) = 0u;
            out += Kcap;
            *reinterpret_cast<uint32_t*>(out) = lo1;
            *reinterpret_cast<uint32_t*>(out + 64) = 0u;
        }
        out += Kcap;
    }
}

template <bool WEIGHTED>
__global__ void __launch_bounds__(256, 3) moe_dispatch_cols_kernel(
    const uint16_t* __restrict__ x, const int32_t* __restrict__ slots, const float* __restrict__ weights,
    const int32_t* __restrict__ offsets, int E, int64_t M, FastDiv k, uint32_t C, uint8_t* __restrict__ qt,
    float* __restrict__ st, int64_t Kcap)
{
    griddep_launch_dependents();
    griddep_wait();
    extern __shared__ __align__(16) uint8_t smem[];
    int* s_token = reinterpret_cast<int*>(smem + GatherSmem::token);
    float* s_weight = reinterpret_cast<float*>(smem + GatherSmem::weight);
    int* s_rows = reinterpret_cast<int*>(smem + GatherSmem::rows);
    const GroupTable table(smem + GatherSmem::table, E);
    if (!group_table(table, offsets, E, M, Kcap)) return;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const uint32_t stage = smem_u32(smem);
    TileWalk at(table.pre[E], C >> 7), ahead = at, later = at;   // this tile, the next one, an item to look up

    // The token (and weight) of row `tid` of an item, for the threads that have one.
    int token, nvalid = 0;
    float weight;
    auto look_up = [&]() {
        token = -1;
        weight = 0.0f;
        if (tid < 128 && later.live()) {
            int64_t r0;
            group_rows(table, E, (int)later.g, r0, nvalid);
            if (tid < nvalid) {
                const int32_t slot = __ldg(slots + r0 + tid);
                if (slot >= 0 && slot < M) {
                    token = (int)div_by((uint32_t)slot, k);
                    if (WEIGHTED) weight = __ldg(weights + slot);
                } else {
                    latch_status(kDevBadIndex);
                }
            }
        }
    };
    auto note = [&]() {
        if (tid < 128) {
            s_token[128 * later.slot + tid] = token;
            if (WEIGHTED) s_weight[128 * later.slot + tid] = weight;
            if (tid == 0) s_rows[later.slot] = nvalid;
        }
    };
    // Copies of a tile's rows: half-warp (w, half) brings rows 16w + 8 half + i.  Rows 64 .. of a group that
    // has none there are not read.
    auto fetch = [&](const TileWalk& t, int buf) {
        if (t.live() && (w < 4 || s_rows[t.slot] > 64)) {
            const int row = 16 * w + 8 * (lane >> 4), c = lane & 15;
            const int4 ta = *reinterpret_cast<const int4*>(s_token + 128 * t.slot + row);
            const int4 tb = *reinterpret_cast<const int4*>(s_token + 128 * t.slot + row + 4);
            const int n[8] = {ta.x, ta.y, ta.z, ta.w, tb.x, tb.y, tb.z, tb.w};
            const uint16_t* src = x + t.cb * 128 + 8 * c;
            const uint32_t dst = stage + buf * kStageBytes;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                copy16(dst + stage_at(row + i, c), src + (uint64_t)(uint32_t)max(n[i], 0) * C, n[i] >= 0);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    look_up();
    note();
    later.next_item();
    look_up();
    note();
    later.next_item();
    __syncthreads();
    fetch(ahead, 0);
    ahead.next();
    // An item's tokens are looked up while the first tile of the item before the one before it is
    // quantised, and noted at that tile's end: a barrier before the first copy that needs them, and after
    // the last use of the three items older ones in that place.
    for (int buf = 0; at.live(); at.next(), buf ^= 1) {
        const uint32_t cb = at.cb, g = at.g;
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();   // this tile has landed, and the other buffer is free
        fetch(ahead, buf ^ 1);
        ahead.next();
        if (at.at_first()) look_up();

        const uint8_t* tile = smem + buf * kStageBytes;
        const float* weights_of = s_weight + 128 * at.slot;
        float* scales = st + (uint64_t)g * C + cb * 128 + 16 * w;
        uint8_t* codes = qt + (int64_t)(cb * 128 + 16 * w) * Kcap + (int64_t)g * 128;
        if (s_rows[at.slot] > 64)
            quantise_columns<WEIGHTED, 8>(tile, weights_of, w, lane, scales, codes, Kcap);
        else
            quantise_columns<WEIGHTED, 4>(tile, weights_of, w, lane, scales, codes, Kcap);
        if (at.at_first()) {
            note();
            later.next_item();
        }
    }
}

// ------------------------------------------------------------------------------------------
// Combine: out[t] = add[t] + sum_j w[t,j] y[rows[t,j]], summed in FP32 in the order of j and rounded
// once.  A slot of weight zero is not read.  A CTA takes 1024 channels of one token, a thread 8 of them;
// the loads of eight rows are in flight together.
// Bound by HBM: 65536 rows of 7168 channels to 8192 tokens, with an addend, take 179 us, 6.55 TB/s (198 us
// with one row's load after another).
// ------------------------------------------------------------------------------------------
__device__ __forceinline__ void fma8(float (&acc)[8], float w, const uint4& u)
{
    const uint32_t p[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        acc[2 * i] = fmaf(w, bf16_lo(p[i]), acc[2 * i]);
        acc[2 * i + 1] = fmaf(w, bf16_hi(p[i]), acc[2 * i + 1]);
    }
}

constexpr int kCombineThreads = 128;

__global__ void __launch_bounds__(kCombineThreads) moe_combine_kernel(
    const uint16_t* __restrict__ y, const int32_t* __restrict__ rows, const float* __restrict__ weights,
    const uint16_t* __restrict__ add, uint32_t T, uint32_t k, uint32_t C, uint16_t* __restrict__ out)
{
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t units = C >> 3, chunks = (units + kCombineThreads - 1) / kCombineThreads, items = T * chunks;
    const int32_t M = (int32_t)(T * k);
    for (uint32_t it = blockIdx.x; it < items; it += gridDim.x) {
        const uint32_t t = it / chunks, u = (it - t * chunks) * kCombineThreads + threadIdx.x;
        if (u >= units) continue;
        float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        for (uint32_t j0 = 0; j0 < k; j0 += 8) {
            float w[8];
            uint4 v[8];
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) {
                w[j] = 0.0f;
                v[j] = make_uint4(0u, 0u, 0u, 0u);
                if (j0 + j < k) {
                    w[j] = weights ? __ldg(weights + t * k + j0 + j) : 1.0f;
                    const int32_t r = __ldg(rows + t * k + j0 + j);
                    if (r < 0 || r >= M) {
                        if (w[j] != 0.0f) latch_status(kDevBadIndex);
                        w[j] = 0.0f;
                    }
                    if (w[j] != 0.0f) v[j] = __ldg(reinterpret_cast<const uint4*>(y + (size_t)r * C) + u);
                }
            }
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j)
                if (w[j] != 0.0f) fma8(acc, w[j], v[j]);
        }
        if (add) fma8(acc, 1.0f, __ldg(reinterpret_cast<const uint4*>(add + (size_t)t * C) + u));
        reinterpret_cast<uint4*>(out + (size_t)t * C)[u] =
            make_uint4(bf16_rn(acc[0]) | (bf16_rn(acc[1]) << 16), bf16_rn(acc[2]) | (bf16_rn(acc[3]) << 16),
                       bf16_rn(acc[4]) | (bf16_rn(acc[5]) << 16), bf16_rn(acc[6]) | (bf16_rn(acc[7]) << 16));
    }
}

// dw[t,j] = <dout[t], y[rows[t,j]]>: one warp per slot, eight FP32 partial sums a lane.  Bound by HBM:
// 65536 rows of 7168 channels take 168 us, 6.3 TB/s.
__global__ void __launch_bounds__(256) moe_combine_dweight_kernel(const uint16_t* __restrict__ dout,
                                                                  const uint16_t* __restrict__ y,
                                                                  const int32_t* __restrict__ rows, int64_t T, int k,
                                                                  int64_t C, float* __restrict__ dw)
{
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t M = T * k;
    const int64_t slot = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (slot >= M) return;
    const int32_t r = rows[slot];
    if (r < 0 || r >= M) {
        if (lane == 0) {
            latch_status(kDevBadIndex);
            dw[slot] = 0.0f;
        }
        return;
    }
    const uint4* a = reinterpret_cast<const uint4*>(dout + (slot / k) * C);
    const uint4* b = reinterpret_cast<const uint4*>(y + (int64_t)r * C);
    float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t u = lane; u < (C >> 3); u += 32) {
        const uint4 p = __ldg(a + u), z = __ldg(b + u);
        const uint32_t pu[4] = {p.x, p.y, p.z, p.w}, zu[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            acc[2 * i] = fmaf(bf16_lo(pu[i]), bf16_lo(zu[i]), acc[2 * i]);
            acc[2 * i + 1] = fmaf(bf16_hi(pu[i]), bf16_hi(zu[i]), acc[2 * i + 1]);
        }
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += acc[i];
    sum = warp_sum(sum);
    if (lane == 0) dw[slot] = sum;
}

// ------------------------------------------------------------------------------------------
// SwiGLU: a = silu(g) u with g = h[:, :I], u = h[:, I:], quantised from FP32; with `hq`, the 1x128
// codes of h itself are the checkpoint that the backward pass starts from.  Eight lanes own one
// 128-element tile of a (and the two tiles of h that it comes from), a warp four neighbouring tiles of
// `rows` rows, one row after another, the next one's loads in flight: with eight rows, the scales of a
// tile column leave as whole 32-byte sectors.  One lane of the eight forms each of the three scales.
// Bound by HBM: 65536 x 2048 with the checkpoint takes 158 us, 6.0 TB/s (the two MUFU operations an
// element alone would take 60 us).  Two CTAs an SM with 110 registers; three with 80 spill: 176 us.
// ------------------------------------------------------------------------------------------
// sigmoid of two values by ex2 and a fast reciprocal.  In units of 2^-24 of the result: 1.25 |x| from x log2 e and its
// rounding, 3 and 2 from the two functions, 1 from the sum: below 8 + 1.5 |x|.  Results below 2^-126 are 0.
__device__ __forceinline__ float2 sigmoid2(float2 x)
{
    const float2 t = mul2(x, both(-1.442695041f));   // -log2 e
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
    e = add2(e, both(1.0f));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.y));
    return e;
}

template <bool CKPT>
__global__ void __launch_bounds__(256, 2) swiglu_quant_kernel(const uint16_t* __restrict__ h, uint32_t M, uint32_t I,
                                                              uint32_t rows, uint8_t* __restrict__ q,
                                                              float* __restrict__ s, uint8_t* __restrict__ hq,
                                                              float* __restrict__ hs)
{
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t IB = I >> 7, quads = (IB + 3) >> 2, bands = (M + rows - 1) / rows, items = bands * quads;
    const uint32_t lane = threadIdx.x & 31, sub = lane & 7;
    const uint32_t warps = (gridDim.x * blockDim.x) >> 5;
    for (uint32_t it = (blockIdx.x * blockDim.x + threadIdx.x) >> 5; it < items; it += warps) {
        const uint32_t band = it / quads, ib = (it - band * quads) * 4 + (lane >> 3);
        const bool live = ib < IB;
        const uint32_t m0 = band * rows, n = min(rows, M - m0);
        const uint16_t* src = h + (size_t)m0 * 2 * I + ib * 128 + 16 * sub;
        uint8_t* qa = q + (size_t)m0 * I + ib * 128 + 16 * sub;
        uint8_t* qh = CKPT ? hq + (size_t)m0 * 2 * I + ib * 128 + 16 * sub : nullptr;
        float sa = 0.0f, sg = 0.0f, su = 0.0f;   // lane sub: the scales of row m0 + sub
        uint4 g0 = make_uint4(0u, 0u, 0u, 0u), g1 = g0, u0 = g0, u1 = g0;
        if (live) {
            g0 = __ldg(reinterpret_cast<const uint4*>(src));
            g1 = __ldg(reinterpret_cast<const uint4*>(src) + 1);
            u0 = __ldg(reinterpret_cast<const uint4*>(src + I));
            u1 = __ldg(reinterpret_cast<const uint4*>(src + I) + 1);
        }
        uint4 h0 = g0, h1 = g0, v0 = g0, v1 = g0;   // the next row's, loaded while this one is worked on
        for (uint32_t i = 0; i < n; ++i, qa += I, qh += CKPT ? 2 * I : 0, g0 = h0, g1 = h1, u0 = v0, u1 = v1) {
            src += 2 * I;
            if (live && i + 1 < n) {
                h0 = __ldg(reinterpret_cast<const uint4*>(src));
                h1 = __ldg(reinterpret_cast<const uint4*>(src) + 1);
                v0 = __ldg(reinterpret_cast<const uint4*>(src + I));
                v1 = __ldg(reinterpret_cast<const uint4*>(src + I) + 1);
            }
            float a[16];
            const uint32_t gw[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
            const uint32_t uw[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 g = widen(gw[j]), v = mul2(mul2(g, sigmoid2(g)), widen(uw[j]));
                a[2 * j] = v.x;
                a[2 * j + 1] = v.y;
            }
            const float ma = max8(amax16f(a));
            float inv_a, inv_g = 0.0f, inv_u = 0.0f;
            if (CKPT) {
                const float mg = max8(amax16(g0, g1)), mu = max8(amax16(u0, u1));
                float sc, inv;
                group_scale<false>(sub == 0 ? ma : sub == 1 ? mg : mu, sc, inv);
                inv_a = __shfl_sync(kFull, inv, 0, 8);
                inv_g = __shfl_sync(kFull, inv, 1, 8);
                inv_u = __shfl_sync(kFull, inv, 2, 8);
                const float ka = __shfl_sync(kFull, sc, 0, 8), kg = __shfl_sync(kFull, sc, 1, 8),
                            ku = __shfl_sync(kFull, sc, 2, 8);
                if (sub == i) {
                    sa = ka;
                    sg = kg;
                    su = ku;
                }
            } else {
                float sc;
                group_scale<false>(ma, sc, inv_a);
                if (sub == i) sa = sc;
            }
            if (live) {
                *reinterpret_cast<uint4*>(qa) = quant16f(a, inv_a);
                if (CKPT) {
                    const uint2 p = quant8(g0, inv_g), r = quant8(g1, inv_g), v = quant8(u0, inv_u), z = quant8(u1, inv_u);
                    *reinterpret_cast<uint4*>(qh) = make_uint4(p.x, p.y, r.x, r.y);
                    *reinterpret_cast<uint4*>(qh + I) = make_uint4(v.x, v.y, z.x, z.y);
                }
            }
        }
        if (live && sub < n) {
            s[(size_t)ib * M + m0 + sub] = sa;
            if (CKPT) {
                hs[(size_t)ib * M + m0 + sub] = sg;
                hs[(size_t)(IB + ib) * M + m0 + sub] = su;
            }
        }
    }
}

// ------------------------------------------------------------------------------------------
// SwiGLU backward from the checkpoint h^ = code * scale, r = sigmoid(g):
//   dg = da u r (1 + g (1 - r)),   du = da g r,   a = g r u
// Outputs: dh = [dg, du] in both forms (Dgrad's and Wgrad's operand) and a in the 128x1 form (the
// second GEMM's Wgrad operand), so a is never kept between the passes.
// One CTA of 16 warps takes tiles of one padded group (128 rows) x 128 columns of I, whose inputs come
// into shared memory by asynchronous copies while the tile before is worked on.  Warp w owns columns
// 8w .. 8w+7, its lane r rows 4r .. 4r+3 (2r, 2r+1 in a group of at most 64 rows: 2000 rows over 256 experts
// take 86 us instead of 101): the 96 values, three an element, are computed once and stay in
// registers until both quantisations are done.  Columns lie inside a warp, so their scales need shuffles
// only and their codes leave as whole lines; rows meet in shared memory.
// The values fill the register file with one CTA an SM, four warps a scheduler, and what bounds it is that these
// are too few: 0.57 of the issue slots and no pipe above 0.42 (ALU; FMA 0.34, MUFU and conversions 0.23) in use, and of
// the 7.0 cycles between two instructions of a warp 0.9 at barriers, 0.9 in fixed latencies, 0.8 behind another
// warp in a pipe, 0.75 for shared memory and MUFU results.  65536 x 2048 in 645 groups take 300 us, 4.1 TB/s.
// ------------------------------------------------------------------------------------------
constexpr int kBackThreads = 512;
constexpr int kBackStage = 128 * 256 + 2 * 128 * 128 + 2 * 128 * 4;   // da, the codes of g and u, their scales
struct BackSmem {   // byte offsets
    static constexpr int codes = 2 * kBackStage;              // row codes of dg and du: [2][128][128]
    static constexpr int red = codes + 2 * 128 * 128;         // [2][16 warps][128 rows]
    static constexpr int inv_row = red + 2 * 16 * 128 * 4;    // [2][128]
    static constexpr int inv_col = inv_row + 2 * 128 * 4;     // [16 warps][24], 32 apart
    static constexpr int place = inv_col + 16 * 32 * 4;       // [4] int4
    static constexpr int table = place + 64;
};
constexpr int back_smem(int E) { return BackSmem::table + group_table_bytes(E); }

__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool live)   // zero unless live
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(live ? 4 : 0) : "memory");
}

// The values of four E4M3 codes; fp16 is widened by a mixed-precision x + (-0), as bf16 in widen().
__device__ __forceinline__ void dec_e4m3x4(uint32_t w, float2 (&f)[2])
{
    asm("{.reg .b16 c0, c1, l, h;\n\t"
        ".reg .b32 p;\n\t"
        "mov.b32 {c0, c1}, %4;\n\t"
        "cvt.rn.f16x2.e4m3x2 p, c0;\n\t"
        "mov.b32 {l, h}, p;\n\t"
        "add.f32.f16 %0, l, %5;\n\t"
        "add.f32.f16 %1, h, %5;\n\t"
        "cvt.rn.f16x2.e4m3x2 p, c1;\n\t"
        "mov.b32 {l, h}, p;\n\t"
        "add.f32.f16 %2, l, %5;\n\t"
        "add.f32.f16 %3, h, %5;}"
        : "=f"(f[0].x), "=f"(f[0].y), "=f"(f[1].x), "=f"(f[1].y)
        : "r"(w), "f"(-0.0f));
}

// max |.| over the warp's 32 lanes of eight values each: lane l ends with that of value l & 7.
__device__ __forceinline__ float max_of_eight(float (&m)[8], int lane)
{
#pragma unroll
    for (int h = 4; h >= 1; h >>= 1) {
        const bool up = lane & h;
#pragma unroll
        for (int i = 0; i < h; ++i) {
            const float send = up ? m[i] : m[i + h], keep = up ? m[i + h] : m[i];
            m[i] = fmaxf(keep, __shfl_xor_sync(kFull, send, h));
        }
    }
    m[0] = fmaxf(m[0], __shfl_xor_sync(kFull, m[0], 8));
    return fmaxf(m[0], __shfl_xor_sync(kFull, m[0], 16));
}

__global__ void __launch_bounds__(kBackThreads, 1) swiglu_backward_kernel(
    const uint16_t* __restrict__ da, const uint8_t* __restrict__ hq, const float* __restrict__ hs,
    const int32_t* __restrict__ offsets, int E, int64_t M, uint32_t I, uint8_t* __restrict__ q, float* __restrict__ s,
    uint8_t* __restrict__ qt, float* __restrict__ st, uint8_t* __restrict__ aqt, float* __restrict__ ast, int64_t Kcap)
{
    griddep_launch_dependents();
    griddep_wait();
    extern __shared__ __align__(16) uint8_t smem[];
    const GroupTable table(smem + BackSmem::table, E);
    if (!group_table(table, offsets, E, M, Kcap)) return;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const uint32_t base = smem_u32(smem);
    const uint32_t IB = I >> 7, groups = table.pre[E], tiles = groups * IB;
    float* red = reinterpret_cast<float*>(smem + BackSmem::red);
    float* inv_row = reinterpret_cast<float*>(smem + BackSmem::inv_row);
    float* inv_col = reinterpret_cast<float*>(smem + BackSmem::inv_col) + 32 * w;

    // A tile's place, looked up by one warp two tiles ahead: first row, rows, group, column block.
    int4* place = reinterpret_cast<int4*>(smem + BackSmem::place);
    auto look_up = [&](uint32_t tile, int slot) {
        if (w == kBackThreads / 32 - 1 && tile < tiles) {
            const uint32_t ib = tile / groups, g = tile - ib * groups;
            int64_t r0;
            int nvalid;
            group_rows(table, E, (int)g, r0, nvalid);
            if (lane == 0) place[slot] = make_int4((int)r0, nvalid, (int)g, (int)ib);
        }
    };
    // Copies of a tile's inputs.  16-byte piece c of a row's 256 (da) or 128 bytes (codes) lies at piece
    // c ^ ((row >> 2) & 7): eight neighbouring lanes then read different banks.
    auto fetch = [&](uint32_t tile, int slot, int buf) {
        if (tile < tiles) {
            const int4 at = place[slot];
            const uint32_t dst = base + buf * kBackStage;
            {
                const int row = tid >> 4, c = tid & 15;
                const uint16_t* src = da + (int64_t)at.x * I + at.w * 128 + 8 * c;
                const uint32_t to = dst + row * 256 + ((c ^ ((row >> 2) & 7)) << 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {   // rows 32 apart: the same swizzle
                    const bool live = row + 32 * i < at.y;
                    copy16(to + i * 32 * 256, src + (uint64_t)(live ? (uint32_t)(row + 32 * i) : 0u) * I, live);
                }
            }
            {
                const int row = tid >> 3, c = tid & 7;
                const uint8_t* src = hq + (int64_t)at.x * 2 * I + at.w * 128 + 16 * c;
                const uint32_t to = dst + 32768 + row * 128 + ((c ^ ((row >> 2) & 7)) << 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool live = row + 64 * (i & 1) < at.y;
                    copy16(to + 16384 * (i >> 1) + 64 * 128 * (i & 1),
                           src + (uint64_t)(live ? (uint32_t)(row + 64 * (i & 1)) : 0u) * (2 * I) + (i >> 1) * I, live);
                }
            }
            if (tid < 256) {
                const int row = tid & 127;
                const bool live = row < at.y;
                copy4(dst + 65536 + 4 * tid, hs + (int64_t)((tid >> 7) * IB + at.w) * M + at.x + (live ? row : 0), live);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    // The staged row codes of a tile (below) as whole lines.
    auto store_rows = [&](const int4& at) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int v = i >> 1, row = (tid >> 3) + 64 * (i & 1), c = tid & 7, f = (row >> 2) & 15;
            const uint4 u = *reinterpret_cast<const uint4*>(smem + BackSmem::codes + v * 16384 + row * 128 + (((2 * c) ^ (f & 14)) << 3));
            if (row < at.y)
                *reinterpret_cast<uint4*>(q + (int64_t)(at.x + row) * 2 * I + v * I + at.w * 128 + 16 * c) =
                    (f & 1) ? make_uint4(u.z, u.w, u.x, u.y) : u;
        }
    };

    look_up(blockIdx.x, 0);
    look_up(blockIdx.x + gridDim.x, 1);
    __syncthreads();
    fetch(blockIdx.x, 0, 0);
    int buf = 0, slot = 0;   // slot: the tile's number modulo 4
    for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1, slot = (slot + 1) & 3) {
        const int4 at = place[slot];
        const int64_t r0 = at.x;
        const int nvalid = at.y, g = at.z, ib = at.w;
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();   // this tile has landed; the tile before is done with the other buffer
        fetch(tile + gridDim.x, (slot + 1) & 3, buf ^ 1);
        look_up(tile + 2 * gridDim.x, (slot + 2) & 3);
        if (tile != blockIdx.x) store_rows(place[(slot + 3) & 3]);   // the tile before's

        const uint8_t* in = smem + buf * kBackStage;
        const auto work = [&](auto rows_of_a_lane) {
            constexpr int R = decltype(rows_of_a_lane)::value;
            float2 dg[R][4], du[R][4], ac[R][4];   // [row][pair of columns]
            float rg[R], ru[R];                    // row maxima of dg and du
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int row = R * lane + i, turn = (row >> 2) & 7;
                const uint8_t* code = in + 32768 + row * 128 + (((w >> 1) ^ turn) << 4) + 8 * (w & 1);
                const uint4 dw = *reinterpret_cast<const uint4*>(in + row * 256 + ((w ^ turn) << 4));
                const uint2 gc = *reinterpret_cast<const uint2*>(code);
                const uint2 uc = *reinterpret_cast<const uint2*>(code + 16384);
                const float gs = *reinterpret_cast<const float*>(in + 65536 + 4 * row);
                const float us = *reinterpret_cast<const float*>(in + 65536 + 512 + 4 * row);
                rg[i] = ru[i] = 0.0f;
                float2 gf[4], uf[4];
                dec_e4m3x4(gc.x, reinterpret_cast<float2 (&)[2]>(gf[0]));
                dec_e4m3x4(gc.y, reinterpret_cast<float2 (&)[2]>(gf[2]));
                dec_e4m3x4(uc.x, reinterpret_cast<float2 (&)[2]>(uf[0]));
                dec_e4m3x4(uc.y, reinterpret_cast<float2 (&)[2]>(uf[2]));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 d = widen(word(dw, j)), x = mul2(gf[j], both(gs)), u = mul2(uf[j], both(us));
                    const float2 r = sigmoid2(x), sx = mul2(x, r);
                    // r + sx (1 - r)
                    dg[i][j] = mul2(mul2(d, u), fma2(sx, fma2(r, both(-1.0f), both(1.0f)), r));
                    du[i][j] = mul2(d, sx);
                    ac[i][j] = mul2(u, sx);
                    rg[i] = max_abs(rg[i], dg[i][j].x, dg[i][j].y);
                    ru[i] = max_abs(ru[i], du[i][j].x, du[i][j].y);
                }
            }
#pragma unroll
            for (int i = 0; i < R; i += 2) {
                *reinterpret_cast<float2*>(red + w * 128 + R * lane + i) = make_float2(rg[i], rg[i + 1]);
                *reinterpret_cast<float2*>(red + 2048 + w * 128 + R * lane + i) = make_float2(ru[i], ru[i + 1]);
            }
            __syncthreads();
            if (tid < 256) {   // the row scales: thread (dg or du, row); rows from nvalid on hold anything
                const int row = tid & 127;
                const float* p = red + (tid >> 7) * 2048 + row;
                float m = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; i += 2) m = fmaxf(fmaxf(m, p[128 * i]), p[128 * i + 128]);
                float sc, inv;
                group_scale<false>(m, sc, inv);
                inv_row[tid] = inv;
                if (row < nvalid) s[(int64_t)((tid >> 7) * IB + ib) * M + r0 + row] = sc;
            }
            // Columns.  Lanes 8v + c: the scale of column c of value v (dg, du, a).
            auto column_max = [&](const float2 (&x)[R][4]) {
                float m[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    m[2 * j] = m[2 * j + 1] = 0.0f;
#pragma unroll
                    for (int i = 0; i < R; i += 2) {
                        m[2 * j] = max_abs(m[2 * j], x[i][j].x, x[i + 1][j].x);
                        m[2 * j + 1] = max_abs(m[2 * j + 1], x[i][j].y, x[i + 1][j].y);
                    }
                }
                return max_of_eight(m, lane);
            };
            {
                const float m0 = column_max(dg), m1 = column_max(du), m2 = column_max(ac);
                const int v = lane >> 3;
                float sc, inv;
                group_scale<false>(v == 0 ? m0 : v == 1 ? m1 : m2, sc, inv);
                const uint32_t col = ib * 128 + 8 * w + (lane & 7);
                if (v < 2) st[(int64_t)g * 2 * I + v * I + col] = sc;
                if (v == 2) ast[(int64_t)g * I + col] = sc;
                if (v < 3) inv_col[lane] = inv;
            }
            __syncwarp();
            const int64_t corner = (int64_t)(ib * 128 + 8 * w) * Kcap + (int64_t)g * 128 + R * lane;
            auto columns = [&](const float2 (&x)[R][4], const float* inv, uint8_t* out) {
                const float4 i0 = *reinterpret_cast<const float4*>(inv), i1 = *reinterpret_cast<const float4*>(inv + 4);
                const float2 f[4] = {{i0.x, i0.y}, {i0.z, i0.w}, {i1.x, i1.y}, {i1.z, i1.w}};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint8_t* even = out + (uint64_t)(2 * j) * (uint32_t)Kcap;
                    uint8_t* odd = out + (uint64_t)(2 * j + 1) * (uint32_t)Kcap;
                    const float2 a = mul2(x[0][j], f[j]), b = mul2(x[1][j], f[j]);
                    if (R == 4) {
                        const float2 c = mul2(x[R - 2][j], f[j]), d = mul2(x[R - 1][j], f[j]);
                        *reinterpret_cast<uint32_t*>(even) = codes4(a.x, b.x, c.x, d.x);
                        *reinterpret_cast<uint32_t*>(odd) = codes4(a.y, b.y, c.y, d.y);
                    } else {   // rows 64 .. 127 are padding
                        *reinterpret_cast<uint16_t*>(even) = (uint16_t)e4m3x2(a.x, b.x);
                        *reinterpret_cast<uint16_t*>(odd) = (uint16_t)e4m3x2(a.y, b.y);
                        *reinterpret_cast<uint16_t*>(even + 64) = 0;
                        *reinterpret_cast<uint16_t*>(odd + 64) = 0;
                    }
                }
            };
            columns(ac, inv_col + 16, aqt + corner);
            columns(dg, inv_col, qt + corner);
            columns(du, inv_col + 8, qt + (int64_t)I * Kcap + corner);
            __syncthreads();
            // Rows: 8 bytes of a row from each warp, staged (8-byte unit w of row r at w ^ ((r >> 2) & 15)); they
            // are written behind the next tile's first barrier.
            auto stage_rows = [&](const float2 (&x)[R][4], const float* inv, uint8_t* to) {
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const int row = R * lane + i;
                    const float2 f = both(inv[row]);
                    const float2 a = mul2(x[i][0], f), b = mul2(x[i][1], f), c = mul2(x[i][2], f), d = mul2(x[i][3], f);
                    *reinterpret_cast<uint2*>(to + row * 128 + ((w ^ ((row >> 2) & 15)) << 3)) =
                        make_uint2(codes4(a.x, a.y, b.x, b.y), codes4(c.x, c.y, d.x, d.y));
                }
            };
            stage_rows(dg, inv_row, smem + BackSmem::codes);
            stage_rows(du, inv_row + 128, smem + BackSmem::codes + 16384);
        };
        if (nvalid > 64)
            work(std::integral_constant<int, 4>());
        else
            work(std::integral_constant<int, 2>());
    }
    __syncthreads();
    if (blockIdx.x < tiles) store_rows(place[(slot + 3) & 3]);
}

}  // namespace fp8q
