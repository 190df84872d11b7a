// route_scored.cuh - the router's selection with sigmoid or softmax scores, a balancing bias on the
// scores, expert groups and scaled weights.
//
// Per token, from fp32 logits l_e:
//   s_e   = 1 / (1 + e^-l_e)  (sigmoid)   or   e^(l_e - max l) / sum e^(l - max l)  (softmax)
//   key_e = s_e + bias_e; an expert whose logit or bias is -inf is masked (key -inf)
//   groups of E / n_group consecutive experts; a group's value is its largest key, or the sum of its
//   two largest unmasked keys; the topk_group groups of largest value stay (ties -> lower group)
//   slots = the k largest keys of the groups that stay, descending (ties -> lower expert)
//   w_j   = scale * s_idx_j, divided by the sum of the k selected scores when renormalising
// A slot that no unmasked expert is left for holds expert -1 and weight 0, which the permutation
// drops; a row of -inf (a padded token) is k such slots.
//
// Keys are compared as if computed in 64 bits: two scores that differ by less than a 32-bit rounding
// still have a defined order.  Without a bias, and with groups valued by their best expert, the order
// of the keys is the order of the logits, which are compared themselves.
#pragma once

#include <cfloat>
#include <type_traits>

#include "route_permute_combine.cuh"

namespace moe {

constexpr int ROUTE_MAX_GROUPS = 32;

struct RouteScored {
    const float* logits;      // [T, E], or nsplit partial sums [nsplit][T][E]
    int nsplit;
    long long split_stride;   // floats between two partial sums
    float* logits_out;        // receives the sums when nsplit > 1 (nullable)
    const float* bias;        // [E], nullable
    int T, E, k;
    int sigmoid;              // 1: sigmoid scores, 0: softmax
    int n_group, topk_group, top2, renorm;
    float scale;
    int by_logit;             // keys ordered as the logits are: compare those
    int32_t* idx;             // [T, k]
    float* w;                 // [T, k]
};

// The logit of expert e: the partial sums added in slice order, as moe_route adds them.
__device__ __forceinline__ float scored_logit(const RouteScored& p, const float* row, int e) {
    float l = __ldg(row + e);
    for (int s = 1; s < p.nsplit; ++s) l = __fadd_rn(l, __ldg(row + s * p.split_stride + e));
    return l;
}

// floats as integers of the same order (no NaN; -0 must have been made +0)
__device__ __forceinline__ int ordered(float f) {
    const int b = __float_as_int(f);
    return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float from_ordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }
constexpr int ORD_LOWEST = (int)0x80800000;    // ordered(-FLT_MAX): every unmasked key is at least this
constexpr int ORD_EMPTY = (int)0x80000000;

// e^x, subnormal results as 0
__device__ __forceinline__ float exp_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
    return r;
}

// Over the LPT lanes of a token (32: the warp; 16: each half of it for itself): the largest, the sum, a ballot.
template <int LPT>
__device__ __forceinline__ int lanes_max(int v) {
    if constexpr (LPT == 32) {
        return __reduce_max_sync(0xffffffffu, v);
    } else {
#pragma unroll
        for (int o = LPT / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
        return v;
    }
}
template <int LPT>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int LPT>
__device__ __forceinline__ unsigned lanes_ballot(bool v) {
    const unsigned b = __ballot_sync(0xffffffffu, v);
    return LPT == 32 ? b : (threadIdx.x & 16 ? b >> 16 : b & 0xffffu);
}

// The weights of the selected experts: lane j < k holds slot j's expert (-1: none) and logit.
// top / total: the row's largest logit and sum of e^(l - top) over its finite logits, those of experts that the bias
// masks among them (softmax without renormalisation).  Renormalised weights are ratios of scores, which are taken
// relative to the largest selected one where that is small, so that no score underflows before its ratio does:
// s_j ~ e^(l_j - m) in softmax; s_j ~ e^(min(l_j, 0) - min(m, 0)) / (1 + e^-|l_j|) in sigmoid.  That exponential is within 2
// ulp of its rounded argument, and the fast one behind the 1 adds 2 more at most (its error is (2 + 1.2 |l|) 2^-23 of
// e^-|l|).  LPT lanes per token, `lane` among them; warp-collective, writing where `live`.
template <int LPT>
__device__ __forceinline__ void scored_weights(const RouteScored& p, long long t, bool live, int lane, int my_e,
                                               float my_l, float top, float total) {
    const bool have = lane < p.k && my_e >= 0;
    float s = 0.0f;
    if (!p.sigmoid) {
        if (p.renorm) {      // as moe_route computes them: the same weights, bit for bit
            const float m = from_ordered(lanes_max<LPT>(ordered((have ? my_l : -INFINITY) + 0.0f)));
            if (have) s = expf(my_l - m);
            s /= lanes_sum<LPT>(s);
        } else if (have) {
            s = expf(my_l - top) / total;
        }
    } else {
        float m = 0.0f;
        if (p.renorm) m = fminf(from_ordered(lanes_max<LPT>(ordered(have ? my_l : -INFINITY))), 0.0f);
        if (have) s = expf(fminf(my_l, 0.0f) - m) * rcp_approx(1.0f + exp_approx(-fabsf(my_l)));
        if (p.renorm) s *= rcp_approx(lanes_sum<LPT>(s));
    }
    if (live && lane < p.k) {
        p.idx[t * p.k + lane] = have ? my_e : -1;
        p.w[t * p.k + lane] = have ? s * p.scale : 0.0f;
    }
}

// Experts of a token's lanes (a warp, or half of one): group g on 2^lg lanes, each holding up to `per` consecutive
// experts (the last lanes of a group fewer), so that (lane, position) is the order of the experts.
struct RouteLanes {
    int lg, per;
    int each;     // E / n_group
};
struct RouteLane {
    int group, e0, cnt;
    __device__ __forceinline__ RouteLane(const RouteScored& p, const RouteLanes& m, int lane) {
        const int part = lane & ((1 << m.lg) - 1);
        group = lane >> m.lg;
        e0 = group * m.each + part * m.per;
        cnt = group < p.n_group ? max(0, min(m.per, m.each - part * m.per)) : 0;
    }
};

// doubles as integers of the same order (no NaN, no -0)
__device__ __forceinline__ long long ordered64(double d) {
    const long long b = __double_as_longlong(d);
    return b ^ ((b >> 63) & 0x7fffffffffffffffll);
}

// One token by one warp with every key in 64 bits, in the caller's shared memory (32 `per` doubles, expert i of
// lane q at [32 i + q]).  Experts whose logit or bias is NaN or +inf are masked (the caller has reported them).
__device__ __noinline__ void route_token_f64(const RouteScored& p, const RouteLanes& m, long long t, int lane,
                                             double* keys) {
    const unsigned all = 0xffffffffu;
    const float* row = p.logits + t * p.E;
    const RouteLane at(p, m, lane);
    float top = -INFINITY;
    double total = 0.0;
    if (!p.sigmoid) {
        for (int i = 0; i < at.cnt; ++i) {
            const float l = scored_logit(p, row, at.e0 + i);
            if (l < INFINITY) top = fmaxf(top, l);
        }
        top = warp_max(top);
#pragma unroll 4
        for (int i = 0; i < at.cnt; ++i) {
            const float l = scored_logit(p, row, at.e0 + i);
            total += l < INFINITY && l > -INFINITY ? exp((double)l - (double)top) : 0.0;
        }
        total = warp_sum(total);
    }
    double a = -INFINITY, b = -INFINITY;          // the lane's two largest keys
    int best = 0;                                 // position of a
#pragma unroll 4
    for (int i = 0; i < at.cnt; ++i) {
        const float l = scored_logit(p, row, at.e0 + i), bias = p.bias ? __ldg(p.bias + at.e0 + i) : 0.0f;
        double key = l;
        if (!p.by_logit)
            key = (p.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)top) / total) + (double)bias;
        if (!(l < INFINITY && l > -INFINITY && bias < INFINITY && bias > -INFINITY)) key = -INFINITY;
        key += 0.0;                               // -0 -> +0
        keys[32 * i + lane] = key;
        if (key > a) {
            b = a;
            a = key;
            best = i;
        } else if (key > b) {
            b = key;
        }
    }
    if (p.n_group > 1) {
        double v = a, w = b;
        for (int o = 1; o < (1 << m.lg); o <<= 1) {
            const double v2 = __shfl_xor_sync(all, v, o), w2 = __shfl_xor_sync(all, w, o);
            w = fmax(fmax(w, w2), fmin(v, v2));
            v = fmax(v, v2);
        }
        if (p.top2 && w > -INFINITY) v += w;
        int rank = 0;
        for (int q = 0; q < p.n_group; ++q) {
            const double o = __shfl_sync(all, v, q << m.lg);
            rank += o > v || (o == v && q < at.group);
        }
        if (at.group >= p.n_group || rank >= p.topk_group) a = -INFINITY;
    }
    int my_e = -1;
    for (int j = 0; j < p.k; ++j) {
        // the largest head, the lowest lane of equal ones
        const long long o = ordered64(a);
        const int hi = (int)(o >> 32);
        const bool first = hi == __reduce_max_sync(all, hi);
        const unsigned lo = (unsigned)o;
        const unsigned most = __reduce_max_sync(all, first ? lo : 0u);
        const int owner = __ffs(__ballot_sync(all, first && lo == most)) - 1;
        if (!(__shfl_sync(all, a, owner) > -INFINITY)) break;      // no unmasked expert left
        const int e = __shfl_sync(all, at.e0 + best, owner);
        if (lane == j) my_e = e;
        if (lane == owner) {
            keys[32 * best + lane] = -INFINITY;
            a = -INFINITY;
#pragma unroll 4
            for (int i = 0; i < at.cnt; ++i) {
                const double key = keys[32 * i + lane];
                if (key > a) {
                    a = key;
                    best = i;
                }
            }
        }
    }
    const float my_l = my_e >= 0 ? scored_logit(p, row, my_e) : 0.0f;
    scored_weights<32>(p, t, true, lane, my_e, my_l, top, (float)total);
}

// ---------------------------------------------------------------- the kernel: keys in 32 bits
//
// One warp per token, or two tokens per warp, the experts on the lanes as RouteLanes has them, EPL >= per.
// Keys are integers of the floats' order whose last BITS bits hold the position in the lane: a comparison carries the expert along and a lane's keys are distinct.
//   lanes       sort their four largest keys (8 experts: 32 minima and maxima)
//   groups      the two largest keys merged over the group's lanes; the topk_group largest of them, one by one
//   slots       k + 1 times: the largest list head, taken off its lane's list; a lane whose four are used up sorts its
//               next four
//   certainty   keys are off by at most route_err and 2^BITS steps.  Neighbours in the order that are closer than that
//               are put in order by 64-bit keys of the slots alone (one token in 400 for scores of unit variance, 256
//               experts); where it is the last slot and the key after it, or the last group that stays and the first
//               that does not, the token is done again in 64 bits (route_token_f64: one in some thousands)
// Bound by what a token's steps wait for, not by the 33.5 MB of logits (5.2 us at the measured copy rate), nor by the
// instruction rate alone: 32768 tokens of 256 experts in 8 groups take 36 us, their 18.3 M warp instructions (557 a token) 16
// at one per cycle.  Each round of the groups and of the slots is a maximum over the lanes, a ballot and a shift, every one of
// which needs the one before it.  At 24 warps per SM an instruction issues in 59 % of the cycles; per issue, warps wait 2.2
// cycles for shuffles and the special functions, 2.2 for fixed latencies, 1.2 for memory, 0.8 for the integer pipe, which half
// of the instructions use.  A few thousand tokens are one per warp: one token's latency (4099 x 160: 7.8 us).
// 39 of the 48 kernels keep 4 to 172 bytes per thread on the stack under the launch bounds below, where more blocks with fewer
// registers gave nothing or lost 8 %.
constexpr int ROUTE_WARPS = 8;

// Errors in units of 2^-23.  The fast exponential of x is off by at most 2 + 1.16 |x| of its value (x = -l, or
// l - top in softmax, whose rounding adds |x| / 2), the fast reciprocal by 1, a rounding by 1/2.
//   sigmoid  the exponential's part reaches s by the factor 1 - s: s (2 + (1 - s) (2 + 1.25 |x|))
//   softmax  the sum has its terms' mean error, at most 2 + 1.66 ln E < 13.6 (the mean of |x| is below the entropy), and
//            its roundings, a lane's experts and five joins: (EPL + 5) / 2; with the reciprocal, the product and the
//            exponential's own 2: s (20 + EPL / 2 + 2.5 |x|)
// and the key's rounding half of |key|.  route_err: of a key whose score and x are known.  route_err_any: of any
// key with that value, whose score is at most S = |key| + bmax and at most smax (1; in softmax the largest of the row):
// sigmoid, s (1 - s) (2 + 1.25 |x|) < 0.8; softmax, s |x| <= s ln(1 / s), which grows with s up to 1 / e.  With smax one
// large finite bias (an expert switched off by -1e9) leaves the other keys' bounds small.  A bound grows slower than the
// keys do, so that key + route_err_any(key) bounds every smaller key too.  sum: ROUTE_ERR_SUM.
template <int EPL>
constexpr float ROUTE_ERR_SUM = 20.0f + 0.5f * EPL;

template <bool SIG>
__device__ __forceinline__ float route_err(float sum, float s, float x, float key) {
    const float rel = SIG ? fmaf(1.0f - s, fmaf(1.25f, fabsf(x), 2.0f), 2.0f) : fmaf(2.5f, fabsf(x), sum);
    return 1.1920929e-7f * fmaf(s, rel, fabsf(key)) + 1e-36f;
}
template <bool SIG>
__device__ __forceinline__ float route_err_any(float sum, float key, float bmax, float smax) {
    const float S = fminf(fabsf(key) + bmax, smax);
    if (SIG) return 1.1920929e-7f * (2.0f * S + 0.8f + fabsf(key));
    const float sx = S < 0.36f ? -S * __logf(S + 1e-30f) : 0.37f;
    return 1.1920929e-7f * (fmaf(sum, S, fabsf(key)) + 2.5f * sx) + 1e-36f;
}

__device__ __forceinline__ void order2(int& a, int& b) {      // a >= b
    const int hi = max(a, b);
    b = min(a, b);
    a = hi;
}

// The D = min(EPL, 4) largest of key[] below `bound`, in descending order.
template <int EPL, int D>
__device__ __forceinline__ void largest(const int (&key)[EPL], int bound, int (&top)[D]) {
    if (EPL < 4) {
#pragma unroll
        for (int i = 0; i < D; ++i) top[i] = key[i] < bound ? key[i] : ORD_EMPTY;
        if (D == 2) order2(top[0], top[D - 1]);
    } else {
#pragma unroll
        for (int q = 0; q < EPL; q += 4) {
            int v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = key[(q + i) % EPL] < bound ? key[(q + i) % EPL] : ORD_EMPTY;
            order2(v[0], v[1]); order2(v[2], v[3]); order2(v[0], v[2]); order2(v[1], v[3]); order2(v[1], v[2]);
            if (q == 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) top[i % D] = v[i];
            } else {      // the larger half of two sorted lists, then in order
#pragma unroll
                for (int i = 0; i < 4; ++i) top[i % D] = max(top[i % D], v[3 - i]);
                order2(top[0], top[2 % D]); order2(top[1 % D], top[3 % D]);
                order2(top[0], top[1 % D]); order2(top[2 % D], top[3 % D]);
            }
        }
    }
}

enum { ROUTE_LOGIT = 0, ROUTE_SIGMOID = 1, ROUTE_SOFTMAX = 2 };   // what a key is

// LPT lanes per token: 32, or 16 with a token on each half of the warp, which shares all that goes over the lanes
// (k < 16, at most 16 experts per lane).
template <int LPT, int EPL, bool VEC, int KIND>
__global__ void __launch_bounds__(ROUTE_WARPS * 32, EPL <= 8 ? 4 : EPL <= 16 && LPT == 16 ? 3 : 1)
route_scored_kernel(const __grid_constant__ RouteScored p, const __grid_constant__ RouteLanes m,
                    const __grid_constant__ RouteLanes m64) {
    extern __shared__ double route_keys[];      // route_token_f64: 32 m64.per doubles per warp
    constexpr int TOKENS = 32 / LPT;            // of a warp
    constexpr int BITS = EPL <= 1 ? 0 : EPL <= 2 ? 1 : EPL <= 4 ? 2 : EPL <= 8 ? 3 : EPL <= 16 ? 4 : EPL <= 32 ? 5 : 6;
    constexpr int POS = (1 << BITS) - 1;
    constexpr int D = EPL < 4 ? EPL : 4;
    constexpr float TRUNC = 1.1920929e-7f * (1 << BITS);       // relative, of the position's bits
    constexpr float SUM = ROUTE_ERR_SUM<EPL>;
    const int lane = threadIdx.x & (LPT - 1), warp = threadIdx.x >> 5, half = (threadIdx.x & 31) / LPT;
    const unsigned all = 0xffffffffu;
    const RouteLane at(p, m, lane);
    const int g = at.group, e0 = at.e0, cnt = at.cnt;
    // the bias, NaN and +inf as -inf (reported): in registers, or for many experts per lane in shared memory
    constexpr bool KEEP_BIAS = EPL <= 8;
    float bias[KEEP_BIAS ? EPL : 1];
    __shared__ float4 s_bias[KEEP_BIAS ? 1 : EPL / 4 * LPT];   // experts 4 q .. 4 q + 3 of a lane at [q LPT + lane]
    grid_wait();
    grid_launch_next();
    float bmax = 0.0f;                           // of the finite biases
    {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            float b = p.bias && i < cnt ? __ldg(p.bias + e0 + i) : 0.0f;
            bad |= !(b < INFINITY);
            b = b < INFINITY ? b : -INFINITY;
            if (b > -INFINITY) bmax = fmaxf(bmax, fabsf(b));
            if (KEEP_BIAS) bias[KEEP_BIAS ? i : 0] = b;
            else if (warp == 0 && half == 0) reinterpret_cast<float*>(&s_bias[(i >> 2) * LPT + lane])[i & 3] = b;
        }
        bmax = __int_as_float(__reduce_max_sync(all, __float_as_int(bmax)));   // every half has all experts
        if (bad) record_error(-7 /* MOE_ERR_CHECK */);
        if (!KEEP_BIAS) __syncthreads();
    }
    const long long stride = (long long)gridDim.x * ROUTE_WARPS * TOKENS;
    long long t0 = ((long long)blockIdx.x * ROUTE_WARPS + warp) * TOKENS;      // the warp's first token
    float l[EPL];
    auto load = [&](long long tok) {
        const float* row = p.logits + tok * p.E;
        const int cnt = tok < p.T ? at.cnt : 0;               // a half without a token: every expert masked
        if (VEC) {
#pragma unroll
            for (int i = 0; i < EPL; i += 4) {
                float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                if (i < cnt) v = __ldg(reinterpret_cast<const float4*>(row + e0 + i));
                l[i] = v.x; l[i + 1] = v.y; l[i + 2] = v.z; l[i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) l[i] = i < cnt ? __ldg(row + e0 + i) : -INFINITY;
            for (int sp = 1; sp < p.nsplit; ++sp) {
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (i < cnt) l[i] = __fadd_rn(l[i], __ldg(row + sp * p.split_stride + e0 + i));
            }
            if (p.nsplit > 1 && p.logits_out) {
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (i < cnt) p.logits_out[tok * p.E + e0 + i] = l[i];
            }
        }
    };
    if (t0 < p.T) load(t0 + half);
    for (; t0 < p.T; t0 += stride) {
        const long long t = t0 + half;
        const float* row = p.logits + t * p.E;
        // ---- keys
        float top = -INFINITY, total = 1.0f, inv = 1.0f;
        float zero = 0.0f;                                    // stays 0 while every logit is finite
#pragma unroll
        for (int i = 0; i < EPL; ++i) zero = fmaf(l[i], 0.0f, zero);
        const bool finite = __all_sync(all, zero == 0.0f);
        if (!finite) {
            bool bad = false;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                bad |= !(l[i] < INFINITY);
                l[i] = l[i] < INFINITY ? l[i] : -INFINITY;
            }
            if (__any_sync(all, bad) && threadIdx.x % 32 == 0) record_error(-7 /* MOE_ERR_CHECK */);
        }
        float ex[EPL];                                        // e^(l - top) or e^-l
        if (KIND == ROUTE_SOFTMAX || (KIND == ROUTE_LOGIT && !p.sigmoid && !p.renorm)) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) top = fmaxf(top, l[i]);
            top = from_ordered(lanes_max<LPT>(ordered(top + 0.0f)));
            const float ref = top > -INFINITY ? top : 0.0f;
            float part_sum = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                ex[i] = exp_approx(l[i] - ref);               // 0 for -inf
                part_sum += ex[i];
            }
            total = lanes_sum<LPT>(part_sum);
            inv = 1.0f / total;
        }
        const float smax = KIND == ROUTE_SOFTMAX ? inv * 1.0001f : 1.0f;   // no score is above it, errors included
        int key[EPL];
        constexpr int Q = EPL < 4 ? EPL : 4;
        auto keys = [&](auto masks) {                         // masks: some logits are -inf
#pragma unroll
            for (int q = 0; q < EPL; q += Q) {
                float b4[4];
                if (!KEEP_BIAS && KIND != ROUTE_LOGIT) {
                    const float4 v = s_bias[(q >> 2) * LPT + lane];
                    b4[0] = v.x; b4[1] = v.y; b4[2] = v.z; b4[3] = v.w;
                }
#pragma unroll
                for (int r = 0; r < Q; ++r) {
                    const int i = q + r;
                    float k32 = l[i] + 0.0f;                  // no -0 (a sum with a score is none)
                    if (KIND != ROUTE_LOGIT) {
                        const float s = KIND == ROUTE_SIGMOID ? rcp_approx(1.0f + exp_approx(-l[i])) : ex[i] * inv;
                        k32 = s + (KEEP_BIAS ? bias[KEEP_BIAS ? i : 0] : b4[r]);
                        if (decltype(masks)::value && !(l[i] > -INFINITY)) k32 = -INFINITY;
                    }
                    key[i] = (ordered(k32) & ~POS) | (POS - i);
                }
            }
        };
        if (finite) keys(std::false_type());
        else keys(std::true_type());
        if (t0 + stride < p.T) load(t + stride);              // on its way while this token is finished
        int head[D];
        largest<EPL, D>(key, 0x7fffffff, head);
        bool sure = true;
        // ---- groups
        if (p.n_group > 1) {
            int a = head[0], b = D > 1 ? head[D > 1 ? 1 : 0] : ORD_EMPTY;
            for (int o = 1; o < (1 << m.lg); o <<= 1) {
                const int a2 = __shfl_xor_sync(all, a, o), b2 = __shfl_xor_sync(all, b, o);
                b = max(max(b, b2), min(a, a2));
                a = max(a, a2);
            }
            // the value (without positions) as an ordered integer, and the error of its one or two keys and of their sum;
            // EMPTY: no expert left.  Largest finite keys may add up to an infinity: clamped
            const bool both = p.top2 && b >= ORD_LOWEST;
            const float fa = from_ordered(a & ~POS), fb = both ? from_ordered(b & ~POS) : 0.0f;
            const float value = fminf(fmaxf(fa + fb, -FLT_MAX), FLT_MAX);
            int v = g < p.n_group && a >= ORD_LOWEST ? ordered(value + 0.0f) : ORD_EMPTY;
            float err = 0.0f;                                 // logits are compared as they are
            if (KIND != ROUTE_LOGIT) {
                constexpr bool SIG = KIND == ROUTE_SIGMOID;
                err = route_err_any<SIG>(SUM, fa, bmax, smax) + TRUNC * fabsf(fa) + 2.4e-7f * fabsf(value);
                if (both) err += route_err_any<SIG>(SUM, fb, bmax, smax) + TRUNC * fabsf(fb);
            }
            // the topk_group largest, one by one
            bool kept = false;
            for (int q = 0; q < p.topk_group; ++q) {
                const int most = lanes_max<LPT>(v);
                const int owner = __ffs(lanes_ballot<LPT>(v == most)) - 1;
                if (g == (owner >> m.lg) && most != ORD_EMPTY) {
                    kept = true;
                    v = ORD_EMPTY;
                }
            }
            // certain where the least that a kept group can be is above the most that another can be
            const int most = lanes_max<LPT>(v != ORD_EMPTY ? ordered(value + err) : ORD_EMPTY);
            const int least = lanes_max<LPT>(kept ? ordered(err - value) : ORD_EMPTY);
            if (most != ORD_EMPTY) sure = -from_ordered(least) > from_ordered(most);
            if (!kept) {
#pragma unroll
                for (int i = 0; i < D; ++i) head[i] = ORD_EMPTY;
            }
        }
        // ---- slots: lane j takes the j-th largest key and its lane; lane k (k < LPT) the one that comes next
        const int last = min(p.k, LPT - 1);
        int mine = ORD_EMPTY, from = 0;
#pragma unroll 1
        for (int j = 0; j <= last; ++j) {                     // past the last unmasked key: keys below ORD_LOWEST
            const int hi = lanes_max<LPT>(head[0]);
            const int owner = __ffs(lanes_ballot<LPT>(head[0] == hi)) - 1;
            const bool taken = lane == owner;
            mine = lane == j ? hi : mine;
            from = lane == j ? owner : from;
#pragma unroll
            for (int i = 0; i + 1 < D; ++i) head[i] = taken ? head[i + 1] : head[i];
            head[D - 1] = taken ? ORD_EMPTY : head[D - 1];
            if (EPL > 4 && __any_sync(all, taken && head[0] == ORD_EMPTY && hi >= ORD_LOWEST)) {
                if (taken) largest<EPL, D>(key, hi, head);
            }
        }
        const bool entry = lane <= last && mine >= ORD_LOWEST;
        int my_e = -1;
        float my_l = 0.0f;
        if (entry) {
            my_e = (from >> m.lg) * m.each + (from & ((1 << m.lg) - 1)) * m.per + (POS - (mine & POS));
            my_l = scored_logit(p, row, my_e);
        }
        // ---- is the order certain?  Slot j against slot j + 1, by their whole keys, and every slot against `rest`, the
        // most that any other key can be
        const int next = p.k < LPT ? __shfl_sync(all, mine, p.k & (LPT - 1), LPT) : lanes_max<LPT>(head[0]);
        const float rest = from_ordered(next | POS);
        constexpr bool SIG = KIND == ROUTE_SIGMOID;
        float ka = my_l, ea = 0.0f;
        if (KIND != ROUTE_LOGIT) {
            const float x = SIG ? my_l : my_l - top;
            const float s = SIG ? rcp_approx(1.0f + exp_approx(-x)) : exp_approx(x) * inv;
            ka = s + (p.bias && entry ? __ldg(p.bias + my_e) : 0.0f);
            ea = route_err<SIG>(SUM, s, x, ka);
        }
        const float kb = __shfl_down_sync(all, ka, 1), eb = __shfl_down_sync(all, ea, 1);
        const int after = __shfl_down_sync(all, mine, 1);
        bool order = true;
        if (entry && lane < p.k) {
            // equal logits of two lanes may have come in the order of their positions
            if (lane + 1 < p.k && after >= ORD_LOWEST) order = ka - kb > ea + eb;
            if (next >= ORD_LOWEST)
                sure = sure && (KIND == ROUTE_LOGIT ? ka > rest : ka - rest > ea + route_err_any<SIG>(SUM, rest, bmax, smax));
        }
        // The slots are the right experts if all are certainly above the rest; otherwise, and where the groups were in
        // doubt, the token is done again.  Their order among themselves is put right here.
        const unsigned certain = lanes_ballot<LPT>(order);
        const unsigned doubt = ~certain & (p.k < 32 ? (1u << p.k) - 1u : all);
        if (__any_sync(all, doubt != 0)) {
            double t64 = 1.0;
            if (KIND == ROUTE_SOFTMAX) {
                double part_sum = 0.0;
                if (t < p.T) {
#pragma unroll 2
                    for (int i = 0; i < cnt; ++i) {
                        const float v = scored_logit(p, row, e0 + i);
                        part_sum += v < INFINITY && v > -INFINITY ? exp((double)v - (double)top) : 0.0;
                    }
                }
#pragma unroll
                for (int o = LPT / 2; o > 0; o >>= 1) part_sum += __shfl_xor_sync(all, part_sum, o);
                t64 = part_sum;
            }
            double k64 = my_l;
            if (KIND != ROUTE_LOGIT && entry)
                k64 = (KIND == ROUTE_SIGMOID ? 1.0 / (1.0 + exp(-(double)my_l)) : exp((double)my_l - (double)top) / t64) +
                      (double)(p.bias ? __ldg(p.bias + my_e) : 0.0f);
            if (!entry) k64 = -INFINITY;
            int rank = 0;
            for (int j = 0; j <= last; ++j) {                 // this entry's place among the entries
                const double o = __shfl_sync(all, k64, j, LPT);
                const int oe = __shfl_sync(all, my_e, j, LPT);
                rank += o > k64 || (o == k64 && oe < my_e);
            }
            int e2 = -1;
            float l2 = 0.0f;
            for (int j = 0; j <= last; ++j) {
                const int r = __shfl_sync(all, entry ? rank : LPT, j, LPT), oe = __shfl_sync(all, my_e, j, LPT);
                const float ol = __shfl_sync(all, my_l, j, LPT);
                if (r == lane) {
                    e2 = oe;
                    l2 = ol;
                }
            }
            my_e = e2;
            my_l = l2;
        }
        const unsigned unsure = __ballot_sync(all, !sure && t < p.T);
        scored_weights<LPT>(p, t, t < p.T && (LPT == 32 ? unsure == 0 : (unsure >> (16 * half) & 0xffffu) == 0), lane, my_e,
                            my_l, top, total);
        if (unsure) {
            if (unsure & (LPT == 32 ? all : 0xffffu))
                route_token_f64(p, m64, t0, threadIdx.x & 31, route_keys + (size_t)warp * 32 * m64.per);
            if (LPT == 16 && unsure >> 16) {
                __syncwarp();
                route_token_f64(p, m64, t0 + 1, threadIdx.x & 31, route_keys + (size_t)warp * 32 * m64.per);
            }
        }
    }
}

}  // namespace moe
