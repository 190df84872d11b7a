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

// key order in 64 bits: larger first, equal keys -> lower expert
__device__ __forceinline__ bool key64_before(double ka, int ea, double kb, int eb) {
    return ka > kb || (ka == kb && ea < eb);
}

// The weights of the selected experts: lane j < k holds slot j's expert (-1: none) and logit.
// top / total: the row's largest logit and sum of e^(l - top) over its unmasked experts (softmax
// without renormalisation).  Renormalised weights are ratios of scores, taken relative to the largest
// selected one so that scores that underflow still have their ratio:
//   softmax  s_j ~ e^(l_j - m),  sigmoid  s_j = e^l_j / (1 + e^l_j) ~ e^(l_j - m) / (1 + e^l_j)
// with m the largest selected logit (sigmoid: at most 0).  Warp-collective.
// kw: a power of two >= k, the lanes that the sums run over.
__device__ __forceinline__ void scored_weights(const RouteScored& p, long long t, int lane, int my_e, float my_l,
                                               float top, float total, int kw) {
    const bool have = lane < p.k && my_e >= 0;
    float s = 0.0f;
    if (p.renorm) {
        float m = have ? my_l : -INFINITY;
        for (int o = kw >> 1; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (p.sigmoid) m = fminf(m, 0.0f);
        if (have) {
            if (!p.sigmoid) s = expf(my_l - m);
            else s = my_l >= 0.0f ? 1.0f / (1.0f + expf(-my_l)) : expf(my_l - m) / (1.0f + expf(my_l));
        }
        float sum = s;
        for (int o = kw >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (have) s /= sum;
    } else if (have) {
        s = p.sigmoid ? 1.0f / (1.0f + expf(-my_l)) : expf(my_l - top) / total;
    }
    if (lane < p.k) {
        p.idx[t * p.k + lane] = have ? my_e : -1;
        p.w[t * p.k + lane] = have ? s * p.scale : 0.0f;
    }
}

// One token by one warp with every key in 64 bits, in the caller's shared memory (E doubles).
// bad: set when a logit or bias is NaN or +inf (that expert is masked).
__device__ __noinline__ void route_token_f64(const RouteScored& p, long long t, int lane, double* keys) {
    const float* row = p.logits + t * p.E;
    bool bad = false;
    float top = -INFINITY;
    auto usable = [&](float l, float b) { return l < INFINITY && l > -INFINITY && b < INFINITY && b > -INFINITY; };
    for (int e = lane; e < p.E; e += 32) {
        const float l = scored_logit(p, row, e), b = p.bias ? __ldg(p.bias + e) : 0.0f;
        bad |= !(l < INFINITY) || !(b < INFINITY);
        if (l < INFINITY) top = fmaxf(top, l);
        if (p.nsplit > 1 && p.logits_out) p.logits_out[t * p.E + e] = l;
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) record_error(-7 /* MOE_ERR_CHECK */);
    top = warp_max(top);
    double total = 0.0;
    if (!p.sigmoid) {
        for (int e = lane; e < p.E; e += 32) {
            const float l = scored_logit(p, row, e);
            if (l < INFINITY && l > -INFINITY) total += exp((double)l - (double)top);
        }
        total = warp_sum(total);
    }
    for (int e = lane; e < p.E; e += 32) {
        const float l = scored_logit(p, row, e), b = p.bias ? __ldg(p.bias + e) : 0.0f;
        double key = -INFINITY;
        if (usable(l, b)) {
            if (p.by_logit) key = l;
            else key = (p.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)top) / total) + (double)b;
        }
        keys[e] = key;
    }
    __syncwarp();
    if (p.n_group > 1) {
        // lane g: the value of group g, then its rank among all
        const int each = p.E / p.n_group;
        double v = -INFINITY;
        if (lane < p.n_group) {
            double a = -INFINITY, b = -INFINITY;
            for (int i = 0; i < each; ++i) {
                const double x = keys[lane * each + i];
                if (x > a) { b = a; a = x; } else if (x > b) { b = x; }
            }
            v = p.top2 && b > -INFINITY ? a + b : a;
        }
        int rank = 0;
        for (int g = 0; g < p.n_group; ++g) {
            const double o = __shfl_sync(0xffffffffu, v, g);
            rank += key64_before(o, g, v, lane);
        }
        const uint32_t kept = __ballot_sync(0xffffffffu, lane < p.n_group && rank < p.topk_group);
        __syncwarp();
        for (int e = lane; e < p.E; e += 32)
            if (!((kept >> (e / each)) & 1u)) keys[e] = -INFINITY;
        __syncwarp();
    }
    int my_e = -1;
    for (int j = 0; j < p.k; ++j) {
        double bk = -INFINITY;
        int be = 0x7fffffff;
        for (int e = lane; e < p.E; e += 32)
            if (keys[e] > bk) { bk = keys[e]; be = e; }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double ok = __shfl_xor_sync(0xffffffffu, bk, o);
            const int oe = __shfl_xor_sync(0xffffffffu, be, o);
            if (key64_before(ok, oe, bk, be)) { bk = ok; be = oe; }
        }
        if (be >= p.E) break;               // no unmasked expert left
        if (lane == j) my_e = be;
        __syncwarp();
        if (lane == 0) keys[be] = -INFINITY;
        __syncwarp();
    }
    const float my_l = my_e >= 0 ? scored_logit(p, row, my_e) : 0.0f;
    scored_weights(p, t, lane, my_e, my_l, top, (float)total, 32);
}

// ---------------------------------------------------------------- the kernel: keys in 32 bits
//
// One warp per token; group g of experts lies on LPG = 2^x <= 32 / n_group lanes, each holding up to EPL
// consecutive experts, so that (lane, position) is the order of the experts.  Keys are kept as integers of the
// same order.
//   groups      two largest keys per lane, merged over the group's lanes; rank by n_group shuffles
//   candidates  the lanes of the groups that stay form at least k blocks of 2^sub lanes; the smallest of the blocks'
//               maxima is exceeded by at least k keys.  The keys not below it (less their error) are moved to shared
//               memory, typically 2 k to 3 k of them, and each is ranked against all.  More than ROUTE_CAND: the k + 1
//               largest are taken out one by one instead.
//   certainty   32-bit keys are at most route_err off.  Where two neighbours in the order, or the last group that
//               stays and the first that does not, are closer than that, the token is done again in 64 bits
//               (route_token_f64): about one token in a thousand for scores of unit variance.
//   weights     from the selected logits, with the library's expf
// 32768 x 256, 8 groups, k = 8: the logits alone are 33.5 MB, 5.2 us at the measured copy rate.
constexpr int ROUTE_CAND = 64;
constexpr int ROUTE_WARPS = 8;

// Errors in units of 2^-23.  The fast exponential of x is off by at most 2 + 1.16 |x| of its value (x = -l, or
// l - top in softmax, whose rounding adds |x| / 2), the divide by 2.
//   sigmoid  the exponential's part reaches s by the factor 1 - s: s (5 + 1.25 |x|)
//   softmax  the sum adds its terms' mean error, at most 2 + 1.7 ln E, and its roundings, at most (E / 32 + 5) / 2:
//            s (40 + 2.5 |x|) for E <= 1024
// and the key's rounding half of |key|.  route_err: of a key whose score and x are known.  route_err_any: of any
// key with that value; sigmoid: s (1 - s) |x| < 0.23; softmax: s <= |key| + bmax, and |x| <= 40 or s < 1e-17.
__device__ __forceinline__ float route_err(bool sigmoid, float s, float x, float key) {
    const float rel = sigmoid ? fmaf(1.25f, fabsf(x), 5.0f) : fmaf(2.5f, fabsf(x), 40.0f);
    return 1.1920929e-7f * fmaf(s, rel, fabsf(key)) + 1e-36f;
}
__device__ __forceinline__ float route_err_any(bool sigmoid, float key, float bmax) {
    return sigmoid ? 4.8e-7f * (1.0f + fabsf(key)) : 1.7e-5f * (fabsf(key) + bmax) + 1e-17f;
}

// floats as integers of the same order (no NaN; -0 must have been made +0)
__device__ __forceinline__ int ordered(float f) {
    const int b = __float_as_int(f);
    return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float from_ordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }
constexpr int ORD_NONE = (int)0x807fffff;      // ordered(-inf): a masked expert

struct RouteLanes {
    int lpg;      // lanes per group
    int per;      // experts per lane (the last lanes of a group may hold fewer)
    int sub;      // log2 of the lanes of a candidate block; < 0: every key is a candidate
    int kw;       // power of two >= k
};

template <int EPL, bool VEC>
__global__ void __launch_bounds__(ROUTE_WARPS * 32) route_scored_kernel(const __grid_constant__ RouteScored p,
                                                                        const __grid_constant__ RouteLanes m) {
    extern __shared__ double route_keys[];      // route_token_f64: E doubles per warp
    __shared__ __align__(16) int c_key[ROUTE_WARPS][ROUTE_CAND + 4];
    __shared__ int c_idx[ROUTE_WARPS][ROUTE_CAND];
    __shared__ float c_l[ROUTE_WARPS][ROUTE_CAND];
    __shared__ int o_key[ROUTE_WARPS][MAX_TOPK + 1], o_idx[ROUTE_WARPS][MAX_TOPK + 1];
    __shared__ float o_l[ROUTE_WARPS][MAX_TOPK + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned all = 0xffffffffu;
    const int each = p.E / p.n_group;
    const int g = lane / m.lpg, part = lane - g * m.lpg;
    const int e0 = g * each + part * m.per;
    const int cnt = g < p.n_group ? max(0, min(m.per, each - part * m.per)) : 0;
    constexpr bool KEEP_BIAS = EPL <= 8;
    float bias[KEEP_BIAS ? EPL : 1];
    grid_wait();
    grid_launch_next();
    float bmax = 0.0f;                           // of the finite biases
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const float b = i < cnt ? __ldg(p.bias + e0 + i) : 0.0f;
            if (KEEP_BIAS) bias[KEEP_BIAS ? i : 0] = b;
            if (fabsf(b) < INFINITY) bmax = fmaxf(bmax, fabsf(b));
        }
        bmax = __int_as_float(__reduce_max_sync(all, __float_as_int(bmax)));
    } else if (KEEP_BIAS) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) bias[KEEP_BIAS ? i : 0] = 0.0f;
    }
    for (long long t = (long long)blockIdx.x * ROUTE_WARPS + warp; t < p.T; t += (long long)gridDim.x * ROUTE_WARPS) {
        const float* row = p.logits + t * p.E;
        float l[EPL];
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
                    if (i < cnt) p.logits_out[t * p.E + e0 + i] = l[i];
            }
        }
        // ---- keys (ordered integers); masked experts ORD_NONE
        bool bad = false;
        float top = -INFINITY, total = 1.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            if (!(l[i] < INFINITY)) {
                bad = true;
                l[i] = -INFINITY;
            }
            if (!p.sigmoid) top = fmaxf(top, l[i]);
        }
        int key[EPL];
        if (!p.sigmoid && !(p.by_logit && p.renorm)) {
            top = from_ordered(__reduce_max_sync(all, ordered(top + 0.0f)));
            float part_sum = 0.0f;
            const float ref = top > -INFINITY ? top : 0.0f;
            float ex[EPL];
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                ex[i] = __expf(l[i] - ref);                   // 0 for -inf
                part_sum += ex[i];
            }
            total = warp_sum(part_sum);
            const float inv = __fdividef(1.0f, total);
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const float b = KEEP_BIAS ? bias[KEEP_BIAS ? i : 0] : (p.bias && i < cnt ? __ldg(p.bias + e0 + i) : 0.0f);
                bad |= !(b < INFINITY);
                const float k32 = (p.by_logit ? l[i] : ex[i] * inv + b) + 0.0f;
                key[i] = l[i] > -INFINITY && b > -INFINITY && b < INFINITY ? ordered(k32) : ORD_NONE;
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const float b = KEEP_BIAS ? bias[KEEP_BIAS ? i : 0] : (p.bias && i < cnt ? __ldg(p.bias + e0 + i) : 0.0f);
                bad |= !(b < INFINITY);
                const float k32 = (p.by_logit ? l[i] : __fdividef(1.0f, 1.0f + __expf(-l[i])) + b) + 0.0f;
                key[i] = l[i] > -INFINITY && b > -INFINITY && b < INFINITY ? ordered(k32) : ORD_NONE;
            }
        }
        if (__any_sync(all, bad) && lane == 0) record_error(-7 /* MOE_ERR_CHECK */);
        bool sure = true;
        // ---- groups
        if (p.n_group > 1) {
            int a = ORD_NONE, b = ORD_NONE;                   // two largest
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                b = max(b, min(a, key[i]));
                a = max(a, key[i]);
            }
            for (int o = 1; o < m.lpg; o <<= 1) {
                const int a2 = __shfl_xor_sync(all, a, o), b2 = __shfl_xor_sync(all, b, o);
                b = max(max(b, b2), min(a, a2));
                a = max(a, a2);
            }
            if (p.top2 && b != ORD_NONE) a = max(ORD_NONE + 1, ordered(from_ordered(a) + from_ordered(b) + 0.0f));
            int rank = 0;
            for (int q = 0; q < p.n_group; ++q) {
                const int o = __shfl_sync(all, a, q * m.lpg);
                rank += o > a || (o == a && q < g);
            }
            const bool kept = g < p.n_group && rank < p.topk_group;
            if (!p.by_logit) {
                const int lo = __reduce_min_sync(all, kept ? a : 0x7fffffff);
                const int hi = __reduce_max_sync(all, !kept && g < p.n_group ? a : ORD_NONE);
                if (hi != ORD_NONE) {
                    const float fl = from_ordered(lo), fh = from_ordered(hi);
                    // a value is one key, or two: each within the error of a key of twice its size
                    sure = fl - fh > 2.0f * (route_err_any(p.sigmoid, 2.0f * fl, bmax) + route_err_any(p.sigmoid, 2.0f * fh, bmax));
                }
            }
            if (!kept) {
#pragma unroll
                for (int i = 0; i < EPL; ++i) key[i] = ORD_NONE;
            }
        }
        // ---- candidates
        int best = ORD_NONE;
#pragma unroll
        for (int i = 0; i < EPL; ++i) best = max(best, key[i]);
        int thr = ORD_NONE + 1;                               // any key that is not masked
        if (m.sub >= 0) {
            int blk = best;
            for (int o = 1; o < (1 << m.sub); o <<= 1) blk = max(blk, __shfl_xor_sync(all, blk, o));
            // lanes outside the groups that stay, or without experts, do not count
            const bool counts = cnt > 0 && best != ORD_NONE;
            const int lowest = __reduce_min_sync(all, counts ? blk : 0x7fffffff);
            const int blocks = __popc(__ballot_sync(all, blk != ORD_NONE && (lane & ((1 << m.sub) - 1)) == 0));
            if (blocks >= p.k) {
                const float f = from_ordered(lowest);
                thr = p.by_logit ? lowest : ordered(f - 2.0f * route_err_any(p.sigmoid, f, bmax) + 0.0f);
                thr = max(thr, ORD_NONE + 1);
            }
        }
        unsigned mask = 0;
        uint32_t mask_hi = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            if (i < 32) mask |= (unsigned)(key[i] >= thr) << (i & 31);
            else mask_hi |= (uint32_t)(key[i] >= thr) << (i & 31);
        }
        const int mine = __popc(mask) + __popc(mask_hi);
        int before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(all, before, o);
            if (lane >= o) before += v;
        }
        const int n = __shfl_sync(all, before, 31);
        before -= mine;
        int found;                                            // entries of o_*: min(k + 1, unmasked)
        if (n <= ROUTE_CAND) {
            int at = before;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                if (key[i] >= thr) {
                    c_key[warp][at] = key[i];
                    c_idx[warp][at] = e0 + i;
                    c_l[warp][at] = l[i];
                    ++at;
                }
            }
            if (lane < 4) c_key[warp][n + lane] = ORD_NONE;   // whole vectors below
            __syncwarp();
            found = min(n, p.k + 1);
            for (int a = lane; a < n; a += 32) {
                const int ka = c_key[warp][a];
                int rank = 0;
                for (int j = 0; j < n; j += 4) {
                    const int4 o = *reinterpret_cast<const int4*>(&c_key[warp][j]);
                    rank += o.x > ka - (j < a);
                    rank += o.y > ka - (j + 1 < a);
                    rank += o.z > ka - (j + 2 < a);
                    rank += o.w > ka - (j + 3 < a);
                }
                if (rank <= p.k) {
                    o_key[warp][rank] = ka;
                    o_idx[warp][rank] = c_idx[warp][a];
                    o_l[warp][rank] = c_l[warp][a];
                }
            }
        } else {
            found = 0;
            for (int j = 0; j <= p.k; ++j) {
                const int hi = __reduce_max_sync(all, best);
                if (hi == ORD_NONE) break;
                const int owner = __ffs(__ballot_sync(all, best == hi)) - 1;
                if (lane == owner) {
                    bool taken = false;
                    best = ORD_NONE;
#pragma unroll
                    for (int i = 0; i < EPL; ++i) {
                        if (!taken && key[i] == hi) {
                            taken = true;
                            key[i] = ORD_NONE;
                            o_key[warp][j] = hi;
                            o_idx[warp][j] = e0 + i;
                            o_l[warp][j] = l[i];
                        }
                        best = max(best, key[i]);
                    }
                }
                found = j + 1;
            }
        }
        __syncwarp();
        // ---- slot j on lane j; the (k + 1)-th key is only compared with
        int my_e = -1;
        float my_l = 0.0f;
        if (lane < min(found, p.k)) {
            my_e = o_idx[warp][lane];
            my_l = o_l[warp][lane];
            if (!p.by_logit && lane + 1 < found) {
                const float ka = from_ordered(o_key[warp][lane]), kb = from_ordered(o_key[warp][lane + 1]);
                const float lb = o_l[warp][lane + 1];
                const float xa = p.sigmoid ? my_l : my_l - top, xb = p.sigmoid ? lb : lb - top;
                const float sa = p.sigmoid ? __fdividef(1.0f, 1.0f + __expf(-xa)) : __fdividef(__expf(xa), total);
                const float sb = p.sigmoid ? __fdividef(1.0f, 1.0f + __expf(-xb)) : __fdividef(__expf(xb), total);
                sure = sure && ka - kb > route_err(p.sigmoid, sa, xa, ka) + route_err(p.sigmoid, sb, xb, kb);
            }
        }
        if (__all_sync(all, sure)) {
            scored_weights(p, t, lane, my_e, my_l, top, total, m.kw);
        } else {
            route_token_f64(p, t, lane, route_keys + (size_t)warp * p.E);
        }
        __syncwarp();                                         // o_*, c_* are free again
    }
}

}  // namespace moe
