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
__device__ __forceinline__ void scored_weights(const RouteScored& p, long long t, int lane, int my_e, float my_l,
                                               float top, float total) {
    const bool have = lane < p.k && my_e >= 0;
    float s = 0.0f;
    if (p.renorm) {
        float m = warp_max(have ? my_l : -INFINITY);
        if (p.sigmoid) m = fminf(m, 0.0f);
        if (have) {
            if (!p.sigmoid) s = expf(my_l - m);
            else s = my_l >= 0.0f ? 1.0f / (1.0f + expf(-my_l)) : expf(my_l - m) / (1.0f + expf(my_l));
        }
        const float sum = warp_sum(s);
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
    scored_weights(p, t, lane, my_e, my_l, top, (float)total);
}

// Warps per block such that their keys fit in 48 KB of shared memory.
inline int route_f64_warps(int E) { return E <= 768 ? 8 : 4; }

__global__ void __launch_bounds__(256) route_scored_f64_kernel(const RouteScored p) {
    extern __shared__ double route_keys[];
    const int warp = threadIdx.x >> 5;
    const long long t = (long long)blockIdx.x * (blockDim.x >> 5) + warp;
    if (t >= p.T) return;
    route_token_f64(p, t, threadIdx.x & 31, route_keys + (size_t)warp * p.E);
}

}  // namespace moe
