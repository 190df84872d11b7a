// linear.cuh - the dense layer y = act(x W^T + bias) + residual on the tcgen05 tensor cores.
//
// x [M, K] (M tokens), W [N, K], both K-major; y [M, N] bf16.  MOE_ACT_SWIGLU: y = silu(x W^T + bias) *
// (x W_up^T + bias_up) + residual.  F8: e4m3 x (one scale per token) and W (one scale per output),
// the fp32 accumulator multiplied by both.  Everything between the product and the one rounding to
// bf16 is in fp32.
//
// Three kernels, chosen by run_linear_as() and plan_linear():
//   linear_rows_kernel   one or two tokens: a stream of weights through registers
//   linear_split_kernel  more tokens: 128 weight rows x up to 128 tokens per tile, K cut over a cluster
//   linear_pair_kernel   many tokens: persistent CTA pairs, 256 weight rows x up to 256 tokens
// In the last two the weights are the MMA's M side (D^T = W x^T), so few tokens cost no padded 128-row tile and
// the token tile can be any multiple of 16.  SwiGLU tiles take 64 rows of W and the same 64 of W_up per CTA.
//
// linear_split_kernel: the K range of a tile is cut over the `split` CTAs of a cluster, which join their partial
// sums through distributed shared memory in rank order: no workspace, no atomics, the same result every
// time.  Warp roles (256 threads): warp 0 TMA producer, warp 1 tensor memory + MMA issuer, warps 2-3 bring the
// epilogue's operands into L2.  Then all eight warps move the accumulator (a lane per output, a column per
// token) to shared memory as fp32 [slice][token][128], each token's sums to the rank of the cluster that owns
// the token, and each rank adds the slices of its tokens, applies the epilogue and stores.  What bounds it: the
// weights' stream for few tokens (14336 x 4096, 16 tokens: 23.3 us, 5.0 of 6.46 TB/s), the operands' way from
// L2 for hundreds (512 x 4096 x 4096: 23.5 us against the pairs' 18.6, 32 KB per 128 x 128 x 64 products);
// setting up, handing over and joining take about 4 us besides.  Tried: pairs of CTAs (cta_group::2) in this
// kernel, which halve the token traffic, won or lost under 10 % at 128 to 1024 tokens; prefetching weights into L2
// ahead of the ring cost 5 to 20 %.
#pragma once

#include "grouped_gemm.cuh"
#include "route_permute_combine.cuh"

namespace moe {

enum { LIN_NONE = 0, LIN_RELU = 1, LIN_SILU = 2, LIN_GELU = 3, LIN_GELU_TANH = 4, LIN_SWIGLU = 5 };

constexpr int LIN_BM = 128;                        // weight rows per tile
constexpr int LIN_A_BYTES = LIN_BM * 128;          // one stage of weights: 128-byte rows
constexpr int LIN_THREADS = 256;
constexpr int LIN_MAX_SPLIT = 8;                   // portable cluster size
constexpr int LIN_MAX_STAGES = 8;

struct LinearParams {
    int M, N, K;
    int bn;        // tokens per tile
    int mt;        // token tiles
    int stages, split;
    int own_part;  // 1: the partial sums have shared memory of their own
    int tmem_cols; // power of two >= max(bn, 32)
    int act;
    const float *bias, *bias_up;
    const __nv_bfloat16* residual;
    __nv_bfloat16* y;
    const float *sx, *sw, *sw_up;                  // F8 scales
};

// Partial sums of a CTA: `split` slices of ceil(ntok / split) tokens, at most bn + split - 1 rows.
__host__ __device__ constexpr int linear_part_bytes(int bn, int split) { return (bn + split) * LIN_BM * 4; }
__host__ __device__ constexpr int linear_smem_bytes(int stages, int bn, int own_part_bytes) {
    return stages * (LIN_A_BYTES + bn * 128) + own_part_bytes + 1024 + 256;
}

// Phi(-|z|) of the normal distribution: erfc(u) / 2 with u = |z| / sqrt(2) as t P(t) e^(-u^2) / 2, t = 1 / (1 + 0.4 u).
// P is the degree-8 polynomial of least relative error against e^(u^2) erfc(u) / t on 0 < t <= 1 (1.3e-7, found by a
// weighted least-squares iteration), halved here: the tail keeps its relative precision, at 20 instructions
// where the library's erfc takes about twice as many (1152 x 7680 x 896: 45 us with that, 25.5 with this).
__device__ __forceinline__ float normal_tail(float z) {
    const float u = fabsf(z) * 0.70710678118654752f;
    const float t = __fdividef(1.0f, fmaf(0.4f, u, 1.0f));
    float q = 0.5f * 0.05026210844516754f;
    q = fmaf(q, t, 0.5f * -0.18290141224861145f);
    q = fmaf(q, t, 0.5f * 0.16908535361289978f);
    q = fmaf(q, t, 0.5f * -0.005607480648905039f);
    q = fmaf(q, t, 0.5f * 0.14143140614032745f);
    q = fmaf(q, t, 0.5f * 0.16854198276996613f);
    q = fmaf(q, t, 0.5f * 0.20784269273281097f);
    q = fmaf(q, t, 0.5f * 0.22566959261894226f);
    q = fmaf(q, t, 0.5f * 0.22567586600780487f);
    return q * t * __expf(-u * u);
}

// z / (1 + e^-v), by e^-|v|: the divisor stays within [1, 2], where 1 + e^-v would pass 2^126, from which on its fast
// reciprocal is 0, while the quotient is still a normal bf16 (z = v = -88: -5e-37).
__device__ __forceinline__ float times_sigmoid(float z, float v) {
    const float e = __expf(-fabsf(v));
    return (v < 0.0f ? z * e : z) * rcp_approx(1.0f + e);
}
__device__ __forceinline__ float linear_swiglu(float g, float u) { return times_sigmoid(g, g) * u; }

// Activation of a pre-activation z (not SwiGLU).  gelu: z Phi(z); gelu_tanh: (1 + tanh v) / 2 = sigmoid(2v), so that
// neither tail cancels.  The fast exponential of a is off by up to (2 + 1.2 |a|) 2^-23 of its value, the reciprocal by 2^-23:
// a few ulp near 0, 2^-16 at a = -90, far below the bf16 rounding that follows.  relu keeps NaN.
__device__ __forceinline__ float linear_act(int act, float z) {
    switch (act) {
        case LIN_RELU: return z < 0.0f ? 0.0f : z;
        case LIN_SILU: return times_sigmoid(z, z);
        case LIN_GELU: {
            const float q = normal_tail(z);
            return z * (z < 0.0f ? q : 1.0f - q);      // infinity stays: q is 0 there, and z - z q would be NaN
        }
        case LIN_GELU_TANH: return times_sigmoid(z, 1.5957691216057308f * fmaf(0.044715f * z * z, z, z));
        default: return z;
    }
}

__device__ __forceinline__ void st_cluster_f1(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// act of C values; the branch on act is taken once
template <int C>
__device__ __forceinline__ void linear_acts(int act, float (&z)[C]) {
    switch (act) {
        case LIN_RELU:
#pragma unroll
            for (int i = 0; i < C; ++i) z[i] = linear_act(LIN_RELU, z[i]);
            break;
        case LIN_SILU:
#pragma unroll
            for (int i = 0; i < C; ++i) z[i] = linear_act(LIN_SILU, z[i]);
            break;
        case LIN_GELU:
#pragma unroll
            for (int i = 0; i < C; ++i) z[i] = linear_act(LIN_GELU, z[i]);
            break;
        case LIN_GELU_TANH:
#pragma unroll
            for (int i = 0; i < C; ++i) z[i] = linear_act(LIN_GELU_TANH, z[i]);
            break;
        default: break;
    }
}

__device__ __forceinline__ float4 f4_or(const float* p, bool on, float v) {
    return on ? __ldg(reinterpret_cast<const float4*>(p)) : make_float4(v, v, v, v);
}

__device__ __forceinline__ void bf16x4_to_f32(const uint2& v, float* f) {
    f[0] = __uint_as_float(v.x << 16);
    f[1] = __uint_as_float(v.x & 0xffff0000u);
    f[2] = __uint_as_float(v.y << 16);
    f[3] = __uint_as_float(v.y & 0xffff0000u);
}

// The outputs of one of 256 epilogue threads, with their bias and scales: where rows of y are 8-byte aligned
// (N % 4 == 0), 16 threads share a token and thread i has outputs 4 i .. 4 i + 3 and (not GATED)
// 64 + 4 i .. 64 + 4 i + 3 of the CTA's 128 (GATED: 64).
template <bool F8, bool GATED>
struct LinearCols {
    int f, na, nb;
    bool oka, okb;
    float4 ba, bb, wa, wb;
    __device__ __forceinline__ void load(const LinearParams& p, int tid, int n0, int nout) {
        f = (tid & 15) * 4;
        na = n0 + f;
        nb = GATED ? na : na + 64;
        oka = f < nout;
        okb = GATED ? oka : f + 64 < nout;
        ba = f4_or(p.bias + na, p.bias != nullptr && oka, 0.0f);
        bb = GATED ? f4_or(p.bias_up + nb, p.bias_up != nullptr && okb, 0.0f)
                   : f4_or(p.bias + nb, p.bias != nullptr && okb, 0.0f);
        wa = f4_or(p.sw + na, F8 && oka, 1.0f);
        wb = GATED ? f4_or(p.sw_up + nb, F8 && okb, 1.0f) : f4_or(p.sw + nb, F8 && okb, 1.0f);
    }
    __device__ __forceinline__ void residual(const LinearParams& p, long long token, uint2& ra, uint2& rb) const {
        ra = rb = make_uint2(0u, 0u);
        if (p.residual) {
            const __nv_bfloat16* r = p.residual + token * p.N;
            if (oka) ra = *reinterpret_cast<const uint2*>(r + na);
            if (!GATED && okb) rb = *reinterpret_cast<const uint2*>(r + nb);
        }
    }
    // One token: its SPLIT partial sums at `part` (fp32 [128], `stride` apart) added in slice order, the
    // epilogue, the store.
    template <int SPLIT>
    __device__ __forceinline__ void finish(const LinearParams& p, const float* part, int stride, long long token,
                                           const uint2& ra, const uint2& rb) const {
        float z[8];
#pragma unroll
        for (int r = 0; r < SPLIT; ++r) {
            const float4 a = *reinterpret_cast<const float4*>(part + r * stride + f);
            const float4 b = *reinterpret_cast<const float4*>(part + r * stride + 64 + f);
            if (r == 0) {
                z[0] = a.x; z[1] = a.y; z[2] = a.z; z[3] = a.w;
                z[4] = b.x; z[5] = b.y; z[6] = b.z; z[7] = b.w;
            } else {
                z[0] += a.x; z[1] += a.y; z[2] += a.z; z[3] += a.w;
                z[4] += b.x; z[5] += b.y; z[6] += b.z; z[7] += b.w;
            }
        }
        if (F8) {
            const float sx = __ldg(p.sx + token);
            z[0] *= sx * wa.x; z[1] *= sx * wa.y; z[2] *= sx * wa.z; z[3] *= sx * wa.w;
            z[4] *= sx * wb.x; z[5] *= sx * wb.y; z[6] *= sx * wb.z; z[7] *= sx * wb.w;
        }
        z[0] += ba.x; z[1] += ba.y; z[2] += ba.z; z[3] += ba.w;
        z[4] += bb.x; z[5] += bb.y; z[6] += bb.z; z[7] += bb.w;
        if (GATED) {
#pragma unroll
            for (int i = 0; i < 4; ++i) z[i] = linear_swiglu(z[i], z[i + 4]);
        } else {
            linear_acts(p.act, z);
        }
        if (p.residual) {
            float res[8];
            bf16x4_to_f32(ra, res);
            bf16x4_to_f32(rb, res + 4);
#pragma unroll
            for (int i = 0; i < (GATED ? 4 : 8); ++i) z[i] += res[i];
        }
        __nv_bfloat16* y = p.y + token * p.N;
        if (oka) *reinterpret_cast<uint2*>(y + na) = make_uint2(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]));
        if (!GATED && okb)
            *reinterpret_cast<uint2*>(y + nb) = make_uint2(pack_bf16x2(z[4], z[5]), pack_bf16x2(z[6], z[7]));
    }
};

// The tokens [t0, t0 + ntok) of a CTA's `nout` outputs from n0, by 256 threads; partial sums at `part`
// (fp32 [slice][rows][128], slices `rows` tokens apart).
template <bool F8, bool GATED, int SPLIT>
__device__ __forceinline__ void linear_join(const LinearParams& p, const float* part, int rows, long long t0,
                                            int ntok, int n0, int nout, int tid) {
    const int stride = rows * LIN_BM;
    if ((p.N & 3) == 0) {
        LinearCols<F8, GATED> c;
        c.load(p, tid, n0, nout);
#pragma unroll 2
        for (int tok = tid >> 4; tok < ntok; tok += 16) {
            uint2 ra, rb;
            c.residual(p, t0 + tok, ra, rb);
            c.template finish<SPLIT>(p, part + tok * LIN_BM, stride, t0 + tok, ra, rb);
        }
    } else {
        // rows of y start at any 2-byte address: an output per thread
        constexpr int FT = GATED ? 64 : 128;
        constexpr int STEP = 256 / FT;
        const int f = tid % FT, n = n0 + f;
        if (f >= nout) return;
        const float ba = p.bias ? __ldg(p.bias + n) : 0.0f, bb = GATED && p.bias_up ? __ldg(p.bias_up + n) : 0.0f;
        const float wa = F8 ? __ldg(p.sw + n) : 1.0f, wb = F8 && GATED ? __ldg(p.sw_up + n) : 1.0f;
        constexpr int U = 8;                       // residuals fetched together: a store may alias the next load
        for (int tok0 = tid / FT; tok0 < ntok; tok0 += U * STEP) {
            float res[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int tok = tok0 + u * STEP;
                res[u] = p.residual && tok < ntok ? __bfloat162float(p.residual[(t0 + tok) * p.N + n]) : 0.0f;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int tok = tok0 + u * STEP;
                if (tok >= ntok) break;
                float a = part[tok * LIN_BM + f], b = GATED ? part[tok * LIN_BM + 64 + f] : 0.0f;
#pragma unroll
                for (int r = 1; r < SPLIT; ++r) {
                    a += part[r * stride + tok * LIN_BM + f];
                    if (GATED) b += part[r * stride + tok * LIN_BM + 64 + f];
                }
                if (F8) {
                    const float sx = __ldg(p.sx + t0 + tok);
                    a *= sx * wa;
                    b *= sx * wb;
                }
                a += ba;
                a = GATED ? linear_swiglu(a, b + bb) : linear_act(p.act, a);
                p.y[(t0 + tok) * p.N + n] = __float2bfloat16_rn(p.residual ? a + res[u] : a);
            }
        }
    }
}

// tcgen05 shapes: M = 128, N = bn; tensor maps: W / W_up with boxes of 128 rows (SwiGLU: 64), x with boxes of bn
// rows.  grid = tiles * split, cluster = the split CTAs of one tile.
template <bool F8, bool GATED>
__global__ void __launch_bounds__(LIN_THREADS)
linear_split_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmWup,
                    const __grid_constant__ CUtensorMap tmX, const __grid_constant__ LinearParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int S = p.stages, x_bytes = p.bn * 128;
    uint8_t* sW = smem;
    uint8_t* sX = smem + S * LIN_A_BYTES;
    // partial sums: over the ring, or (small tiles) in shared memory of their own, where another rank may
    // write them while this one's ring is still in use
    float* part = reinterpret_cast<float*>(p.own_part ? sX + S * x_bytes : smem);
    uint64_t* full_bar = reinterpret_cast<uint64_t*>(sX + S * x_bytes + (p.own_part ? linear_part_bytes(p.bn, p.split) : 0));
    uint64_t* empty_bar = full_bar + S;
    uint64_t* done_bar = empty_bar + S;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done_bar + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int tile = blockIdx.x / p.split, slice = blockIdx.x - tile * p.split;   // K slice = cluster rank
    const int m_idx = tile % p.mt, n_idx = tile / p.mt;
    constexpr int FT = GATED ? 64 : 128;           // outputs per CTA
    const int n0 = n_idx * FT;
    const int t0 = m_idx * p.bn;                   // first token
    const int ntok = min(p.bn, p.M - t0);
    constexpr int KB = F8 ? 128 : 64;              // K elements per 128-byte stage row
    const int nk = (p.K + KB - 1) / KB;
    const int kb0 = (int)((long long)nk * slice / p.split), kb1 = (int)((long long)nk * (slice + 1) / p.split);
    const int nout = min(FT, p.N - n0);
    const int own = (ntok + p.split - 1) / p.split;               // tokens joined by each slice's rank
    const int my_t0 = min(slice * own, ntok), my_ntok = min(own, ntok - my_t0);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar + s, 1);
            mbar_init(empty_bar + s, 1);
        }
        mbar_init(done_bar, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tmW);
        prefetch_tensormap(&tmX);
        if (GATED) prefetch_tensormap(&tmWup);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, p.tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    if (p.split > 1) cluster_arrive();             // waited for before the first remote store
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    grid_wait();
    grid_launch_next();

    if (warp == 0) {
        const uint64_t pol_w = p.mt == 1 ? policy_evict_first() : policy_evict_normal();
        const uint64_t pol_x = policy_evict_last();
        const uint32_t bytes = LIN_A_BYTES + (uint32_t)x_bytes;
        int s = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!mbar_wait_warp(empty_bar + s, phase ^ 1u, abort_flag)) { ok = false; break; }
            if (elect_one()) {
                mbar_arrive_expect_tx(full_bar + s, bytes);
                uint8_t* w_dst = sW + s * LIN_A_BYTES;
                tma_load_2d(w_dst, &tmW, full_bar + s, kb * KB, n0, pol_w);
                if (GATED) tma_load_2d(w_dst + 64 * 128, &tmWup, full_bar + s, kb * KB, n0, pol_w);
                tma_load_2d(sX + s * x_bytes, &tmX, full_bar + s, kb * KB, t0, pol_x);
            }
            ++issued;
            if (++s == S) { s = 0; phase ^= 1u; }
        }
        if (!ok) {
            const int n = issued < S ? issued : S;          // copies in flight land before exit
            for (int i = 1; i <= n; ++i)
                mbar_wait(full_bar + ((issued - i) % S), (uint32_t)(((issued - i) / S) & 1), nullptr);
        }
    } else if (warp == 1) {
        const uint32_t idesc = F8 ? idesc_e4m3_f32(LIN_BM, p.bn) : idesc_bf16_f32(LIN_BM, p.bn);
        const uint32_t a0 = smem_desc_lo(smem_u32(sW)), b0 = smem_desc_lo(smem_u32(sX));
        int s = 0;
        uint32_t phase = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!mbar_wait_warp(full_bar + s, phase, abort_flag)) break;
            tc_fence_after();
            if (elect_one()) {
                const uint32_t al = a0 + (uint32_t)s * (LIN_A_BYTES >> 4), bl = b0 + (uint32_t)s * (uint32_t)(x_bytes >> 4);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    umma_lo<F8, false>(tmem_base, al + 2 * kk, bl + 2 * kk, idesc, kk > 0 || kb > kb0);
                umma_commit(empty_bar + s);
            }
            if (++s == S) { s = 0; phase ^= 1u; }
        }
        if (elect_one()) umma_commit(done_bar);      // all MMAs retired: the accumulator is final, the ring is idle
    } else if (warp < 4) {
        const int tid = threadIdx.x - 64;
        if (p.residual) {                                        // a row's segment is at most 3 lines of 128 bytes
            for (int i = tid; i < my_ntok * 3; i += 64) {
                const int tok = i / 3, col = min((i - tok * 3) * 64, nout - 1);
                prefetch_l2(p.residual + (long long)(t0 + my_t0 + tok) * p.N + n0 + col);
            }
        }
        if (tid * 32 < nout) {
            if (p.bias) prefetch_l2(p.bias + n0 + tid * 32);
            if (GATED && p.bias_up) prefetch_l2(p.bias_up + n0 + tid * 32);
            if (F8) prefetch_l2(p.sw + n0 + tid * 32);
            if (F8 && GATED) prefetch_l2(p.sw_up + n0 + tid * 32);
        }
    }
    __syncwarp();
    if (p.split > 1) cluster_wait();                             // every CTA of the cluster runs
    const bool ready = __all_sync(0xffffffffu, mbar_wait(done_bar, 0, nullptr));
    if (p.split > 1 && !p.own_part) cluster_sync_all();          // every rank's ring is idle
    if (ready) {
        tc_fence_after();
        const int sub = warp & 3;
        const uint32_t tbase = tmem_base + ((uint32_t)(sub * 32) << 16);
        const uint32_t part0 = smem_u32(part) + (uint32_t)(sub * 32 + lane) * 4u;
        for (int c = (warp >> 2) * 32; c < ntok; c += 64) {      // tmem_cols is a multiple of 32
            uint32_t v[32];
            __syncwarp();
            tmem_ld_32cols(tbase + c, v);
            tmem_ld_wait();
            if (p.split == 1) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (c + j < ntok) part[(c + j) * LIN_BM + sub * 32 + lane] = __uint_as_float(v[j]);
            } else {
                int q = c / own, in_q = c - q * own;             // the owner of column c, and its place there
                uint32_t at = map_to_cta_addr(part0, (uint32_t)q) + (uint32_t)(slice * own) * (LIN_BM * 4);
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    if (c + j < ntok) st_cluster_f1(at + (uint32_t)in_q * (LIN_BM * 4), __uint_as_float(v[j]));
                    if (++in_q == own) {
                        in_q = 0;
                        ++q;
                        if (c + j + 1 < ntok)
                            at = map_to_cta_addr(part0, (uint32_t)q) + (uint32_t)(slice * own) * (LIN_BM * 4);
                    }
                }
            }
        }
        tc_fence_before();
    }
    __syncwarp();
    if (p.split > 1) cluster_sync_all();                         // all partial sums have arrived
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, p.tmem_cols);
    }
    if (my_ntok <= 0) return;
    const long long first = t0 + my_t0;
    if (p.split == 1) linear_join<F8, GATED, 1>(p, part, own, first, my_ntok, n0, nout, threadIdx.x);
    else if (p.split == 2) linear_join<F8, GATED, 2>(p, part, own, first, my_ntok, n0, nout, threadIdx.x);
    else if (p.split == 4) linear_join<F8, GATED, 4>(p, part, own, first, my_ntok, n0, nout, threadIdx.x);
    else linear_join<F8, GATED, 8>(p, part, own, first, my_ntok, n0, nout, threadIdx.x);
}

// ---------------------------------------------------------------- one or two tokens: a warp per weight rows
//
// A stream of weights with a few multiply-adds per element: four weight rows per warp (GATED: two of W and
// the same two of W_up), each 16-byte piece of a row used for every token straight from registers, four warps
// of a block along K (with 1, 2, 4, 8 of them one token takes 10.4, 8.6, 8.7, 8.7 us at 4096 x 4096, 25.2, 22.1, 20.4,
// 20.8 us at 14336 x 4096 and 15.1, 9.2, 7.4, 8.3 us at 2048 x 7168).  No tensor memory, no ring, no cluster:
// linear_split_kernel, whose tile has to be set up, drained and joined around the loads, takes 11.4, 22.7 and
// 10.6 us for these.  Narrow layers too are faster here, though N / 8 blocks leave SMs idle where the other cuts K over a
// cluster; in us, here and there, weights in L2: one token 64 x 14336 6.0, 9.8; 512 x 7168 4.0, 7.2; 1024 x 1024 2.1, 4.7; two
// tokens 64 x 14336 6.4, 9.8; SwiGLU, one token, 512 x 7168 4.4, 7.2.  It loses by 1 to 3 % for SwiGLU at 2048 x 7168 and by
// 11 % for two tokens at 14336 x 4096 (23.8, 21.4).
constexpr int LINR_THREADS = 256;
constexpr int LINR_MAX_TOKENS = 2;
constexpr int LINR_WK = 4;                          // warps along K
constexpr int LINR_GROUPS = LINR_THREADS / 32 / LINR_WK;   // and side by side along N

__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// (lo, hi) += (a.lo b.lo, a.hi b.hi): two fp32 multiply-adds in one instruction
__device__ __forceinline__ void fma2(unsigned long long& acc, unsigned long long a, unsigned long long b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}
// two bf16 as a pair of fp32
__device__ __forceinline__ unsigned long long bf16x2_pair(uint32_t w) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(w << 16), "r"(w & 0xffff0000u));
    return r;
}

template <int MT, bool GATED>
__global__ void __launch_bounds__(LINR_THREADS, 2)
linear_rows_kernel(const uint4* __restrict__ x, const uint4* __restrict__ W, const uint4* __restrict__ W_up,
                   const __grid_constant__ LinearParams p) {
    constexpr int R = 4;                            // weight rows per warp
    constexpr int RO = GATED ? 2 : 4;               // outputs per warp
    __shared__ float sums[LINR_THREADS / 32][R * MT];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = warp / LINR_WK, kw = warp - g * LINR_WK;
    const int n_block = blockIdx.x * LINR_GROUPS * RO;
    const int n0 = n_block + g * RO;
    const int nvec = p.K >> 3;
    grid_wait();
    grid_launch_next();
    // the thread that will finish an output of a token fetches its operands first
    const int ft = threadIdx.x / MT, fm = threadIdx.x - ft * MT;   // output of the block, token
    const int fn = n_block + ft;
    const bool fin = ft < LINR_GROUPS * RO && fn < p.N && fm < p.M;
    float bias = 0.0f, bias_up = 0.0f, res = 0.0f;
    if (fin) {
        if (p.bias) bias = __ldg(p.bias + fn);
        if (GATED && p.bias_up) bias_up = __ldg(p.bias_up + fn);
        if (p.residual) res = __bfloat162float(p.residual[(long long)fm * p.N + fn]);
    }
    const uint4* rows[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int n = min(n0 + (GATED ? r & 1 : r), p.N - 1);
        rows[r] = (GATED && r >= 2 ? W_up : W) + (long long)n * nvec;
    }
    const uint4* xr[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) xr[m] = x + (long long)min(m, p.M - 1) * nvec;
    unsigned long long acc[R][MT];                  // sums over even and over odd K
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[r][m] = 0ull;
    constexpr int step = LINR_WK * 32;
    for (int c = kw * 32 + lane; c - lane < nvec; c += 2 * step) {
        uint4 w[2][R];
        const bool in[2] = {c < nvec, c + step < nvec};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < R; ++r) w[h][r] = in[h] ? ld_stream(rows[r] + c + h * step) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (!in[h]) continue;
            unsigned long long f[R][4];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                f[r][0] = bf16x2_pair(w[h][r].x);
                f[r][1] = bf16x2_pair(w[h][r].y);
                f[r][2] = bf16x2_pair(w[h][r].z);
                f[r][3] = bf16x2_pair(w[h][r].w);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint4 xv = __ldg(xr[m] + c + h * step);
                const unsigned long long xf[4] = {bf16x2_pair(xv.x), bf16x2_pair(xv.y), bf16x2_pair(xv.z),
                                                  bf16x2_pair(xv.w)};
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e) fma2(acc[r][m], f[r][e], xf[e]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const float s = warp_sum(__uint_as_float((uint32_t)acc[r][m]) + __uint_as_float((uint32_t)(acc[r][m] >> 32)));
            if (lane == 0) sums[warp][r * MT + m] = s;
        }
    __syncthreads();
    if (!fin) return;
    const int fg = ft / RO, fr = ft - fg * RO;
    float a = 0.0f, b = 0.0f;
    #pragma unroll
    for (int q = 0; q < LINR_WK; ++q) {             // K order
        a += sums[fg * LINR_WK + q][fr * MT + fm];
        if (GATED) b += sums[fg * LINR_WK + q][(fr + 2) * MT + fm];
    }
    a += bias;
    a = GATED ? linear_swiglu(a, b + bias_up) : linear_act(p.act, a);
    p.y[(long long)fm * p.N + fn] = __float2bfloat16_rn(p.residual ? a + res : a);
}

// ---------------------------------------------------------------- many tokens: persistent CTA pairs
//
// Tiles of 256 weight rows x up to 256 tokens by CTA pairs (cta_group::2: each CTA holds 128 weight rows
// and half of the tokens: 32 KB of operands per 64 K-elements for 256 x 128 outputs per SM), a ring of 6 to 10
// stages and two accumulators, so that a tile's epilogue runs under the next tile's products.
// The last token tile runs its MMAs with N = its tokens rounded up to 16.
constexpr int LINP_MAX_STAGES = 10;
// 8 epilogue warps that finish 32 tokens at a time, or 16 and 16: with more warps a step's waits cost less, but rows
// are moved in smaller pieces.  By K (see launch_linear_pair).
__host__ __device__ constexpr int linear_pair_threads(int warps) { return 64 + 32 * warps; }
constexpr int LINP_EPI_BYTES = 2 * 16384;                          // two buffers per epilogue warp
constexpr int LINP_SMEM_BYTES = GEMM_SMEM_MAX;
// 128 weight rows and half of the tile's tokens; 6 stages at 256 tokens, 10 at 32
__host__ __device__ constexpr int linear_pair_stage_bytes(int bn) { return LIN_A_BYTES + bn / 2 * 128; }
__host__ __device__ constexpr int linear_pair_stages(int bn) {
    const int fit = (LINP_SMEM_BYTES - 1024 - 256 - LINP_EPI_BYTES) / linear_pair_stage_bytes(bn);
    return fit < LINP_MAX_STAGES ? fit : LINP_MAX_STAGES;
}
// Token tiles walked together: the pairs' tiles of one moment are then about 8 x 9, near the fewest distinct
// operand rows, and 8 tiles of 256 tokens stay in L2 while the weights pass by (all token tiles of M = 16384
// would not).  4 to 16 measured alike.
constexpr int LINP_GROUP = 8;

struct LinearTile {
    int t0, ntok, n_idx;
};

__device__ __forceinline__ LinearTile linear_tile(const LinearParams& p, int t, int nt) {
    const int per = LINP_GROUP * nt, g = t / per, m0 = g * LINP_GROUP;
    const int gm = min(LINP_GROUP, p.mt - m0), in = t - g * per;
    LinearTile r;
    r.n_idx = in / gm;
    r.t0 = (m0 + in - r.n_idx * gm) * p.bn;
    r.ntok = min(p.bn, p.M - r.t0);
    return r;
}

// Accumulator fragments: 16 tensor-memory lanes x CH columns (32 or 16).  v[4 i], v[4 i + 1]: lane l / 4, columns
// 8 i + 2 (l % 4), + 1; v[4 i + 2], v[4 i + 3]: lane l / 4 + 8, the same columns (l: this thread's lane).
template <int CH>
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t* v) {
    static_assert(CH == 32 || CH == 16, "");
    if constexpr (CH == 32)
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
            "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
              "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
            : "r"(taddr));
    else
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                     : "r"(taddr));
}
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// One epilogue warp's 32 accumulator lanes of a tile, CH tokens at a time.  The accumulator is read as 8 x 8
// fragments (rows: outputs, columns: tokens), finished in registers, and transposed by stmatrix into shared memory as token rows
// of 64 bytes, from which 16-byte pieces of whole rows go to y; the residual comes in the other way.  Per 8
// outputs that is 4 conversions, one shared-memory instruction each way and an eighth of a global store; with a lane
// per output each of these was 8 instructions (16384 x 2048 x 512 with residual, as first built: 61 us this way,
// 68 us a lane per output, 105 us through fp32 [token][output] in shared memory).  Pieces are XOR-swizzled
// by row: no bank conflicts.
// Rows of y that are not 16-byte aligned (N % 8) are moved an element per lane.
// GATED: lanes 0-63 of the CTA's accumulator hold x W^T, lanes 64-127 x W_up^T of the same 64 outputs.  The two
// warps of a pair swap halves of every CH tokens (through the other's buffer, two of them in turn) and each finishes
// one half.
template <bool F8, bool GATED, int CH>
struct LinearWarp {
    static constexpr int NB = GATED ? CH / 16 : CH / 8;   // blocks of 8 tokens that this warp finishes, of the chunk's CH / 8
    float bias[4], sw[4];     // of outputs l / 4 + 8 b, b = 0..3
    int n, nvalid;            // first output; how many of the 32 exist
    int own;                  // first of this warp's tokens in a chunk
    bool vec;
    uint4 rr[NB];             // residual of the next tokens: row 8 j + l / 4, piece l % 4

    __device__ __forceinline__ void begin(const LinearParams& p, int first, bool up, int lane) {
        n = first;
        nvalid = max(0, min(32, p.N - first));
        own = up ? CH / 2 : 0;
        vec = (p.N & 7) == 0;
        const float* bp = up ? p.bias_up : p.bias;
        const float* sp = up ? p.sw_up : p.sw;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int o = (lane >> 2) + 8 * b;
            bias[b] = bp && o < nvalid ? __ldg(bp + n + o) : 0.0f;
            sw[b] = F8 && o < nvalid ? __ldg(sp + n + o) : 1.0f;
        }
    }
    // cnt: tokens of the chunk that starts at `token`
    __device__ __forceinline__ void load_residual(const LinearParams& p, long long token, int cnt, int lane) {
        const int q = lane & 3;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int r = own + 8 * j + (lane >> 2);
            if (r < cnt && 8 * q < nvalid)
                rr[j] = *reinterpret_cast<const uint4*>(p.residual + (token + r) * p.N + n + 8 * q);
        }
    }
    // The residual of this warp's tokens of the chunk at `token` into its rows in shared memory; VEC: from rr, and
    // the next chunk's into rr.
    template <bool VEC>
    __device__ __forceinline__ void stage_residual(const LinearParams& p, long long token, int rows, int cnt_next,
                                                   int lane, uint8_t* mine) {
        if (VEC) {
            const int q = lane & 3;
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const int r = 8 * j + (lane >> 2);
                reinterpret_cast<uint4*>(mine)[r * 4 + (q ^ ((r >> 1) & 3))] = rr[j];
            }
            load_residual(p, token + CH, cnt_next, lane);
        } else if (nvalid > 0 && rows > 0) {      // all loads at once; masked ones repeat the last element
            const unsigned short* src = reinterpret_cast<const unsigned short*>(p.residual) + (token + own) * p.N + n +
                                        min(lane, nvalid - 1);
            unsigned short u[8 * NB];
#pragma unroll
            for (int r = 0; r < 8 * NB; ++r) u[r] = src[(long long)min(r, rows - 1) * p.N];
#pragma unroll
            for (int r = 0; r < 8 * NB; ++r)
                reinterpret_cast<unsigned short*>(mine)[r * 32 + (((lane >> 3) ^ ((r >> 1) & 3)) << 3) + (lane & 7)] = u[r];
        }
    }
    // tokens [token, token + cnt), 1 <= cnt <= CH, from the accumulator at taddr; cnt_next: tokens after them.
    // mine / other: 64 CH bytes of this warp / of its partner; bar: the pair's barrier; VEC: `vec`
    template <bool VEC>
    __device__ __forceinline__ void chunk(const LinearParams& p, uint32_t taddr, long long token, int cnt, int cnt_next,
                                          int lane, uint8_t* mine, uint8_t* other, int bar) {
        uint32_t v[CH];
        __syncwarp();
        tmem_ld_frag<CH>(taddr, v);
        tmem_ld_frag<CH>(taddr + (16u << 16), v + CH / 2);
        const int q = lane & 3;
        const int rows = min(cnt - own, 8 * NB);             // of this warp's tokens (may be <= 0)
        if (!GATED && p.residual) stage_residual<VEC>(p, token, rows, cnt_next, lane, mine);
        tmem_ld_wait();
        float z[CH];                                          // [8 i + 2 b + h]: token 8 i + 2 (l % 4) + h, output block b
#pragma unroll
        for (int i = 0; i < CH / 8; ++i) {
            float2 sx = make_float2(1.0f, 1.0f);
            if (F8) {
                const int tok = 8 * i + 2 * (lane & 3);
                if (tok < cnt) sx.x = __ldg(p.sx + token + tok);
                if (tok + 1 < cnt) sx.y = __ldg(p.sx + token + tok + 1);
            }
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float a = __uint_as_float(v[CH / 2 * (b >> 1) + 4 * i + 2 * (b & 1) + h]);
                    if (F8) a *= (h ? sx.y : sx.x) * sw[b];
                    z[8 * i + 2 * b + h] = a + bias[b];
                }
        }
        float o[8 * NB];
        if (GATED) {
            // the partner's half of the tokens goes to it, this warp's comes from it
            float4* out = reinterpret_cast<float4*>(other) + lane;
            const float4* in = reinterpret_cast<const float4*>(mine) + lane;
            const bool up = own != 0;
#pragma unroll
            for (int j = 0; j < CH / 8; ++j) {
                float4 w;
                w.x = up ? z[4 * j] : z[CH / 2 + 4 * j];
                w.y = up ? z[4 * j + 1] : z[CH / 2 + 4 * j + 1];
                w.z = up ? z[4 * j + 2] : z[CH / 2 + 4 * j + 2];
                w.w = up ? z[4 * j + 3] : z[CH / 2 + 4 * j + 3];
                out[32 * j] = w;
            }
            __syncwarp();                                     // the barrier takes whole warps
            named_barrier(bar, 64);
#pragma unroll
            for (int j = 0; j < CH / 8; ++j) {
                const float4 w = in[32 * j];
                const float r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float m = up ? z[CH / 2 + 4 * j + e] : z[4 * j + e];
                    o[4 * j + e] = linear_swiglu(up ? r[e] : m, up ? m : r[e]);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8 * NB; ++j) o[j] = z[j];
            linear_acts(p.act, o);
        }
        __syncwarp();                                         // GATED: `mine` has been read
        if (p.residual) {
            if (GATED) stage_residual<VEC>(p, token, rows, cnt_next, lane, mine);
            __syncwarp();
        }
        const uint32_t row = (uint32_t)(lane & 7), blk = (uint32_t)(lane >> 3);   // fragment addresses: row, output block
        const uint32_t frag = smem_u32(mine) + row * 64u + ((blk ^ ((row >> 1) & 3u)) << 4);
        uint32_t pk[NB][4];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            uint32_t r4[4] = {0u, 0u, 0u, 0u};
            if (p.residual) ldmatrix_x4_trans(frag + (uint32_t)i * 512u, r4);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                float lo = o[8 * i + 2 * b], hi = o[8 * i + 2 * b + 1];
                if (p.residual) {
                    lo += __uint_as_float(r4[b] << 16);
                    hi += __uint_as_float(r4[b] & 0xffff0000u);
                }
                pk[i][b] = pack_bf16x2(lo, hi);
            }
        }
        __syncwarp();                                         // the residual has been read
#pragma unroll
        for (int i = 0; i < NB; ++i) stmatrix_x4_trans(frag + (uint32_t)i * 512u, pk[i]);
        __syncwarp();
        if (VEC) {
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const int r = 8 * j + (lane >> 2);
                const uint4 w = reinterpret_cast<const uint4*>(mine)[r * 4 + (q ^ ((r >> 1) & 3))];
                if (r < rows && 8 * q < nvalid)
                    *reinterpret_cast<uint4*>(p.y + (token + own + r) * p.N + n + 8 * q) = w;
            }
        } else {
            unsigned short* dst = reinterpret_cast<unsigned short*>(p.y) + (token + own) * p.N + n + lane;
#pragma unroll
            for (int r = 0; r < 8 * NB; ++r)
                if (r < rows && lane < nvalid)
                    dst[(long long)r * p.N] = reinterpret_cast<const unsigned short*>(
                        mine)[r * 32 + (((lane >> 3) ^ ((r >> 1) & 3)) << 3) + (lane & 7)];
        }
    }
};

// Tensor maps as for linear_split_kernel, x with boxes of bn / 2 rows.
template <bool F8, bool GATED, int WARPS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(linear_pair_threads(WARPS), 1)
linear_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmWup,
                   const __grid_constant__ CUtensorMap tmX, const __grid_constant__ LinearParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int S = p.stages, x_bytes = p.bn / 2 * 128;
    uint8_t* sW = smem;
    uint8_t* sX = smem + S * LIN_A_BYTES;
    uint8_t* rows = sX + S * x_bytes;                               // the epilogue's, see LinearWarp
    uint64_t* full_bar = reinterpret_cast<uint64_t*>(rows + LINP_EPI_BYTES);
    uint64_t* empty_bar = full_bar + S;
    uint64_t* tfull_bar = empty_bar + S;
    uint64_t* tempty_bar = tfull_bar + 2;
    uint64_t* drain_bar = tempty_bar + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    constexpr int FT = GATED ? 64 : 128;           // outputs per CTA
    constexpr int KB = F8 ? 128 : 64;
    const int nk = (p.K + KB - 1) / KB;
    const int nt = (p.N + 2 * FT - 1) / (2 * FT);
    const int total = nt * p.mt;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar + s, 1);
            mbar_init(empty_bar + s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull_bar + a, 1);
            mbar_init(tempty_bar + a, 2 * WARPS);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tmW);
        prefetch_tensormap(&tmX);
        if (GATED) prefetch_tensormap(&tmWup);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, GEMM_TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    grid_wait();
    grid_launch_next();

    if (warp == 0) {
        const uint64_t pol_w = policy_evict_normal(), pol_x = policy_evict_last();
        const uint32_t full_leader = map_to_cta(full_bar, 0);
        const uint32_t bytes = 2u * (uint32_t)(LIN_A_BYTES + x_bytes);
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = pair; t < total && ok; t += npairs) {
            const LinearTile ti = linear_tile(p, t, nt);
            const int n0 = (ti.n_idx * 2 + rank) * FT;
            const int x0 = ti.t0 + rank * (((ti.ntok + 15) & ~15) >> 1);       // this CTA's half of the tokens
            for (int kb = 0; kb < nk; ++kb) {
                if (!mbar_wait_warp(empty_bar + stage, phase ^ 1u, abort_flag)) { ok = false; break; }
                if (elect_one()) {
                    const uint32_t fb = full_leader + (uint32_t)stage * 8u;
                    if (leader) mbar_arrive_expect_tx(full_bar + stage, bytes);
                    uint8_t* w_dst = sW + stage * LIN_A_BYTES;
                    tma_load_2d_pair(w_dst, &tmW, fb, kb * KB, n0, pol_w);
                    if (GATED) tma_load_2d_pair(w_dst + 64 * 128, &tmWup, fb, kb * KB, n0, pol_w);
                    tma_load_2d_pair(sX + stage * x_bytes, &tmX, fb, kb * KB, x0, pol_x);
                }
                ++issued;
                if (++stage == S) { stage = 0; phase ^= 1u; }
            }
        }
        if (!ok && leader) {
            const int n = issued < S ? issued : S;
            for (int i = 1; i <= n; ++i) {
                const int q = issued - i;
                mbar_wait(full_bar + (q % S), (uint32_t)((q / S) & 1), nullptr);
            }
        }
    } else if (warp == 1) {
        if (leader) {
            const uint32_t a0 = smem_desc_lo(smem_u32(sW)), b0 = smem_desc_lo(smem_u32(sX));
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool any = false, ok = true;
            for (int t = pair; t < total && ok; t += npairs) {
                const LinearTile ti = linear_tile(p, t, nt);
                const int n = (ti.ntok + 15) & ~15;
                const uint32_t idesc = F8 ? idesc_e4m3_f32(256, n) : idesc_bf16_f32(256, n);
                if (!mbar_wait_warp(tempty_bar + acc, acc_phase ^ 1u, abort_flag)) break;
                tc_fence_after();
                const uint32_t d = tmem_base + (uint32_t)(acc * GEMM_ACC_COLS);
                for (int kb = 0; kb < nk; ++kb) {
                    if (!mbar_wait_warp(full_bar + stage, phase, abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t al = a0 + (uint32_t)stage * (LIN_A_BYTES >> 4);
                        const uint32_t bl = b0 + (uint32_t)stage * (uint32_t)(x_bytes >> 4);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_lo<F8, true>(d, al + 2 * kk, bl + 2 * kk, idesc, kk > 0 || kb > 0);
                        umma_commit_pair(empty_bar + stage, 0x3);
                    }
                    any = true;
                    if (++stage == S) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                if (elect_one()) umma_commit_pair(tfull_bar + acc, 0x3);
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
            }
            if (any) {
                if (elect_one()) umma_commit_pair(drain_bar, 0x1);
                __syncwarp();
                mbar_wait(drain_bar, 0, nullptr);
            }
        }
    } else {
        // the WARPS / 4 warps of a lane quarter share the tokens; GATED: lane quarters q and q + 2 are partners
        constexpr int CH = 256 / WARPS;                             // tokens of a step
        const int sub = warp & 3, slot = (warp - 2) >> 2;
        const int part = GATED ? sub & 1 : sub;                     // 32 outputs of the CTA
        const bool up = GATED && sub >= 2;
        const int bar = 1 + part + 2 * slot;                     // GATED: the pair's barrier
        const int tid = threadIdx.x - 64;
        uint8_t* mine = rows + (sub + 4 * slot) * (64 * CH);       // the second set 16 KB further on
        uint8_t* other = rows + ((sub ^ 2) + 4 * slot) * (64 * CH);
        const uint32_t tempty_leader = map_to_cta(tempty_bar, 0);
        int acc = 0;
        uint32_t acc_phase = 0, turn = 0;
        for (int t = pair; t < total; t += npairs) {
            const LinearTile ti = linear_tile(p, t, nt);
            const int n0 = (ti.n_idx * 2 + rank) * FT, nout = min(FT, p.N - n0);
            const int share = (p.bn / (WARPS / 4) + CH - 1) / CH * CH;
            const int c0 = slot * share, c1 = min(c0 + share, ti.ntok);
            LinearWarp<F8, GATED, CH> e;
            e.begin(p, n0 + part * 32, up, lane);
            if (p.residual && e.vec && c0 < c1) e.load_residual(p, ti.t0 + c0, c1 - c0, lane);
            if (p.residual && nout > 0) {
                for (int i = tid; i < ti.ntok * 3; i += 32 * WARPS) {   // a row's piece is at most 3 lines
                    const int tok = i / 3, col = min((i - tok * 3) * 64, nout - 1);
                    prefetch_l2(p.residual + (long long)(ti.t0 + tok) * p.N + n0 + col);
                }
            }
            // all lanes leave the wait together: the barrier behind it takes whole warps
            bool ready = mbar_wait_warp(tfull_bar + acc, acc_phase, abort_flag);
            if (GATED) {
                __syncwarp();
                ready = named_barrier_all(bar, 64, ready);           // both partners go on, or neither
            }
            if (!__all_sync(0xffffffffu, ready)) break;
            tc_fence_after();
            const uint32_t tb = tmem_base + (uint32_t)(acc * GEMM_ACC_COLS) + ((uint32_t)(sub * 32) << 16);
            for (int c = c0; c < c1; c += CH) {
                const uint32_t set = (turn & 1u) * 16384u;
                if (e.vec)
                    e.template chunk<true>(p, tb + c, ti.t0 + c, min(CH, c1 - c), c1 - c - CH, lane, mine + set,
                                           other + set, bar);
                else
                    e.template chunk<false>(p, tb + c, ti.t0 + c, min(CH, c1 - c), c1 - c - CH, lane, mine + set,
                                            other + set, bar);
                ++turn;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(tempty_leader + (uint32_t)acc * 8u);
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
    }

    __syncthreads();
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, GEMM_TMEM_COLS);
    }
}

}  // namespace moe
