// linear.cuh - the dense layer y = act(x W^T + bias) + residual on the tcgen05 tensor cores.
//
// x [M, K] (M tokens), W [N, K], both K-major; y [M, N] bf16.  MOE_ACT_SWIGLU: y = silu(x W^T + bias) *
// (x W_up^T + bias_up) + residual.  F8: e4m3 x (one scale per token) and W (one scale per output),
// the fp32 accumulator multiplied by both.  Everything between the product and the one rounding to
// bf16 is in fp32.
//
// linear_split_kernel: the weights are the MMA's M side (D^T = W x^T): a tile is 128 weight rows by
// `bn` tokens (a multiple of 16, at most 256), so a single token costs no padded 128-row tile, and the
// K range of a tile is cut over the CTAs of a cluster, which join their partial sums through
// distributed shared memory in rank order: no workspace, no atomics, the same result every time.
// SwiGLU tiles take 64 rows of W and the same 64 rows of W_up.
//
// Warp roles (192 threads): warp 0 TMA producer, warp 1 tensor memory + MMA issuer, warps 2-5 move the
// accumulator to shared memory (over the ring, idle by then) as fp32 [token][128]; then all threads
// add the partial sums, apply the epilogue and store 16 bytes (8 outputs of a token) at a time.
#pragma once

#include "grouped_gemm.cuh"
#include "route_permute_combine.cuh"

namespace moe {

enum { LIN_NONE = 0, LIN_RELU = 1, LIN_SILU = 2, LIN_GELU = 3, LIN_GELU_TANH = 4, LIN_SWIGLU = 5 };

constexpr int LIN_BM = 128;                        // weight rows per tile
constexpr int LIN_A_BYTES = LIN_BM * 128;          // one stage of weights: 128-byte rows
constexpr int LIN_THREADS = 192;
constexpr int LIN_MAX_STAGES = 8;
constexpr int LIN_MAX_SPLIT = 8;                   // portable cluster size

struct LinearParams {
    int M, N, K;
    int bn;        // tokens per tile
    int mt;        // token tiles
    int stages, split;
    int tmem_cols; // power of two >= max(bn, 32)
    int act;
    const float *bias, *bias_up;
    const __nv_bfloat16* residual;
    __nv_bfloat16* y;
    const float *sx, *sw, *sw_up;                  // F8 scales
};

__host__ __device__ constexpr int linear_smem_bytes(int stages, int bn) {
    return stages * (LIN_A_BYTES + bn * 128) + 1024 + 256;
}

// Activation of a pre-activation z (not SwiGLU).  gelu: z times the normal distribution function,
// through erfc so that its tail keeps its relative precision; gelu_tanh: (1 + tanh u) / 2 =
// sigmoid(2u) for the same reason.  The fast exponential and divide are a few ulp of fp32 off, far
// below the bf16 rounding that follows.  relu keeps NaN.
__device__ __forceinline__ float linear_act(int act, float z) {
    switch (act) {
        case LIN_RELU: return z < 0.0f ? 0.0f : z;
        case LIN_SILU: return __fdividef(z, 1.0f + __expf(-z));
        case LIN_GELU: return 0.5f * z * erfcf(-0.70710678118654752f * z);
        case LIN_GELU_TANH: return __fdividef(z, 1.0f + __expf(-1.5957691216057308f * fmaf(0.044715f * z * z, z, z)));
        default: return z;
    }
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ float ld_cluster_f1(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// tcgen05 shapes: M = 128, N = bn; tensor maps: W / W_up with boxes of 128 rows (SwiGLU: 64), x with
// boxes of bn rows.  grid = tiles * split, cluster = split CTAs of one tile.
template <bool F8, bool GATED>
__global__ void __launch_bounds__(LIN_THREADS)
linear_split_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmWup,
                    const __grid_constant__ CUtensorMap tmX, const __grid_constant__ LinearParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int S = p.stages, x_bytes = p.bn * 128;
    uint8_t* sW = smem;
    uint8_t* sX = smem + S * LIN_A_BYTES;
    uint64_t* full_bar = reinterpret_cast<uint64_t*>(sX + S * x_bytes);
    uint64_t* empty_bar = full_bar + S;
    uint64_t* done_bar = empty_bar + S;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done_bar + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = blockIdx.x / p.split, rank = blockIdx.x - tile * p.split;
    const int m_idx = tile % p.mt, n_idx = tile / p.mt;
    constexpr int FT = GATED ? 64 : 128;           // outputs per tile
    const int n0 = n_idx * FT;
    const int t0 = m_idx * p.bn;                   // first token
    const int ntok = min(p.bn, p.M - t0);
    constexpr int KB = F8 ? 128 : 64;              // K elements per 128-byte stage row
    const int nk = (p.K + KB - 1) / KB;
    const int kb0 = (int)((long long)nk * rank / p.split), kb1 = (int)((long long)nk * (rank + 1) / p.split);

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
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol_w = p.mt == 1 ? policy_evict_first() : policy_evict_normal();
            const uint64_t pol_x = policy_evict_last();
            const uint32_t bytes = LIN_A_BYTES + (uint32_t)x_bytes;
            int issued = 0;
            bool ok = true;
            for (int kb = kb0; kb < kb1; ++kb) {
                const int s = issued % S;
                if (!mbar_wait(empty_bar + s, ((issued / S) & 1) ^ 1u, abort_flag)) { ok = false; break; }
                mbar_arrive_expect_tx(full_bar + s, bytes);
                uint8_t* w_dst = sW + s * LIN_A_BYTES;
                tma_load_2d(w_dst, &tmW, full_bar + s, kb * KB, n0, pol_w);
                if (GATED) tma_load_2d(w_dst + 64 * 128, &tmWup, full_bar + s, kb * KB, n0, pol_w);
                tma_load_2d(sX + s * x_bytes, &tmX, full_bar + s, kb * KB, t0, pol_x);
                ++issued;
            }
            if (!ok) {
                const int n = issued < S ? issued : S;      // copies in flight land before exit
                for (int i = 1; i <= n; ++i)
                    mbar_wait(full_bar + ((issued - i) % S), (uint32_t)(((issued - i) / S) & 1), nullptr);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = F8 ? idesc_e4m3_f32(LIN_BM, p.bn) : idesc_bf16_f32(LIN_BM, p.bn);
            for (int kb = kb0, i = 0; kb < kb1; ++kb, ++i) {
                const int s = i % S;
                if (!mbar_wait(full_bar + s, (i / S) & 1, abort_flag)) break;
                tc_fence_after();
                const uint64_t ad = smem_desc_k_sw128(sW + s * LIN_A_BYTES);
                const uint64_t bd = smem_desc_k_sw128(sX + s * x_bytes);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    if (F8) umma_e4m3(tmem_base, ad + 2ull * kk, bd + 2ull * kk, idesc, (i | kk) != 0);
                    else umma_bf16(tmem_base, ad + 2ull * kk, bd + 2ull * kk, idesc, (i | kk) != 0);
                }
                umma_commit(empty_bar + s);
            }
            umma_commit(done_bar);       // all MMAs retired: the accumulator is final, the ring is idle
            mbar_wait(done_bar, 0, nullptr);
        }
    } else {
        const bool ready = mbar_wait(done_bar, 0, nullptr);
        if (__all_sync(0xffffffffu, ready)) {
            tc_fence_after();
            const int sub = warp & 3;
            float* stage = reinterpret_cast<float*>(smem);
            const uint32_t tbase = tmem_base + ((uint32_t)(sub * 32) << 16);
            for (int c = 0; c < ntok; c += 32) {            // tmem_cols is a multiple of 32
                uint32_t v[32];
                __syncwarp();
                tmem_ld_32cols(tbase + c, v);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (c + j < ntok) stage[(c + j) * LIN_BM + sub * 32 + lane] = __uint_as_float(v[j]);
            }
            tc_fence_before();
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, p.tmem_cols);
    }
    if (p.split > 1) cluster_sync_all();                     // every rank's partial sums are staged

    // ---- join the ranks' sums, epilogue, store: rank r takes an equal share of the tile's units
    const uint32_t stage0 = smem_u32(smem);
    auto peer = [&](int r) {
        uint32_t a;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(stage0), "r"(r));
        return a;
    };
    const int nout = min(FT, p.N - n0);
    if ((p.N & 7) == 0) {
        const int per_tok = nout >> 3;                       // units of 8 outputs of a token
        const int units = ntok * per_tok;
        const int u0 = (int)((long long)units * rank / p.split), u1 = (int)((long long)units * (rank + 1) / p.split);
        for (int u = u0 + threadIdx.x; u < u1; u += LIN_THREADS) {
            const int tok = u / per_tok, f = (u - tok * per_tok) * 8;
            const long long row = t0 + tok;
            float z[8], up[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = up[i] = 0.0f;
            for (int r = 0; r < p.split; ++r) {
                const uint32_t a = peer(r) + (uint32_t)(tok * LIN_BM + f) * 4u;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float4 v = ld_cluster_f4(a + 16 * h);
                    z[4 * h] += v.x; z[4 * h + 1] += v.y; z[4 * h + 2] += v.z; z[4 * h + 3] += v.w;
                    if (GATED) {
                        const float4 q = ld_cluster_f4(a + 256 + 16 * h);
                        up[4 * h] += q.x; up[4 * h + 1] += q.y; up[4 * h + 2] += q.z; up[4 * h + 3] += q.w;
                    }
                }
            }
            const int n = n0 + f;
            const float sx = F8 ? __ldg(p.sx + row) : 1.0f;
            float res[8];
            if (p.residual) bf16x8_to_f32(*reinterpret_cast<const uint4*>(p.residual + row * p.N + n), res);
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float a = z[i];
                if (F8) a *= sx * __ldg(p.sw + n + i);
                if (p.bias) a += __ldg(p.bias + n + i);
                if (GATED) {
                    float b = up[i];
                    if (F8) b *= sx * __ldg(p.sw_up + n + i);
                    if (p.bias_up) b += __ldg(p.bias_up + n + i);
                    a = swiglu_f32(a, b);
                } else {
                    a = linear_act(p.act, a);
                }
                o[i] = p.residual ? a + res[i] : a;
            }
            *reinterpret_cast<uint4*>(p.y + row * p.N + n) =
                make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]),
                           pack_bf16x2(o[6], o[7]));
        }
    } else {
        const int units = ntok * nout;                       // output rows start at any 2-byte address
        const int u0 = (int)((long long)units * rank / p.split), u1 = (int)((long long)units * (rank + 1) / p.split);
        for (int u = u0 + threadIdx.x; u < u1; u += LIN_THREADS) {
            const int tok = u / nout, f = u - tok * nout;
            const long long row = t0 + tok;
            const int n = n0 + f;
            float a = 0.0f, b = 0.0f;
            for (int r = 0; r < p.split; ++r) {
                const uint32_t q = peer(r) + (uint32_t)(tok * LIN_BM + f) * 4u;
                a += ld_cluster_f1(q);
                if (GATED) b += ld_cluster_f1(q + 256);
            }
            const float sx = F8 ? __ldg(p.sx + row) : 1.0f;
            if (F8) a *= sx * __ldg(p.sw + n);
            if (p.bias) a += __ldg(p.bias + n);
            if (GATED) {
                if (F8) b *= sx * __ldg(p.sw_up + n);
                if (p.bias_up) b += __ldg(p.bias_up + n);
                a = swiglu_f32(a, b);
            } else {
                a = linear_act(p.act, a);
            }
            if (p.residual) a += __bfloat162float(p.residual[row * p.N + n]);
            p.y[row * p.N + n] = __float2bfloat16_rn(a);
        }
    }
    __syncwarp();
    if (p.split > 1) cluster_sync_all();                     // no peer reads this CTA's shared memory any more
}

}  // namespace moe
