// Softmax cross entropy over the int8 table (the tied embedding / LM head) and its gradient with
// respect to the hidden state, without keeping the logits.
//
// The hidden state comes in the layer's int8 form (q, s_x):
//   l[t, v] = s_x[t] s[v] sum_j E[v, j] q[t, j];  lse[t] = log sum_v exp l[t, v]
//   nll[t]  = lse[t] - l[t, target];  a target of DFSSM_IGNORE_TARGET gives 0
//   dh[t]   = grad[t] (sum_v exp(l[t, v] - lse[t]) s[v] E[v] - s[target] E[target])
//
// Both directions need the logits once: 2 m V d int8 operations, on the 5th-generation tensor
// cores. xent_logits_kernel computes them tile by tile (128 tokens x 256 rows of the table, one
// tcgen05 accumulator, int32, exact) and consumes each tile from TMEM while the next one is
// multiplied:
//   kLse   one thread holds one token's row of the tile: running maximum and sum of 2^(l log2 e -
//          max) over 128 columns, one (max, sum) pair per token and half tile to the workspace;
//          xent_lse_kernel joins the pairs of a token and takes the target's logit by a dp4a dot;
//   kGrad  g = exp(l - lse) s[v] K as fp16 to the workspace, for a piece of the vocabulary.
// xent_dh_kernel multiplies such a piece with its rows of the table (kind::f16): the table's
// bytes go through registers, where eight rows x four columns become four 16-byte pieces along K
// (prmt, lop3 and one packed subtraction make an exact fp16 integer of a byte), so the table is
// read as int8 and never stored in a wider form. Partial sums stay in fp32; xent_dh_out_kernel
// adds the splits in order, takes the target's row off in fp32, scales by grad and rounds to bf16.
//
// fp16, not bf16, for g: it only rounds once to 11 bits (2^-12 of the value), and K, a power of
// two with max |s| K in [2^13, 2^14), keeps exp(l - lse) s[v] K below 2^14 and its smallest
// kept step at 2^-38 max |s|, far below what bf16 output can show. Every order is fixed.
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "dfssm_internal.cuh"
#include "epilogue.cuh"
#include "ptx.cuh"

namespace dfssm {

namespace {

constexpr int kBM = 128;                 // tokens per tile (TMEM lanes)
constexpr int kBN = 256;                 // table rows (logits) or channels (gradient) per tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// -- logits kernel
constexpr int kLgStages = 4;
constexpr int kLgA = kBM * 128, kLgB = kBN * 128, kLgStage = kLgA + kLgB;     // 128 K bytes per stage
constexpr int kLgThreads = 12 * 32;      // TMA, MMA, 2 idle warps; 8 epilogue warps
constexpr int kLgEpi = 256;
constexpr int kLgSmem = kLgStages * kLgStage + 2 * kBN * 4 + 256 + 1024;

// -- gradient kernel
constexpr int kDhStages = 4;
constexpr int kDhA = kBM * 128, kDhB = kBN * 128, kDhStage = kDhA + kDhB;     // 64 K values per stage
constexpr int kDhConv = 256;             // converter threads (8 warps), the epilogue afterwards
constexpr int kDhThreads = 4 * 32 + kDhConv;
constexpr int kDhSmem = kDhStages * kDhStage + 256 + 1024;

constexpr int kTokBlock = 2048;          // tokens whose gradient is worked on at a time
constexpr size_t kGradBytes = 80u << 20; // about the fp16 piece that stays in the 126 MB L2

struct LogitsArgs {
    const float* scale;
    const float* sx;
    int vocab, d, m;
    int v0, v_end;                       // table rows of this call (a multiple of kBN at v0)
    float2* part;                        // kLse: [2 * v tiles][m]
    const float* lse;                    // kGrad
    const int32_t* targets;              // kGrad
    const uint32_t* smax;                // kGrad: bits of max |scale|
    __half* g;                           // kGrad: [m][ldg]
    int ldg;
    uint32_t* err;
};

__device__ __forceinline__ bool is_token(int target, int vocab) { return target >= 0 && target < vocab; }

// the power of two K of the fp16 gradients: max |scale| K lies in [2^13, 2^14)
__device__ __forceinline__ float grad_scale(uint32_t smax_bits) {
    const int e = (int)(smax_bits >> 23) - 127;          // floor log2 (a zero or denormal maximum: -127)
    const int k = 13 - e;
    return __int_as_float((min(max(k, -126), 127) + 127) << 23);
}

__device__ __forceinline__ void give_up(uint32_t* err, volatile uint32_t* flag) {
    atomicOr(err, DFSSM_DEVERR_TIMEOUT);
    *flag = 1;
}

enum { kLse = 0, kGrad = 1 };

template <int MODE>
__global__ void __launch_bounds__(kLgThreads, 1)
xent_logits_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_e,
                   const LogitsArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    float* s_scale = reinterpret_cast<float*>(smem + kLgStages * kLgStage);          // [2][kBN]
    uint64_t* full = reinterpret_cast<uint64_t*>(s_scale + 2 * kBN);                 // TMA bytes
    uint64_t* empty = full + kLgStages;                                              // MMA commit
    uint64_t* acc_full = empty + kLgStages;                                          // [2] MMA commit
    uint64_t* acc_empty = acc_full + 2;                                              // [2] epilogue threads
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_tt = (a.m + kBM - 1) / kBM;
    const int n_tiles = n_tt * ((a.v_end - a.v0 + kBN - 1) / kBN);
    const int n_k = (a.d + 127) / 128;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kLgStages; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(&acc_full[b], 1);
            ptx::mbar_init(&acc_empty[b], kLgEpi);
        }
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(tmem_slot, 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            for (int tile = blockIdx.x; tile < n_tiles && !*abort_flag; tile += gridDim.x) {
                const int vt = tile / n_tt, tt = tile - vt * n_tt;
                for (int k = 0; k < n_k; ++k, ++it) {
                    const int s = it % kLgStages;
                    if (!ptx::mbar_wait(&empty[s], ((uint32_t)(it / kLgStages) & 1u) ^ 1u)) {
                        give_up(a.err, abort_flag);
                        break;
                    }
                    uint8_t* st = smem + s * kLgStage;
                    ptx::mbar_arrive_expect_tx(&full[s], kLgStage);
                    ptx::tma_load_2d(st, &map_q, k * 128, tt * kBM, &full[s]);
                    ptx::tma_load_2d(st + kLgA, &map_e, k * 128, a.v0 + vt * kBN, &full[s]);
                }
            }
            // after a wait that gave up: the copies still in flight land before the CTA ends
            if (*abort_flag)
                for (int i = max(0, it - kLgStages); i < it; ++i)
                    ptx::mbar_wait(&full[i % kLgStages], (uint32_t)(i / kLgStages) & 1u);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // kind::i8: D s32, A and B s8, both K-major
            constexpr uint32_t idesc = (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kBN >> 3) << 17) |
                                       ((uint32_t)(kBM >> 4) << 24);
            int it = 0, tc = 0;
            bool ok = true;
            for (int tile = blockIdx.x; tile < n_tiles && ok && !*abort_flag; tile += gridDim.x, ++tc) {
                const int buf = tc & 1;
                if (!ptx::mbar_wait(&acc_empty[buf], ((uint32_t)(tc >> 1) & 1u) ^ 1u)) {
                    give_up(a.err, abort_flag);
                    break;
                }
                ptx::tc_fence_after();
                for (int k = 0; k < n_k; ++k, ++it) {
                    const int s = it % kLgStages;
                    if (!ptx::mbar_wait(&full[s], (uint32_t)(it / kLgStages) & 1u)) {
                        give_up(a.err, abort_flag);
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint64_t ad = ptx::kmajor_sw128_desc(ptx::smem_u32(smem + s * kLgStage));
                    const uint64_t bd = ptx::kmajor_sw128_desc(ptx::smem_u32(smem + s * kLgStage + kLgA));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        ptx::mma_i8(tmem + (uint32_t)(buf * kBN), ad + 2 * kk, bd + 2 * kk, idesc, (k | kk) != 0);
                    ptx::mma_commit(&empty[s]);
                }
                if (ok) ptx::mma_commit(&acc_full[buf]);
            }
            if (*abort_flag)           // the MMAs issued so far complete before TMEM is given back
                for (int i = max(0, it - kLgStages); i < it; ++i)
                    ptx::mbar_wait(&empty[i % kLgStages], (uint32_t)(i / kLgStages) & 1u);
        }
    } else if (warp >= 4) {
        const int e = threadIdx.x - 4 * 32, q4 = warp & 3, half = (warp - 4) >> 2;
        float gk = 0.0f;
        if (MODE == kGrad) gk = grad_scale(*a.smax);
        int tc = 0;
        bool got = true;
        for (int tile = blockIdx.x; tile < n_tiles; tile += gridDim.x, ++tc) {
            const int vt = tile / n_tt, tt = tile - vt * n_tt;
            const int buf = tc & 1;
            const int vbase = a.v0 + vt * kBN;
            float* sc = s_scale + buf * kBN;
            sc[e] = vbase + e < a.v_end ? a.scale[vbase + e] : 0.0f;
            const int t = tt * kBM + 32 * q4 + lane;
            const bool live = t < a.m;
            const float k2 = live ? __fmul_rn(a.sx[t], kLog2e) : 0.0f;      // logits in units of log 2
            float lse2 = 0.0f;
            bool counted = live;
            if (MODE == kGrad) {
                counted = live && is_token(a.targets[t], a.vocab);
                lse2 = live ? __fmul_rn(a.lse[t], kLog2e) : 0.0f;
            }
            // the scales are there, and the last tile's are done with; a warp that gave up takes all along
            if (ptx::named_barrier_or(1, kLgEpi, !got)) break;
            if (lane == 0) got = ptx::mbar_wait(&acc_full[buf], (uint32_t)(tc >> 1) & 1u);
            got = __shfl_sync(0xffffffffu, got, 0);
            if (!got) {
                if (lane == 0) give_up(a.err, abort_flag);
                continue;
            }
            ptx::tc_fence_after();
            float mx = -INFINITY, sum = 0.0f;
            const int c_end = min(kBN / 2, a.v_end - vbase - half * (kBN / 2));     // live columns of this half
#pragma unroll 1
            for (int c = 0; c < kBN / 2; c += 32) {
                const int col = half * (kBN / 2) + c;
                uint32_t r[32];
                ptx::tmem_ld_32x32b_x32(tmem + (uint32_t)(buf * kBN + col) + ((uint32_t)(32 * q4) << 16), r);
                ptx::tmem_ld_wait();
                if (c + 32 == kBN / 2) {           // the last read of this accumulator
                    ptx::tc_fence_before();
                    ptx::mbar_arrive(&acc_empty[buf]);
                }
                float z[32];
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 s4 = *reinterpret_cast<const float4*>(sc + col + i);
                    z[i] = __fmul_rn(__fmul_rn((float)(int)r[i], s4.x), k2);
                    z[i + 1] = __fmul_rn(__fmul_rn((float)(int)r[i + 1], s4.y), k2);
                    z[i + 2] = __fmul_rn(__fmul_rn((float)(int)r[i + 2], s4.z), k2);
                    z[i + 3] = __fmul_rn(__fmul_rn((float)(int)r[i + 3], s4.w), k2);
                }
                if (MODE == kLse) {
                    if (c + 32 > c_end) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (c + i >= c_end) z[i] = -INFINITY;
                    }
                    float cm = mx;
#pragma unroll
                    for (int i = 0; i < 32; ++i) cm = fmaxf(cm, z[i]);
                    const float ref = cm == -INFINITY ? 0.0f : cm;       // no live column yet: 2^(-inf - 0) = 0
                    float s0 = __fmul_rn(sum, exp2f(__fsub_rn(mx, ref))), s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        s0 = __fadd_rn(s0, exp2f(__fsub_rn(z[i], ref)));
                        s1 = __fadd_rn(s1, exp2f(__fsub_rn(z[i + 1], ref)));
                        s2 = __fadd_rn(s2, exp2f(__fsub_rn(z[i + 2], ref)));
                        s3 = __fadd_rn(s3, exp2f(__fsub_rn(z[i + 3], ref)));
                    }
                    sum = __fadd_rn(__fadd_rn(s0, s1), __fadd_rn(s2, s3));
                    mx = cm;
                } else if (live) {
                    uint32_t o[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float f0 = __fmul_rn(sc[col + i], gk), f1 = __fmul_rn(sc[col + i + 1], gk);
                        const float g0 = counted && c + i < c_end ? __fmul_rn(exp2f(__fsub_rn(z[i], lse2)), f0) : 0.0f;
                        const float g1 =
                            counted && c + i + 1 < c_end ? __fmul_rn(exp2f(__fsub_rn(z[i + 1], lse2)), f1) : 0.0f;
                        const __half2 h = __floats2half2_rn(g0, g1);
                        o[i / 2] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                    uint4* dst = reinterpret_cast<uint4*>(a.g + (int64_t)t * a.ldg + vt * kBN + col);
#pragma unroll
                    for (int i = 0; i < 4; ++i) dst[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                }
            }
            if (MODE == kLse && live) a.part[(int64_t)(2 * vt + half) * a.m + t] = make_float2(mx, sum);
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// One warp per token: joins the token's (max, sum) pairs, lane i taking pairs i, i + 32, ... in
// order, then a shuffle tree; the target's logit from an int32 dot product.
__global__ void __launch_bounds__(256) xent_lse_kernel(const float2* __restrict__ part, int n_part,
                                                       const int8_t* __restrict__ table,
                                                       const float* __restrict__ scale, int vocab, int d,
                                                       const int8_t* __restrict__ q, const float* __restrict__ sx,
                                                       const int32_t* __restrict__ targets, int m, float* nll,
                                                       float* lse_out, uint32_t* err) {
    const int t = (int)((blockIdx.x * blockDim.x + threadIdx.x) >> 5), lane = threadIdx.x & 31;
    if (t >= m) return;
    float mx = -INFINITY, sum = 0.0f;
    auto join = [&](float m2, float s2) {
        const float nm = fmaxf(mx, m2);
        const float ref = nm == -INFINITY ? 0.0f : nm;
        sum = __fadd_rn(__fmul_rn(sum, exp2f(__fsub_rn(mx, ref))), __fmul_rn(s2, exp2f(__fsub_rn(m2, ref))));
        mx = nm;
    };
    for (int i = lane; i < n_part; i += 32) {
        const float2 p = part[(int64_t)i * m + t];
        join(p.x, p.y);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, mx, o), s2 = __shfl_xor_sync(0xffffffffu, sum, o);
        join(m2, s2);
    }
    const float lse = __fmul_rn(__fadd_rn(mx, log2f(sum)), kLn2);
    const int tg = targets[t];
    float loss = 0.0f;
    if (is_token(tg, vocab)) {
        const uint4* ep = reinterpret_cast<const uint4*>(table + (int64_t)tg * d);
        const uint4* qp = reinterpret_cast<const uint4*>(q + (int64_t)t * d);
        int acc = 0;
        for (int i = lane; i < (d >> 4); i += 32) {
            const uint4 x = ep[i], y = qp[i];
            acc = __dp4a((int)x.x, (int)y.x, acc);
            acc = __dp4a((int)x.y, (int)y.y, acc);
            acc = __dp4a((int)x.z, (int)y.z, acc);
            acc = __dp4a((int)x.w, (int)y.w, acc);
        }
        acc = __reduce_add_sync(0xffffffffu, acc);
        loss = __fsub_rn(lse, __fmul_rn(sx[t], __fmul_rn(scale[tg], (float)acc)));
    } else if (tg != DFSSM_IGNORE_TARGET && lane == 0) {
        atomicOr(err, DFSSM_DEVERR_TOKEN_ID);
    }
    if (lane == 0) {
        nll[t] = loss;
        lse_out[t] = lse;
    }
}

// max |scale| as bits (one CTA)
__global__ void __launch_bounds__(1024) xent_smax_kernel(const float* __restrict__ scale, int vocab, uint32_t* out) {
    __shared__ uint32_t red[32];
    uint32_t v = 0u;
    const int n4 = vocab >> 2;
    for (int i = threadIdx.x; i < n4; i += 1024) {
        const uint4 x = reinterpret_cast<const uint4*>(scale)[i];
        v = max(max(max(x.x & 0x7FFFFFFFu, x.y & 0x7FFFFFFFu), max(x.z & 0x7FFFFFFFu, x.w & 0x7FFFFFFFu)), v);
    }
    if (threadIdx.x < (vocab & 3)) v = max(v, __float_as_uint(scale[4 * n4 + threadIdx.x]) & 0x7FFFFFFFu);
    v = __reduce_max_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        v = __reduce_max_sync(0xffffffffu, red[threadIdx.x]);
        if (threadIdx.x == 0) *out = v;
    }
}

// ------------------------------------------------------------------------------- gradient

struct DhArgs {
    const int8_t* table;
    int d, m;
    int v0, k_total;        // table row of the piece's column 0; its live columns
    int k_split;            // columns per split (a multiple of 64)
    float* part;            // [splits][m][d]
    int add;                // 1: add to part (a later piece), 0: write it
    uint32_t* err;
};

// CTA (split, channel tile, token tile). Warp 0 loads the fp16 gradients by TMA, warps 4..11 turn the
// table's bytes into the B operand and write the accumulator out afterwards, warp 1 issues the MMAs.
__global__ void __launch_bounds__(kDhThreads, 1)
xent_dh_kernel(const __grid_constant__ CUtensorMap map_g, const DhArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* full_a = reinterpret_cast<uint64_t*>(smem + kDhStages * kDhStage);     // TMA bytes
    uint64_t* full_b = full_a + kDhStages;                                           // kDhConv arrivals
    uint64_t* empty = full_b + kDhStages;                                            // MMA commit
    uint64_t* acc_full = empty + kDhStages;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tok0 = blockIdx.x * kBM, c0 = blockIdx.y * kBN, sp = blockIdx.z;
    const int k0 = sp * a.k_split;
    const int k_end = min(a.k_total, k0 + a.k_split);
    const int n_k = k_end > k0 ? (k_end - k0 + 63) / 64 : 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kDhStages; ++s) {
            ptx::mbar_init(&full_a[s], 1);
            ptx::mbar_init(&full_b[s], kDhConv);
            ptx::mbar_init(&empty[s], 1);
        }
        ptx::mbar_init(acc_full, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(tmem_slot, 256);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            int k = 0;
            for (; k < n_k && !*abort_flag; ++k) {
                const int s = k % kDhStages;
                if (!ptx::mbar_wait(&empty[s], ((uint32_t)(k / kDhStages) & 1u) ^ 1u)) {
                    give_up(a.err, abort_flag);
                    break;
                }
                ptx::mbar_arrive_expect_tx(&full_a[s], kDhA);
                ptx::tma_load_2d(smem + s * kDhStage, &map_g, k0 + 64 * k, tok0, &full_a[s]);
            }
            if (*abort_flag)
                for (int i = max(0, k - kDhStages); i < k; ++i)
                    ptx::mbar_wait(&full_a[i % kDhStages], (uint32_t)(i / kDhStages) & 1u);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // kind::f16: D fp32, A and B fp16, both K-major
            constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(kBN >> 3) << 17) | ((uint32_t)(kBM >> 4) << 24);
            int k = 0;
            for (; k < n_k && !*abort_flag; ++k) {
                const int s = k % kDhStages;
                const uint32_t ph = (uint32_t)(k / kDhStages) & 1u;
                if (!ptx::mbar_wait(&full_a[s], ph) || !ptx::mbar_wait(&full_b[s], ph)) {
                    give_up(a.err, abort_flag);
                    break;
                }
                ptx::tc_fence_after();
                const uint64_t ad = ptx::kmajor_sw128_desc(ptx::smem_u32(smem + s * kDhStage));
                const uint64_t bd = ptx::kmajor_sw128_desc(ptx::smem_u32(smem + s * kDhStage + kDhA));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) ptx::mma_f16(tmem, ad + 2 * kk, bd + 2 * kk, idesc, (k | kk) != 0);
                ptx::mma_commit(&empty[s]);
            }
            if (!*abort_flag) ptx::mma_commit(acc_full);
            else
                for (int i = max(0, k - kDhStages); i < k; ++i)
                    ptx::mbar_wait(&empty[i % kDhStages], (uint32_t)(i / kDhStages) & 1u);
        }
    } else if (warp >= 4) {
        // Converter: a warp's unit is 8 table rows (K) x 128 channels, lane l the channels 4 l .. 4 l + 3;
        // warp w takes K rows 8 w .. 8 w + 7 of the stage, both channel halves. A 16-byte piece holds
        // one channel's 8 K values: row n, piece w ^ (n & 7) of the 128-byte swizzle. Lane l stores its
        // channels in the order i = (j + l/2) % 4, so that the 8 lanes of a store phase hit 8 pieces.
        const int w = warp - 4;
        uint32_t sel[4], row[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t i = (uint32_t)(j + (lane >> 1)) & 3u;
            sel[j] = i | (i << 4) | ((4 + i) << 8) | ((4 + i) << 12);
            row[j] = 4 * lane + i;
        }
        const bool in0 = c0 + 4 * lane < a.d, in1 = c0 + 128 + 4 * lane < a.d;
        uint32_t x[2][16];           // two stages in flight: [half][8 rows]
        auto load = [&](int k, uint32_t* r) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int kr = k0 + 64 * k + 8 * w + i;
                const bool in = k < n_k && kr < k_end;
                const uint32_t* p =
                    reinterpret_cast<const uint32_t*>(a.table + (int64_t)(a.v0 + (in ? kr : 0)) * a.d + c0) + lane;
                r[i] = in && in0 ? __ldg(p) : 0u;
                r[8 + i] = in && in1 ? __ldg(p + 32) : 0u;
            }
        };
        auto convert = [&](int k, const uint32_t* r) -> bool {
            const int s = k % kDhStages;
            bool got = true;
            if (lane == 0) got = ptx::mbar_wait(&empty[s], ((uint32_t)(k / kDhStages) & 1u) ^ 1u) && !*abort_flag;
            got = __shfl_sync(0xffffffffu, got, 0);
            if (!got) {
                if (lane == 0) give_up(a.err, abort_flag);
                return false;
            }
            uint8_t* bs = smem + s * kDhStage + kDhA;
            const __half2 off = __floats2half2_rn(1152.0f, 1152.0f);          // 1024 + 128
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t o[4];
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        // bytes b0, b1 of two K rows -> fp16 (1024 + (b ^ 128)) pairs -> minus 1152: exact
                        const uint32_t t2 = __byte_perm(r[8 * h + 2 * p], r[8 * h + 2 * p + 1], sel[j]);
                        const uint32_t u2 = (t2 & 0x00FF00FFu) ^ 0x64806480u;
                        const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&u2), off);
                        o[p] = *reinterpret_cast<const uint32_t*>(&v);
                    }
                    const uint32_t n = 128 * h + row[j];
                    *reinterpret_cast<uint4*>(bs + n * 128 + 16 * ((uint32_t)w ^ (n & 7u))) =
                        make_uint4(o[0], o[1], o[2], o[3]);
                }
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(&full_b[s]);
            return true;
        };
        load(0, x[0]);
        load(1, x[1]);
        bool ok = true;
        for (int k = 0; k < n_k && ok; k += 2) {
            ok = convert(k, x[0]);
            load(k + 2, x[0]);
            if (ok && k + 1 < n_k) ok = convert(k + 1, x[1]);
            load(k + 3, x[1]);
        }
        // ---- the accumulator: lane quarter warp & 3, channel half (warp - 4) / 4
        const int q4 = warp & 3, half = (warp - 4) >> 2;
        const int t = tok0 + 32 * q4 + lane;
        float* dst = a.part + ((int64_t)sp * a.m + t) * a.d + c0 + half * (kBN / 2);
        const int c_end = min(kBN / 2, a.d - c0 - half * (kBN / 2));
        bool got = ok;
        if (n_k > 0) {
            if (got && lane == 0) got = ptx::mbar_wait(acc_full, 0u);
            got = __shfl_sync(0xffffffffu, got, 0);
            if (!got && lane == 0) give_up(a.err, abort_flag);
        }
        ptx::tc_fence_after();
        if (got && !(n_k == 0 && a.add)) {
#pragma unroll 1
            for (int c = 0; c < kBN / 2; c += 32) {
                uint32_t r[32];
                if (n_k > 0) {
                    ptx::tmem_ld_32x32b_x32(tmem + (uint32_t)(half * (kBN / 2) + c) + ((uint32_t)(32 * q4) << 16), r);
                    ptx::tmem_ld_wait();
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) r[i] = 0u;
                }
                if (t >= a.m) continue;
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    if (c + i >= c_end) continue;              // d is a multiple of 16
                    float4 v = make_float4(__uint_as_float(r[i]), __uint_as_float(r[i + 1]), __uint_as_float(r[i + 2]),
                                           __uint_as_float(r[i + 3]));
                    float4* p = reinterpret_cast<float4*>(dst + c + i);
                    if (a.add) {
                        const float4 o = *p;
                        v = make_float4(__fadd_rn(o.x, v.x), __fadd_rn(o.y, v.y), __fadd_rn(o.z, v.z), __fadd_rn(o.w, v.w));
                    }
                    *p = v;
                }
            }
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 256);
    }
}

// dh = bf16(grad (sum of the splits / K - s[target] E[target])): 8 channels per thread
__global__ void __launch_bounds__(256) xent_dh_out_kernel(const float* __restrict__ part, int splits,
                                                          const int8_t* __restrict__ table,
                                                          const float* __restrict__ scale, int vocab, int d,
                                                          const int32_t* __restrict__ targets,
                                                          const float* __restrict__ grad, int m,
                                                          const uint32_t* __restrict__ smax, uint16_t* dh,
                                                          uint32_t* err) {
    const int per = d >> 3;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)m * per) return;
    const int t = (int)(i / per), c = 8 * (int)(i - (int64_t)t * per);
    const int tg = targets[t];
    uint4 out = make_uint4(0u, 0u, 0u, 0u);
    if (is_token(tg, vocab)) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 0.0f;
        for (int s = 0; s < splits; ++s) {
            const float4* p = reinterpret_cast<const float4*>(part + ((int64_t)s * m + t) * d + c);
            const float4 x = p[0], y = p[1];
            v[0] = __fadd_rn(v[0], x.x); v[1] = __fadd_rn(v[1], x.y); v[2] = __fadd_rn(v[2], x.z);
            v[3] = __fadd_rn(v[3], x.w); v[4] = __fadd_rn(v[4], y.x); v[5] = __fadd_rn(v[5], y.y);
            v[6] = __fadd_rn(v[6], y.z); v[7] = __fadd_rn(v[7], y.w);
        }
        const float back = __fdiv_rn(1.0f, grad_scale(*smax)), g = grad[t], s = scale[tg];
        const uint2 e = *reinterpret_cast<const uint2*>(table + (int64_t)tg * d + c);
        uint32_t b[4];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float w = small_int_to_float((int)(int8_t)((k < 4 ? e.x : e.y) >> (8 * (k & 3))));
            v[k] = __fmul_rn(g, __fmaf_rn(-s, w, __fmul_rn(v[k], back)));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) b[k] = bf16x2_of(make_float2(v[2 * k], v[2 * k + 1]));
        out = make_uint4(b[0], b[1], b[2], b[3]);
    } else if (tg != DFSSM_IGNORE_TARGET && c == 0) {
        atomicOr(err, DFSSM_DEVERR_TOKEN_ID);
    }
    *reinterpret_cast<uint4*>(dh + (int64_t)t * d + c) = out;
}

// ------------------------------------------------------------------------------- host

inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// How a gradient call is cut: token blocks, vocabulary pieces, splits of a piece over the CTAs.
struct DhPlan {
    int tok_block;      // tokens per block
    int piece;          // table rows per piece (a multiple of kBN)
    int splits;         // K splits of a piece
    int k_split;        // columns per split (a multiple of 64)
};

DhPlan dh_plan(int m, int vocab, int d) {
    DhPlan p;
    p.tok_block = m < kTokBlock ? m : kTokBlock;
    const size_t bytes = (size_t)p.tok_block * vocab * 2;
    const int pieces = (int)((bytes + kGradBytes - 1) / kGradBytes);
    p.piece = ((vocab + pieces - 1) / pieces + kBN - 1) / kBN * kBN;
    // as many splits as fill 148 SMs with one CTA each, at least 1024 columns (16 stages) per split
    const int tiles = ((p.tok_block + kBM - 1) / kBM) * ((d + kBN - 1) / kBN);
    int s = 148 / tiles;
    const int most = (p.piece + 1023) / 1024;
    p.splits = s < 1 ? 1 : s > most ? most : s;
    p.k_split = ((p.piece + p.splits - 1) / p.splits + 63) / 64 * 64;
    p.splits = (p.piece + p.k_split - 1) / p.k_split;
    return p;
}

struct XentWs {
    size_t part, smax, g, dh, total;
};
XentWs xent_ws(int m, int vocab, int d, bool backward) {
    XentWs w{};
    size_t o = 256;                                       // error word
    if (!backward) {
        w.part = o;
        o = up256(o + (size_t)2 * ((vocab + kBN - 1) / kBN) * m * sizeof(float2));
    } else {
        const DhPlan p = dh_plan(m, vocab, d);
        w.smax = o;
        o += 256;
        w.g = o;
        o = up256(o + (size_t)p.tok_block * p.piece * sizeof(__half));
        w.dh = o;
        o = up256(o + (size_t)p.splits * p.tok_block * d * sizeof(float));
    }
    w.total = o;
    return w;
}

bool encode_rows(CUtensorMap* map, CUtensorMapDataType type, int elem, const void* base, int64_t cols, int64_t rows,
                 int64_t ld, int box_rows) {
    EncodeTiledFn enc = get_encode_fn();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)(ld * elem)};
    cuuint32_t box[2] = {(cuuint32_t)(128 / elem), (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return enc(map, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct XentSetup {
    int sm_count = 0;
    bool ready = false;
};
XentSetup g_xent_setup[64];
std::mutex g_xent_mu;

dfssm_status xent_setup(int* sm_count) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DFSSM_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_xent_mu);
    XentSetup& t = g_xent_setup[dev];
    if (!t.ready) {
        if (cudaDeviceGetAttribute(&t.sm_count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaFuncSetAttribute(xent_logits_kernel<kLse>, cudaFuncAttributeMaxDynamicSharedMemorySize, kLgSmem) !=
                cudaSuccess ||
            cudaFuncSetAttribute(xent_logits_kernel<kGrad>, cudaFuncAttributeMaxDynamicSharedMemorySize, kLgSmem) !=
                cudaSuccess ||
            cudaFuncSetAttribute(xent_dh_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kDhSmem) != cudaSuccess)
            return DFSSM_ERR_CUDA;
        t.ready = true;
    }
    *sm_count = t.sm_count;
    return DFSSM_OK;
}

dfssm_status check_xent(const dfssm_int8_table* t, int32_t m) {
    if (!t || !t->table || !t->scale || !al16(t->table) || !al16(t->scale)) return DFSSM_ERR_INVALID_ARG;
    if (t->d < 16 || t->d > kMaxDIn || t->d % 16 != 0 || t->vocab < 1 || t->vocab > (1 << 24))
        return DFSSM_ERR_UNSUPPORTED_SHAPE;
    if (m < 1 || m > kMaxM) return DFSSM_ERR_UNSUPPORTED_SHAPE;
    return DFSSM_OK;
}

bool al4(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

}  // namespace dfssm

using namespace dfssm;

extern "C" dfssm_status dfssm_xent_workspace_bytes(const dfssm_int8_table* table, int32_t m, int32_t backward,
                                                   size_t* bytes) {
    const dfssm_status st = check_xent(table, m);
    if (st != DFSSM_OK) return st;
    if (!bytes) return DFSSM_ERR_INVALID_ARG;
    *bytes = xent_ws(m, table->vocab, table->d, backward != 0).total;
    return DFSSM_OK;
}

extern "C" dfssm_status dfssm_xent_fwd(const dfssm_int8_table* table, const int8_t* q, const float* sx,
                                       const int32_t* targets, int32_t m, float* nll, float* lse, void* workspace,
                                       size_t workspace_bytes, void* stream) {
    dfssm_status st = check_xent(table, m);
    if (st != DFSSM_OK) return st;
    if (!q || !al16(q) || !al4(sx) || !al4(targets) || !al4(nll) || !al4(lse)) return DFSSM_ERR_INVALID_ARG;
    const int vocab = table->vocab, d = table->d;
    const XentWs w = xent_ws(m, vocab, d, false);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < w.total)
        return DFSSM_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = xent_setup(&sms)) != DFSSM_OK) return st;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    uint32_t* err = reinterpret_cast<uint32_t*>(ws);
    float2* part = reinterpret_cast<float2*>(ws + w.part);
    CUtensorMap mq, me;
    if (!encode_rows(&mq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, q, d, m, d, kBM) ||
        !encode_rows(&me, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, table->table, d, vocab, d, kBN))
        return DFSSM_ERR_CUDA;
    LogitsArgs a{};
    a.scale = table->scale;
    a.sx = sx;
    a.vocab = vocab;
    a.d = d;
    a.m = m;
    a.v0 = 0;
    a.v_end = vocab;
    a.part = part;
    a.err = err;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int n_vt = (vocab + kBN - 1) / kBN;
    const int64_t tiles = (int64_t)n_vt * ((m + kBM - 1) / kBM);
    if (tiles > (1 << 30)) return DFSSM_ERR_UNSUPPORTED_SHAPE;
    xent_logits_kernel<kLse><<<(int)(tiles < sms ? tiles : sms), kLgThreads, kLgSmem, s>>>(mq, me, a);
    if (cudaGetLastError() != cudaSuccess) return DFSSM_ERR_CUDA;
    xent_lse_kernel<<<(m + 7) / 8, 256, 0, s>>>(part, 2 * n_vt, table->table, table->scale, vocab, d, q, sx, targets, m,
                                                nll, lse, err);
    return cudaGetLastError() == cudaSuccess ? DFSSM_OK : DFSSM_ERR_CUDA;
}

extern "C" dfssm_status dfssm_xent_bwd(const dfssm_int8_table* table, const int8_t* q, const float* sx,
                                       const int32_t* targets, const float* lse, const float* grad, int32_t m, void* dh,
                                       void* workspace, size_t workspace_bytes, void* stream) {
    dfssm_status st = check_xent(table, m);
    if (st != DFSSM_OK) return st;
    if (!q || !al16(q) || !al4(sx) || !al4(targets) || !al4(lse) || !al4(grad) || !dh || !al16(dh))
        return DFSSM_ERR_INVALID_ARG;
    const int vocab = table->vocab, d = table->d;
    const XentWs w = xent_ws(m, vocab, d, true);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < w.total)
        return DFSSM_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = xent_setup(&sms)) != DFSSM_OK) return st;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    uint32_t* err = reinterpret_cast<uint32_t*>(ws);
    uint32_t* smax = reinterpret_cast<uint32_t*>(ws + w.smax);
    __half* g = reinterpret_cast<__half*>(ws + w.g);
    float* part = reinterpret_cast<float*>(ws + w.dh);
    const DhPlan p = dh_plan(m, vocab, d);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CUtensorMap me;
    if (!encode_rows(&me, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, table->table, d, vocab, d, kBN)) return DFSSM_ERR_CUDA;
    xent_smax_kernel<<<1, 1024, 0, s>>>(table->scale, vocab, smax);
    for (int t0 = 0; t0 < m; t0 += p.tok_block) {
        const int mb = m - t0 < p.tok_block ? m - t0 : p.tok_block;
        CUtensorMap mq, mg;
        if (!encode_rows(&mq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, q + (int64_t)t0 * d, d, mb, d, kBM) ||
            !encode_rows(&mg, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, g, p.piece, mb, p.piece, kBM))
            return DFSSM_ERR_CUDA;
        const int n_tt = (mb + kBM - 1) / kBM;
        for (int v0 = 0; v0 < vocab; v0 += p.piece) {
            LogitsArgs a{};
            a.scale = table->scale;
            a.sx = sx + t0;
            a.vocab = vocab;
            a.d = d;
            a.m = mb;
            a.v0 = v0;
            a.v_end = vocab - v0 < p.piece ? vocab : v0 + p.piece;
            a.lse = lse + t0;
            a.targets = targets + t0;
            a.smax = smax;
            a.g = g;
            a.ldg = p.piece;
            a.err = err;
            const int tiles = n_tt * ((a.v_end - v0 + kBN - 1) / kBN);
            xent_logits_kernel<kGrad><<<tiles < sms ? tiles : sms, kLgThreads, kLgSmem, s>>>(mq, me, a);
            DhArgs b{table->table, d, mb, v0, a.v_end - v0, p.k_split, part, v0 > 0 ? 1 : 0, err};
            xent_dh_kernel<<<dim3(n_tt, (d + kBN - 1) / kBN, p.splits), kDhThreads, kDhSmem, s>>>(mg, b);
            if (cudaGetLastError() != cudaSuccess) return DFSSM_ERR_CUDA;
        }
        const int64_t n = (int64_t)mb * (d >> 3);
        xent_dh_out_kernel<<<(int)((n + 255) / 256), 256, 0, s>>>(part, p.splits, table->table, table->scale, vocab, d,
                                                                   targets + t0, grad + t0, mb, smax,
                                                                   static_cast<uint16_t*>(dh) + (int64_t)t0 * d, err);
        if (cudaGetLastError() != cudaSuccess) return DFSSM_ERR_CUDA;
    }
    return DFSSM_OK;
}
