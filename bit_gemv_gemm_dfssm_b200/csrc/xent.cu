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
//          xent_lse_kernel joins the pairs of a token and takes the target's logit by a dp4a dot, which nll =
//          log sum exp(l - l[target]) is formed from (a small loss keeps its digits beside large logits);
//   kGrad  g = exp(l - lse) s[v] K as fp16 to the workspace, for a piece of the vocabulary, with 0 in the target's
//          column, whose factor exp(l - lse) - 1 goes to the workspace in fp32.
// xent_dh_kernel multiplies such a piece with its rows of the table (kind::f16): the table's
// bytes go through registers, where eight rows x four columns become four 16-byte pieces along K
// (prmt, lop3 and one packed subtraction make an exact fp16 integer of a byte), so the table is
// read as int8 and never stored in a wider form. Partial sums stay in fp32; xent_dh_out_kernel
// adds the splits in order and the target's row in fp32, scales by grad and rounds to bf16.
//
// fp16, not bf16, for g: it rounds once to 11 bits (2^-11 of the value at most), and K, a power of
// two with max |s| K in [2^13, 2^14), keeps exp(l - lse) s[v] K below 2^14 and its smallest
// kept step at 2^-38 max |s|. The target's column stays out of it: in the sum of a token whose target has the
// probability p, p s E would cancel against s E to (p - 1) s E, and 2^-12 of it, the rounding, is more than what is left
// from 1 - p = 2^-12 on (dh then off by its own size at p = 0.9999). exp(l - lse) - 1 is taken from the exact sum
// in 64 bits, one number per token. Every order is fixed.
//
// Measured, 50,288 x 2048, 20 calls back to back from a graph at 1,965 MHz (some seconds of the 2,048-token calls meet the
// power cap: 161 us at 1,485 MHz, 665 at 1,650). 2,048 tokens: loss 138 us, of it the logits 122, 82 to 84 % of the tensor
// pipe (256 columns of kind::i8 take about 200 cycles per 32 bytes of K); gradient 563 us in three pieces of 56 + 130 and 33 at
// the end, 67 and 54 % of the tensor pipe, the second's bytes-to-fp16 conversion and shared-memory traffic bound it. 1 token:
// 23 us on a cold table (4.5 TB/s), the join 5 beside it; 16 tokens: gradient 64 us, the table twice, 23 + 45.
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
constexpr int kLgRing = 4 * (kBM + kBN) * 128;          // stages of 128 K bytes of the tokens and of the table rows
constexpr int kLgStages = 8;                            // at most; 4 of full tiles
constexpr int kLgThreads = 12 * 32;      // TMA, MMA, 2 idle warps; 8 epilogue warps
constexpr int kLgEpi = 256;
constexpr int kLgOut = 8 * 2048;         // kGrad: an epilogue warp's 32 tokens x 32 columns
constexpr int kLgSmem = kLgRing + kLgOut + 2 * kBN * 4 + 256 + 1024;

// -- gradient kernel
constexpr int kDhA = kBM * 128, kDhB = kBN * 128;      // 64 K values per stage and accumulator
// 4 stages of one A tile and B, or 3 of two and B. As many converter groups of four warps, so that a group keeps to one
// stage and its waits for it are one phase apart; they write the accumulators out afterwards.
constexpr int dh_stages(int nm) { return nm == 1 ? 4 : 3; }
constexpr int dh_threads(int nm) { return 4 * 32 + 128 * dh_stages(nm); }
// the stages; barriers; the accumulators' staging rows, 2 KB for each of up to 16 warps
constexpr int kDhSmem = 192 * 1024 + 256 + 16 * 2048 + 1024;

// Most tokens whose gradient is worked on at a time (8,192 tokens x 50,288 x 2048, the best of 30 calls: 2,294 us, with 1,024
// 2,403, with 4,096 2,333; the workspace grows with it)
constexpr int kTokBlock = 2048;
constexpr int kTokTile = 256;            // the blocks' sizes are multiples of it
constexpr size_t kGradBytes = 80u << 20; // about the fp16 piece that stays in the 126 MB L2

struct LogitsArgs {
    const float* scale;
    const float* sx;
    int vocab, d, m;
    int bn;                              // table rows per tile: kBN, or one of kBNFew
    int a_bytes, stages;                 // of a stage: the tokens' rows; how many stages
    int v0, v_end;                       // table rows of this call
    float2* part;                        // kLse: [2 * v tiles][m]
    const float* lse;                    // kGrad
    const int32_t* targets;              // kGrad
    const uint32_t* smax;                // kGrad: bits of max |scale|
    __half* g;                           // kGrad: [m][ldg]
    float* hit;                          // kGrad: [m] exp(l - lse) - 1 of the target
    int ldg;
    uint32_t* err;
};

// 2^x to 2 ulp, 0 below 2^-126
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// An infinite scale would drop out of a softmax where its row's sum is negative, and zero rows of others: NaN shows in all
__device__ __forceinline__ float finite_or_nan(float v) {
    return (__float_as_uint(v) & 0x7F800000u) == 0x7F800000u ? __int_as_float(0x7FC00000) : v;
}

// A logit in units of log 2, of the exact sum as fp32: rounded alike wherever it is formed
__device__ __forceinline__ float logit_unit(float sx) { return __fmul_rn(finite_or_nan(sx), kLog2e); }
__device__ __forceinline__ float logit2(float dot, float scale, float unit) { return __fmul_rn(__fmul_rn(dot, scale), unit); }

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
    const uint32_t s_out = ptx::smem_u32(smem) + kLgRing;
    float* s_scale = reinterpret_cast<float*>(smem + kLgRing + kLgOut); // [2][kBN]
    uint64_t* full = reinterpret_cast<uint64_t*>(s_scale + 2 * kBN);                 // TMA bytes
    uint64_t* empty = full + kLgStages;                                              // MMA commit
    uint64_t* acc_full = empty + kLgStages;                                          // [2] MMA commit
    uint64_t* acc_empty = acc_full + 2;                                              // [2] one arrival per epilogue warp
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_tt = (a.m + kBM - 1) / kBM;
    const int n_tiles = n_tt * ((a.v_end - a.v0 + a.bn - 1) / a.bn);
    const int hw = a.bn / 2;                          // columns of an epilogue warp's half: a multiple of 32
    const int n_k = (a.d + 127) / 128;
    const int stages = a.stages, stage_bytes = a.a_bytes + a.bn * 128;

    // what follows in the stream may come in as CTAs end here; it waits for the whole grid before it reads
    ptx::pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(&acc_full[b], 1);
            ptx::mbar_init(&acc_empty[b], kLgEpi / 32);
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
            int it = 0, s = 0;
            uint32_t turn = 0;
            for (int tile = blockIdx.x; tile < n_tiles && !*abort_flag; tile += gridDim.x) {
                const int vt = tile / n_tt, tt = tile - vt * n_tt;
                for (int k = 0; k < n_k; ++k, ++it) {
                    if (!ptx::mbar_wait(&empty[s], turn ^ 1u)) {
                        give_up(a.err, abort_flag);
                        break;
                    }
                    uint8_t* st = smem + s * stage_bytes;
                    ptx::mbar_arrive_expect_tx(&full[s], stage_bytes);
                    ptx::tma_load_2d(st, &map_q, k * 128, tt * kBM, &full[s]);
                    ptx::tma_load_2d(st + a.a_bytes, &map_e, k * 128, a.v0 + vt * a.bn, &full[s]);
                    if (++s == stages) {
                        s = 0;
                        turn ^= 1u;
                    }
                }
            }
            // after a wait that gave up: the copies still in flight land before the CTA ends
            if (*abort_flag)
                for (int i = max(0, it - stages); i < it; ++i)
                    ptx::mbar_wait(&full[i % stages], (uint32_t)(i / stages) & 1u);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // kind::i8: D s32, A and B s8, both K-major
            const uint32_t idesc = (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(a.bn >> 3) << 17) |
                                   ((uint32_t)(kBM >> 4) << 24);
            int it = 0, tc = 0, s = 0;
            uint32_t turn = 0;
            bool ok = true;
            for (int tile = blockIdx.x; tile < n_tiles && ok && !*abort_flag; tile += gridDim.x, ++tc) {
                const int buf = tc & 1;
                if (!ptx::mbar_wait(&acc_empty[buf], ((uint32_t)(tc >> 1) & 1u) ^ 1u)) {
                    give_up(a.err, abort_flag);
                    break;
                }
                ptx::tc_fence_after();
                for (int k = 0; k < n_k; ++k, ++it) {
                    if (!ptx::mbar_wait(&full[s], turn)) {
                        give_up(a.err, abort_flag);
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    // 128 rows of tokens from here on, of which those behind the call's last are the table's bytes:
                    // their products go to lanes that nothing reads
                    const uint64_t ad = ptx::kmajor_sw128_desc(ptx::smem_u32(smem + s * stage_bytes));
                    const uint64_t bd = ptx::kmajor_sw128_desc(ptx::smem_u32(smem + s * stage_bytes + a.a_bytes));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        ptx::mma_i8(tmem + (uint32_t)(buf * kBN), ad + 2 * kk, bd + 2 * kk, idesc, (k | kk) != 0);
                    ptx::mma_commit(&empty[s]);
                    if (++s == stages) {
                        s = 0;
                        turn ^= 1u;
                    }
                }
                if (ok) ptx::mma_commit(&acc_full[buf]);
            }
            if (*abort_flag)           // the MMAs issued so far complete before TMEM is given back
                for (int i = max(0, it - stages); i < it; ++i)
                    ptx::mbar_wait(&empty[i % stages], (uint32_t)(i / stages) & 1u);
        }
    } else if (warp >= 4) {
        const int e = threadIdx.x - 4 * 32, q4 = warp & 3, half = (warp - 4) >> 2;
        if (MODE == kGrad) ptx::pdl_wait();        // max |scale|, and the piece's readers before it
        float gk = 0.0f;
        if (MODE == kGrad) gk = grad_scale(*a.smax);
        int tc = 0;
        bool got = true;
        for (int tile = blockIdx.x; tile < n_tiles; tile += gridDim.x, ++tc) {
            const int vt = tile / n_tt, tt = tile - vt * n_tt;
            const int buf = tc & 1;
            const int vbase = a.v0 + vt * a.bn;
            float* sc = s_scale + buf * kBN;
            sc[e] = e < a.bn && vbase + e < a.v_end ? finite_or_nan(a.scale[vbase + e]) : 0.0f;
            const int t = tt * kBM + 32 * q4 + lane;
            const bool live = t < a.m;
            const float k2 = live ? logit_unit(a.sx[t]) : 0.0f;
            float lse2 = 0.0f;
            bool counted = live;
            int target = -1;
            if (MODE == kGrad) {
                if (live) target = a.targets[t];
                counted = is_token(target, a.vocab);
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
            const int c_end = min(hw, a.v_end - vbase - half * hw);      // live columns of this half
#pragma unroll 1
            for (int c = 0; c < hw; c += 32) {
                const int col = half * hw + c;
                uint32_t r[32];
                ptx::tmem_ld_32x32b_x32(tmem + (uint32_t)(buf * kBN + col) + ((uint32_t)(32 * q4) << 16), r);
                ptx::tmem_ld_wait(r);
                if (c + 32 == hw) {           // the last read of this accumulator
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&acc_empty[buf]);
                }
                float z[32];
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 s4 = *reinterpret_cast<const float4*>(sc + col + i);
                    z[i] = logit2((float)(int)r[i], s4.x, k2);
                    z[i + 1] = logit2((float)(int)r[i + 1], s4.y, k2);
                    z[i + 2] = logit2((float)(int)r[i + 2], s4.z, k2);
                    z[i + 3] = logit2((float)(int)r[i + 3], s4.w, k2);
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
                    float s0 = __fmul_rn(sum, ex2(__fsub_rn(mx, ref))), s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        s0 = __fadd_rn(s0, ex2(__fsub_rn(z[i], ref)));
                        s1 = __fadd_rn(s1, ex2(__fsub_rn(z[i + 1], ref)));
                        s2 = __fadd_rn(s2, ex2(__fsub_rn(z[i + 2], ref)));
                        s3 = __fadd_rn(s3, ex2(__fsub_rn(z[i + 3], ref)));
                    }
                    sum = __fadd_rn(__fadd_rn(s0, s1), __fadd_rn(s2, s3));
                    mx = cm;
                } else {
                    const int at = target - vbase - col;
                    if (counted && (unsigned)at < 32u) {                     // once per token
                        int dot = 0;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i == at) {
                                dot = (int)r[i];
                                z[i] = -INFINITY;
                            }
                        const double l = (double)dot * (double)sc[col + at] * (double)a.sx[t];
                        a.hit[t] = expm1f((float)(l - (double)a.lse[t]));
                    }
                    uint32_t o[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float2 f = *reinterpret_cast<const float2*>(sc + col + i);
                        const float g0 = counted && c + i < c_end
                                             ? __fmul_rn(ex2(__fsub_rn(z[i], lse2)), __fmul_rn(f.x, gk)) : 0.0f;
                        const float g1 = counted && c + i + 1 < c_end
                                             ? __fmul_rn(ex2(__fsub_rn(z[i + 1], lse2)), __fmul_rn(f.y, gk)) : 0.0f;
                        const __half2 h = __floats2half2_rn(g0, g1);
                        o[i / 2] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                    // through the warp's staging rows (a token's 32 columns, 64 bytes, pieces swizzled by the row),
                    // so that a store covers 64 bytes of 8 rows: straight from the accumulator's layout, 16 bytes
                    // of 32 rows at a time, the stores bounded the kernel
                    const uint32_t so = s_out + (uint32_t)((warp - 4) * 2048);
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};"
                                     ::"r"(so + (uint32_t)(lane * 64 + 16 * (i ^ ((lane >> 1) & 3)))), "r"(o[4 * i]),
                                     "r"(o[4 * i + 1]), "r"(o[4 * i + 2]), "r"(o[4 * i + 3]) : "memory");
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r0 = 8 * i + (lane >> 2), pc = lane & 3, tr = tt * kBM + 32 * q4 + r0;
                        const uint4 v = ptx::lds128(so + (uint32_t)(r0 * 64 + 16 * (pc ^ ((r0 >> 1) & 3))));
                        if (tr < a.m) *reinterpret_cast<uint4*>(a.g + (int64_t)tr * a.ldg + vt * a.bn + col + 8 * pc) = v;
                    }
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

// WARPS warps per token (one for many tokens, eight for few: the pairs of one token are a chain of
// loads) join the token's (max, sum) pairs: lane i of warp w takes pairs i + 32 w, + 32 WARPS, ... in order, then a
// shuffle tree, then the warps in order. The target's logit comes from an int32 dot product.
template <int WARPS>
__global__ void __launch_bounds__(256) xent_lse_kernel(const float2* __restrict__ part, int n_part,
                                                       const int8_t* __restrict__ table,
                                                       const float* __restrict__ scale, int vocab, int d,
                                                       const int8_t* __restrict__ q, const float* __restrict__ sx,
                                                       const int32_t* __restrict__ targets, int m, float* nll,
                                                       float* lse_out, uint32_t* err) {
    __shared__ float2 s_ms[8];
    __shared__ int s_acc[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = WARPS == 1 ? (int)blockIdx.x * 8 + warp : (int)blockIdx.x, w = WARPS == 1 ? 0 : warp;
    const bool live = t < m;
    const int tg = live ? targets[t] : DFSSM_IGNORE_TARGET;
    int acc = 0;
    if (is_token(tg, vocab)) {
        const uint4* ep = reinterpret_cast<const uint4*>(table + (int64_t)tg * d);
        const uint4* qp = reinterpret_cast<const uint4*>(q + (int64_t)t * d);
        for (int i = lane + 32 * w; i < (d >> 4); i += 32 * WARPS) {
            const uint4 x = ep[i], y = qp[i];
            acc = __dp4a((int)x.x, (int)y.x, acc);
            acc = __dp4a((int)x.y, (int)y.y, acc);
            acc = __dp4a((int)x.z, (int)y.z, acc);
            acc = __dp4a((int)x.w, (int)y.w, acc);
        }
    }
    acc = __reduce_add_sync(0xffffffffu, acc);
    ptx::pdl_wait();                               // the pairs
    float mx = -INFINITY, sum = 0.0f;
    auto join = [&](float m2, float s2) {
        const float nm = fmaxf(mx, m2);
        const float ref = nm == -INFINITY ? 0.0f : nm;
        sum = __fadd_rn(__fmul_rn(sum, ex2(__fsub_rn(mx, ref))), __fmul_rn(s2, ex2(__fsub_rn(m2, ref))));
        mx = nm;
    };
    if (live)
        for (int i = lane + 32 * w; i < n_part; i += 32 * WARPS) {
            const float2 p = part[(int64_t)i * m + t];
            join(p.x, p.y);
        }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, mx, o), s2 = __shfl_xor_sync(0xffffffffu, sum, o);
        join(m2, s2);
    }
    if (WARPS > 1) {
        if (lane == 0) {
            s_ms[warp] = make_float2(mx, sum);
            s_acc[warp] = acc;
        }
        __syncthreads();
        if (threadIdx.x != 0) return;
        for (int k = 1; k < WARPS; ++k) {
            join(s_ms[k].x, s_ms[k].y);
            acc += s_acc[k];
        }
    }
    if (lane != 0 || !live) return;
    const float more = log2f(sum);
    float lse = __fmul_rn(__fadd_rn(mx, more), kLn2), loss = 0.0f;
    if (is_token(tg, vocab)) {
        // The target's logit with the roundings of its column: of the token's largest one, nothing is left but the
        // logarithm of the sum (lse - l, each rounded at its own size, would cancel). lse is then that much above the
        // exact logit.
        const float top = logit2((float)acc, finite_or_nan(scale[tg]), logit_unit(sx[t]));
        loss = __fmul_rn(__fadd_rn(__fsub_rn(mx, top), more), kLn2);
        if (top == mx) lse = (float)((double)acc * (double)scale[tg] * (double)sx[t] + (double)loss);
    } else if (tg != DFSSM_IGNORE_TARGET) {
        atomicOr(err, DFSSM_DEVERR_TOKEN_ID);
    }
    nll[t] = loss;
    lse_out[t] = lse;
}

// max |scale| as bits (one CTA)
__global__ void __launch_bounds__(1024) xent_smax_kernel(const float* __restrict__ scale, int vocab, uint32_t* out) {
    __shared__ uint32_t red[32];
    ptx::pdl_launch_dependents();
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

// The product's work is cut evenly over the CTAs in units of 64 table rows of one output tile; a CTA's range may
// begin inside one tile and end inside another. What a CTA adds up for a tile is one partial sum, in the
// tile's slot (CTA - first CTA of the tile).
struct DhSplit {
    int n_ct, ns;           // channel tiles; units per tile (of a full piece)
    int ctas;
    uint32_t share, more;   // units per CTA; the first `more` CTAs have one more
};
__host__ __device__ inline uint32_t first_unit(const DhSplit& p, uint32_t cta) {
    return cta * p.share + (cta < p.more ? cta : p.more);
}
__host__ __device__ inline int cta_of(const DhSplit& p, uint32_t unit) {
    const uint32_t big = p.more * (p.share + 1);
    return unit < big ? (int)(unit / (p.share + 1)) : (int)(p.more + (unit - big) / p.share);
}

struct DhArgs {
    const int8_t* table;
    int d, m;
    int v0, k_total;        // table row of the piece's column 0; its live columns
    DhSplit sp;
    float* part;            // [slots][m][d] of this piece
    uint32_t* err;
};

// Warp 0 loads the fp16 gradients by TMA, warps 4 and up turn the table's bytes into the B operand and write the
// accumulators out, warp 1 issues the MMAs. A tile is 128 NM tokens x 256 channels: with NM = 2 (more than
// 128 tokens) the expanded bytes serve two accumulators, which takes a quarter off the shared-memory traffic per
// MMA that bounds NM = 1.
template <int NM>
__global__ void __launch_bounds__(dh_threads(NM), 1)
xent_dh_kernel(const __grid_constant__ CUtensorMap map_g, const DhArgs a) {
    constexpr int kStages = dh_stages(NM), kA = NM * kDhA, kStage = kA + kDhB;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* full_a = reinterpret_cast<uint64_t*>(smem + kStages * kStage);         // TMA bytes
    uint64_t* full_b = full_a + kStages;                                             // one arrival per warp of a converter group
    uint64_t* empty = full_b + kStages;                                              // MMA commit
    uint64_t* acc_full = empty + kStages;                                            // MMA commit
    uint64_t* acc_empty = acc_full + 1;                                              // one arrival per converter warp
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 1);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t u0 = first_unit(a.sp, blockIdx.x), u1 = first_unit(a.sp, blockIdx.x + 1);
    const int ns_live = (a.k_total + 63) / 64;
    // the CTA's range tile by tile: f(tile, first unit, units); units may be none in the last, shorter piece
    auto for_tiles = [&](auto f) {
        for (uint32_t u = u0; u < u1;) {
            const int tile = (int)(u / (uint32_t)a.sp.ns), lo = (int)(u - (uint32_t)tile * a.sp.ns);
            const int hi = min(a.sp.ns, lo + (int)(u1 - u));
            if (!f(tile, lo, max(0, min(hi, ns_live) - lo))) return;
            u += hi - lo;
        }
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(&full_a[s], 1);
            ptx::mbar_init(&full_b[s], 4);
            ptx::mbar_init(&empty[s], 1);
        }
        ptx::mbar_init(acc_full, 1);
        ptx::mbar_init(acc_empty, 4 * kStages);
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(tmem_slot, NM * 256);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            ptx::pdl_wait();                       // the gradients of this piece
            int it = 0;
            for_tiles([&](int tile, int lo, int n) {
                for (int k = 0; k < n; ++k, ++it) {
                    const int s = it % kStages;
                    if (*abort_flag || !ptx::mbar_wait(&empty[s], ((uint32_t)(it / kStages) & 1u) ^ 1u)) {
                        give_up(a.err, abort_flag);
                        return false;
                    }
                    ptx::mbar_arrive_expect_tx(&full_a[s], kA);
#pragma unroll
                    for (int i = 0; i < NM; ++i)
                        ptx::tma_load_2d(smem + s * kStage + i * kDhA, &map_g, 64 * (lo + k),
                                         (tile / a.sp.n_ct * NM + i) * kBM, &full_a[s]);
                }
                return true;
            });
            if (*abort_flag)
                for (int i = max(0, it - kStages); i < it; ++i)
                    ptx::mbar_wait(&full_a[i % kStages], (uint32_t)(i / kStages) & 1u);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // kind::f16: D fp32, A and B fp16, both K-major
            constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(kBN >> 3) << 17) | ((uint32_t)(kBM >> 4) << 24);
            int it = 0, seg = 0;
            for_tiles([&](int, int, int n) {
                if (n == 0) return true;
                if (!ptx::mbar_wait(acc_empty, ((uint32_t)seg & 1u) ^ 1u)) {
                    give_up(a.err, abort_flag);
                    return false;
                }
                ptx::tc_fence_after();
                for (int k = 0; k < n; ++k, ++it) {
                    const int s = it % kStages;
                    const uint32_t ph = (uint32_t)(it / kStages) & 1u;
                    if (*abort_flag || !ptx::mbar_wait(&full_a[s], ph) || !ptx::mbar_wait(&full_b[s], ph)) {
                        give_up(a.err, abort_flag);
                        return false;
                    }
                    ptx::tc_fence_after();
                    const uint64_t bd = ptx::kmajor_sw128_desc(ptx::smem_u32(smem + s * kStage + kA));
#pragma unroll
                    for (int i = 0; i < NM; ++i) {
                        const uint64_t ad = ptx::kmajor_sw128_desc(ptx::smem_u32(smem + s * kStage + i * kDhA));
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            ptx::mma_f16(tmem + (uint32_t)(256 * i), ad + 2 * kk, bd + 2 * kk, idesc, (k | kk) != 0);
                    }
                    ptx::mma_commit(&empty[s]);
                }
                ptx::mma_commit(acc_full);
                ++seg;
                return true;
            });
            if (*abort_flag)
                for (int i = max(0, it - kStages); i < it; ++i)
                    ptx::mbar_wait(&empty[i % kStages], (uint32_t)(i / kStages) & 1u);
        }
    } else if (warp >= 4) {
        // Converters, a group of four warps per stage (what a stage costs a warp in latency, from its loads and the wait
        // for its release to the fence behind its stores, is then paid side by side; two groups with two stages'
        // loads each: 2,048 tokens 577 us instead of 563, 16 tokens the same 62). A
        // unit is 8 table rows (K) x 128 channels, lane l the channels 4 l .. 4 l + 3; warp w of a group takes the
        // K octets w and w + 4 of the stage, both channel halves. A 16-byte piece holds one channel's 8 K
        // values: row n, piece octet ^ (n & 7) of the 128-byte swizzle. Lane l stores its channels in the
        // order i = (j + l/2) % 4, so that the 8 lanes of a store phase hit 8 pieces. A group's next
        // stage is in flight behind it. Whole stages take a path without bounds.
        const int w = (warp - 4) & 3, group = (warp - 4) >> 2;
        uint32_t sel[4], off[4];         // off: the thread's pieces of octet 0, first half, in a stage's B tile
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t i = (uint32_t)(j + (lane >> 1)) & 3u, nr = 4 * lane + i;
            sel[j] = i | (i << 4) | ((4 + i) << 8) | ((4 + i) << 12);
            off[j] = nr * 128 + 16 * (nr & 7u);
        }
        const uint32_t smem_b = ptx::smem_u32(smem) + kA, s_out = ptx::smem_u32(smem) + kStages * kStage + 256 + (warp - 4) * 2048;
        const int q4 = warp & 3;
        const uint32_t d32 = (uint32_t)a.d;
        int seg = 0, it0 = 0;            // segments done; stages of all segments before
        bool waited = false;
        for_tiles([&](int tile, int lo, int n) {
            const int tok0 = tile / a.sp.n_ct * NM * kBM, c0 = tile % a.sp.n_ct * kBN;
            const bool in0 = c0 + 4 * lane < a.d, in1 = c0 + 128 + 4 * lane < a.d;
            const bool all_c = c0 + kBN <= a.d;
            const int8_t* src = a.table + (int64_t)(a.v0 + 64 * lo + 8 * w) * a.d + c0 + 4 * lane;
            const int left = a.k_total - 64 * lo - 8 * w;        // live rows from the thread's first one on
            uint32_t x[32];              // [octet, half, 8 rows]
            auto load = [&](int k, uint32_t* r) {
                const int8_t* p = src + (int64_t)k * 64 * d32;
                if (k < n && all_c && 64 * k + 40 <= left) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint32_t* q = reinterpret_cast<const uint32_t*>(p + (uint32_t)(i < 8 ? i : 24 + i) * d32);
                        r[(i >> 3) * 16 + (i & 7)] = __ldg(q);
                        r[(i >> 3) * 16 + 8 + (i & 7)] = __ldg(q + 32);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int row = i < 8 ? i : 24 + i;
                        const bool in = k < n && 64 * k + row < left;
                        const uint32_t* q = reinterpret_cast<const uint32_t*>(p + (uint32_t)row * d32);
                        r[(i >> 3) * 16 + (i & 7)] = in && in0 ? __ldg(q) : 0u;
                        r[(i >> 3) * 16 + 8 + (i & 7)] = in && in1 ? __ldg(q + 32) : 0u;
                    }
                }
            };
            auto convert = [&](int k, const uint32_t* r) -> bool {
                const int it = it0 + k, st = it % kStages;
                bool got = true;
                if (lane == 0) got = ptx::mbar_wait(&empty[st], ((uint32_t)(it / kStages) & 1u) ^ 1u) && !*abort_flag;
                got = __shfl_sync(0xffffffffu, got, 0);
                if (!got) {
                    if (lane == 0) give_up(a.err, abort_flag);
                    return false;
                }
                const uint32_t bs = smem_b + st * kStage;
                const __half2 bias = __floats2half2_rn(1152.0f, 1152.0f);         // 1024 + 128
#pragma unroll
                for (int oc = 0; oc < 2; ++oc)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t o[4];
#pragma unroll
                            for (int p = 0; p < 4; ++p) {
                                // bytes b0, b1 of two K rows -> fp16 (1024 + (b ^ 128)) pairs -> minus 1152: exact
                                const uint32_t t2 = __byte_perm(r[16 * oc + 8 * h + 2 * p], r[16 * oc + 8 * h + 2 * p + 1], sel[j]);
                                const uint32_t u2 = (t2 & 0x00FF00FFu) ^ 0x64806480u;
                                const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&u2), bias);
                                o[p] = *reinterpret_cast<const uint32_t*>(&v);
                            }
                            const uint32_t at = bs + 128 * 128 * h + (off[j] ^ (uint32_t)(16 * (w + 4 * oc)));
                            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};"
                                         ::"r"(at), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]) : "memory");
                        }
                ptx::fence_proxy_async_smem();
                __syncwarp();                      // one arrival per warp: 256 on one barrier serialise
                if (lane == 0) ptx::mbar_arrive(&full_b[st]);
                return true;
            };
            const int k0 = (group + kStages - it0 % kStages) % kStages;      // this group's first stage of the segment
            load(k0, x);
            for (int k = k0; k < n; k += kStages) {
                if (!convert(k, x)) return false;
                load(k + kStages, x);
            }
            it0 += n;
            // ---- the accumulators: lane quarter warp & 3, the groups' turns at blocks of 16 columns
            if (!waited) {
                ptx::pdl_wait();                   // earlier readers of the partial sums
                waited = true;
            }
            if (n > 0) {
                bool got = true;
                if (lane == 0) got = ptx::mbar_wait(acc_full, (uint32_t)seg & 1u);
                got = __shfl_sync(0xffffffffu, got, 0);
                if (!got) {
                    if (lane == 0) give_up(a.err, abort_flag);
                    return false;
                }
                ptx::tc_fence_after();
            }
            const int slot = blockIdx.x - cta_of(a.sp, (uint32_t)tile * a.sp.ns);
#pragma unroll 1
            for (int c = 16 * group; c < NM * kBN; c += 16 * kStages) {
                const int i = c / kBN, col = c % kBN;
                uint32_t r[16];
                if (n > 0) {
                    ptx::tmem_ld_32x32b_x16(tmem + (uint32_t)(256 * i + col) + ((uint32_t)(32 * q4) << 16), r);
                    ptx::tmem_ld_wait(r);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) r[e] = 0u;
                }
                // through the warp's 2 KB, so that a store covers 64 bytes of 8 rows
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};"
                                 ::"r"(s_out + (uint32_t)(lane * 64 + 16 * (e ^ ((lane >> 1) & 3)))), "r"(r[4 * e]),
                                 "r"(r[4 * e + 1]), "r"(r[4 * e + 2]), "r"(r[4 * e + 3]) : "memory");
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int rr = 8 * e + (lane >> 2), pc = lane & 3, t = tok0 + i * kBM + 32 * q4 + rr;
                    const uint4 v = ptx::lds128(s_out + (uint32_t)(rr * 64 + 16 * (pc ^ ((rr >> 1) & 3))));
                    if (t < a.m && c0 + col + 4 * pc < a.d)
                        *reinterpret_cast<uint4*>(a.part + ((int64_t)slot * a.m + t) * a.d + c0 + col + 4 * pc) = v;
                }
            }
            if (n > 0) {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(acc_empty);
                ++seg;
            }
            return true;
        });
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, NM * 256);
    }
}

// dh = bf16(grad (sum of the slots / K + hit s[target] E[target])): 4 channels per thread
__global__ void __launch_bounds__(256) xent_dh_out_kernel(const float* __restrict__ part, const DhSplit sp, int pieces,
                                                          int max_slots, int tile_tokens,
                                                          const int8_t* __restrict__ table,
                                                          const float* __restrict__ scale, int vocab, int d,
                                                          const int32_t* __restrict__ targets,
                                                          const float* __restrict__ grad, int m,
                                                          const uint32_t* __restrict__ smax,
                                                          const float* __restrict__ hit, uint16_t* dh,
                                                          uint32_t* err) {
    const int per = d >> 2;
    const uint32_t i = blockIdx.x * 256u + threadIdx.x;      // m is at most a token block here
    if (i >= (uint32_t)(m * per)) return;
    const int t = (int)(i / (uint32_t)per), c = 4 * (int)(i - (uint32_t)(t * per));
    const int tg = targets[t];
    const bool on = is_token(tg, vocab);
    const uint32_t u = (uint32_t)(t / tile_tokens * sp.n_ct + c / kBN) * sp.ns;
    const int slots = cta_of(sp, u + sp.ns - 1) - cta_of(sp, u) + 1;
    ptx::pdl_wait();                                   // the partial sums
    uint2 out = make_uint2(0u, 0u);
    if (on) {
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        // piece by piece, slot by slot, eight loads at a time
        const int64_t step = (int64_t)m * d, gap = (max_slots - slots) * step;
        const float* at = part + (int64_t)t * d + c;
        int s = 0;
        for (int q = pieces * slots; q > 0; q -= 8) {
            float4 x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                x[k] = k < q ? __ldcs(reinterpret_cast<const float4*>(at)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                at += step;
                if (++s == slots) {
                    s = 0;
                    at += gap;
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < q)
                    v = make_float4(__fadd_rn(v.x, x[k].x), __fadd_rn(v.y, x[k].y), __fadd_rn(v.z, x[k].z), __fadd_rn(v.w, x[k].w));
        }
        const float back = __fdiv_rn(1.0f, grad_scale(*smax)), g = grad[t], es = __fmul_rn(hit[t], scale[tg]);
        const uint32_t e = *reinterpret_cast<const uint32_t*>(table + (int64_t)tg * d + c);
        const float f[4] = {v.x, v.y, v.z, v.w};
        float o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            o[k] = __fmul_rn(g, __fmaf_rn(es, small_int_to_float((int)(int8_t)(e >> (8 * k))), __fmul_rn(f[k], back)));
        out = make_uint2(bf16x2_of(make_float2(o[0], o[1])), bf16x2_of(make_float2(o[2], o[3])));
    } else if (tg != DFSSM_IGNORE_TARGET && c == 0) {
        atomicOr(err, DFSSM_DEVERR_TOKEN_ID);
    }
    *reinterpret_cast<uint2*>(dh + (int64_t)t * d + c) = out;
}

// ------------------------------------------------------------------------------- host

inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

constexpr int kSms = 148;

// A stage holds the tokens' rows that there are (in whole swizzle blocks of 8); the smaller it is, the more of them.
int stage_tokens(int m) { return m < kBM ? (m + 7) / 8 * 8 : kBM; }
int stage_count(int a_bytes, int bn) {
    const int n = kLgRing / (a_bytes + bn * 128);
    return n < kLgStages ? n : kLgStages;
}
constexpr int kBNFew[2] = {128, 192};
static_assert(kBNFew[0] >= kBM, "the 128 rows that a product reads as tokens lie in the stage");

// Table rows per tile. With one token tile the table is streamed once and a call has few tiles: the size that leaves the
// longest CTA the fewest rows, 128 where that is the same (its last epilogue is the shorter one; 256 never leaves
// fewer). Calls back to back over tables of 2048 channels, 1 token, with 128 / 192 / 256 rows, us: 8,000 rows 10.1 / 10.7 /
// 12.2, 32,000 16.9 / 19.8 / 17.0, 37,888 18.4 / 21.0 / 19.9, 50,288 23.0 / 22.7 / 25.4, 65,536 27.6 / 28.3 / 28.7, 128,256
// 47.1 / 48.2 / 48.4.
int tile_rows(int m, int vocab) {
    if (m > kBM) return kBN;
    auto longest = [&](int bn) { return ((vocab + bn - 1) / bn + kSms - 1) / kSms * bn; };
    return longest(kBNFew[1]) < longest(kBNFew[0]) ? kBNFew[1] : kBNFew[0];
}

// How a gradient call is cut: the tokens into blocks of nearly equal numbers of 256-token tiles, each with a product of its own
// size (blocks of 2,048 and a last one that ran the same product for what was left: 2,049 tokens 1,055 us, now 657, 3,000
// 1,048, now 870); the vocabulary into pieces; a block's product into units over the CTAs.
struct DhPlan {
    int blocks;
    int tok_block;      // tokens of the first block, the largest
    int pieces;
    int piece;          // table rows per piece (a multiple of the logits' tile and of 64)
    int nm;             // 128-token accumulators per CTA
};

// tokens in front of block i
int block_begin(int m, int blocks, int i) {
    const int tiles = (m + kTokTile - 1) / kTokTile;
    const int64_t t = (int64_t)kTokTile * (tiles / blocks * i + (i < tiles % blocks ? i : tiles % blocks));
    return t < m ? (int)t : m;
}

DhPlan dh_plan(int m, int vocab) {
    DhPlan p;
    p.blocks = (m + kTokBlock - 1) / kTokBlock;
    p.tok_block = block_begin(m, p.blocks, 1);
    const int bn = tile_rows(p.tok_block, vocab), all = (vocab + bn - 1) / bn;
    const int most = (int)(kGradBytes / ((size_t)p.tok_block * 2 * bn));       // tiles of the largest piece
    p.pieces = (all + most - 1) / most;
    p.piece = (all + p.pieces - 1) / p.pieces * bn;
    p.nm = p.tok_block > kBM ? 2 : 1;
    return p;
}

// The units of a block of mb tokens over the CTAs, and the partial sums that a tile can have
DhSplit dh_split(const DhPlan& p, int mb, int d, int* slots) {
    DhSplit sp;
    sp.n_ct = (d + kBN - 1) / kBN;
    sp.ns = p.piece / 64;
    // at most 8 x 32 tiles of at most 2^18 units
    const uint32_t units = (uint32_t)((mb + p.nm * kBM - 1) / (p.nm * kBM)) * sp.n_ct * sp.ns;
    sp.ctas = units / 8 < 1 ? 1 : units / 8 < (uint32_t)kSms ? (int)(units / 8) : kSms;        // 8 units at least
    sp.share = units / sp.ctas;
    sp.more = units % sp.ctas;
    *slots = (int)((sp.ns + sp.share - 1) / sp.share) + 1;
    return sp;
}

struct XentWs {
    size_t part, smax, hit, g, dh, total;
};
XentWs xent_ws(int m, int vocab, int d, bool backward) {
    XentWs w{};
    size_t o = 256;                                       // error word
    if (!backward) {
        w.part = o;
        o = up256(o + (size_t)2 * ((vocab + tile_rows(m, vocab) - 1) / tile_rows(m, vocab)) * m * sizeof(float2));
    } else {
        const DhPlan p = dh_plan(m, vocab);
        w.smax = o;
        o += 256;
        w.hit = o;
        o = up256(o + (size_t)p.tok_block * sizeof(float));
        w.g = o;
        o = up256(o + (size_t)p.tok_block * p.piece * sizeof(__half));
        w.dh = o;
        size_t rows = 0;                                  // a smaller block's tiles can have more slots
        for (int i = 0; i < p.blocks; ++i) {
            const int mb = block_begin(m, p.blocks, i + 1) - block_begin(m, p.blocks, i);
            int slots;
            dh_split(p, mb, d, &slots);
            rows = rows > (size_t)slots * mb ? rows : (size_t)slots * mb;
        }
        o = up256(o + p.pieces * rows * d * sizeof(float));
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
            cudaFuncSetAttribute(xent_dh_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kDhSmem) != cudaSuccess ||
            cudaFuncSetAttribute(xent_dh_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, kDhSmem) != cudaSuccess)
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
    const int bn = tile_rows(m, vocab);
    if (!encode_rows(&mq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, q, d, m, d, stage_tokens(m)) ||
        !encode_rows(&me, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, table->table, d, vocab, d, bn))
        return DFSSM_ERR_CUDA;
    LogitsArgs a{};
    a.scale = table->scale;
    a.sx = sx;
    a.vocab = vocab;
    a.d = d;
    a.m = m;
    a.bn = bn;
    a.a_bytes = stage_tokens(m) * 128;
    a.stages = stage_count(a.a_bytes, bn);
    a.v0 = 0;
    a.v_end = vocab;
    a.part = part;
    a.err = err;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int n_vt = (vocab + bn - 1) / bn;
    const int64_t tiles = (int64_t)n_vt * ((m + kBM - 1) / kBM);
    if (tiles > (1 << 30)) return DFSSM_ERR_UNSUPPORTED_SHAPE;
    xent_logits_kernel<kLse><<<(int)(tiles < sms ? tiles : sms), kLgThreads, kLgSmem, s>>>(mq, me, a);
    if (cudaGetLastError() != cudaSuccess) return DFSSM_ERR_CUDA;
    const cudaError_t e =
        m < 1024 ? launch_after(xent_lse_kernel<8>, m, 256, 0, s, part, 2 * n_vt, table->table, table->scale, vocab, d, q,
                                sx, targets, m, nll, lse, err)
                 : launch_after(xent_lse_kernel<1>, (m + 7) / 8, 256, 0, s, part, 2 * n_vt, table->table, table->scale, vocab,
                                d, q, sx, targets, m, nll, lse, err);
    return e == cudaSuccess ? DFSSM_OK : DFSSM_ERR_CUDA;
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
    float* hit = reinterpret_cast<float*>(ws + w.hit);
    __half* g = reinterpret_cast<__half*>(ws + w.g);
    float* part = reinterpret_cast<float*>(ws + w.dh);
    const DhPlan p = dh_plan(m, vocab);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CUtensorMap me;
    const int bn = tile_rows(p.tok_block, vocab);
    if (!encode_rows(&me, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, table->table, d, vocab, d, bn)) return DFSSM_ERR_CUDA;
    xent_smax_kernel<<<1, 1024, 0, s>>>(table->scale, vocab, smax);
    cudaError_t e = cudaGetLastError();
    for (int i = 0; i < p.blocks && e == cudaSuccess; ++i) {
        const int t0 = block_begin(m, p.blocks, i), mb = block_begin(m, p.blocks, i + 1) - t0;
        int slots;
        const DhSplit sp = dh_split(p, mb, d, &slots);
        CUtensorMap mq, mg;
        if (!encode_rows(&mq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, q + (int64_t)t0 * d, d, mb, d, stage_tokens(mb)) ||
            !encode_rows(&mg, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, g, p.piece, mb, p.piece, kBM))
            return DFSSM_ERR_CUDA;
        const int n_tt = (mb + kBM - 1) / kBM;
        for (int v0 = 0; v0 < vocab && e == cudaSuccess; v0 += p.piece) {
            LogitsArgs a{};
            a.scale = table->scale;
            a.sx = sx + t0;
            a.vocab = vocab;
            a.d = d;
            a.m = mb;
            a.bn = bn;
            a.a_bytes = stage_tokens(mb) * 128;
            a.stages = stage_count(a.a_bytes, bn);
            a.v0 = v0;
            a.v_end = vocab - v0 < p.piece ? vocab : v0 + p.piece;
            a.lse = lse + t0;
            a.targets = targets + t0;
            a.smax = smax;
            a.g = g;
            a.hit = hit;
            a.ldg = p.piece;
            a.err = err;
            const int tiles = n_tt * ((a.v_end - v0 + bn - 1) / bn);
            e = launch_after(xent_logits_kernel<kGrad>, tiles < sms ? tiles : sms, kLgThreads, kLgSmem, s, mq, me, a);
            const DhArgs b{table->table, d, mb, v0, a.v_end - v0, sp, part + (size_t)(v0 / p.piece) * slots * mb * d, err};
            if (e == cudaSuccess)
                e = launch_after(p.nm == 1 ? xent_dh_kernel<1> : xent_dh_kernel<2>, sp.ctas, dh_threads(p.nm), kDhSmem, s, mg, b);
        }
        const int64_t n = (int64_t)mb * (d >> 2);
        if (e == cudaSuccess)
            e = launch_after(xent_dh_out_kernel, (int)((n + 255) / 256), 256, 0, s, part, sp, p.pieces, slots, p.nm * kBM, table->table,
                             table->scale, vocab, d, targets + t0, grad + t0, mb, smax, hit,
                             static_cast<uint16_t*>(dh) + (int64_t)t0 * d, err);
    }
    return e == cudaSuccess ? DFSSM_OK : DFSSM_ERR_CUDA;
}
