// Gradient of the state recurrence over packed sequences (dfssm_ssm_scan_bwd).
//
// With the state's gradient dS_t = dy_t C_t^T + exp(a_{t+1}) dS_{t+1} (dS_T + dfinal at the end):
//   dx_t = dt_t dS_t B_t + d_skip dy_t;   dB_t = sum_h dt_t dS_t^T x_t;   dC_t = sum_h S_t^T dy_t
//   d dt_t = x_t . dS_t B_t + A da_t,     da_t = <dS_t, exp(a_t) S_{t-1}>,  A = -exp(a_log)
// For a chunk of 64 tokens with the state S in front of it and the gradient dS behind it (both from
// scan_state_kernel, ssm_scan.cu, which leaves one pair per chunk and head in the workspace as two fp16 parts each),
// L[t, s] = exp(cum_t - cum_s) for s <= t:
//   G = C B^T, Z = dy x^T;   M = G o L;   W = sum_h Z o L dt_s
//   dx_s = dt_s (sum_t M[t, s] dy_t + exp(cum_64 - cum_s) dS B_s) + d_skip dy_s
//   dB   = W^T C + sum_h dt_s exp(cum_64 - cum_s) x_s dS
//   dC   = W B   + sum_h exp(cum_t) dy_t S
// G is shared by the heads of a group and W, summed over them in registers, multiplies C and B once
// per chunk, not once per head. da_t is what passes over token t:
//   da_t = sum_{t' >= t, s < t} E[t', s] + sum_{t' >= t} z_t' + sum_{s < t} w_s + exp(cum_64) <dS, S>
// with E = M o Z dt_s, z_t = exp(cum_t) dy_t . S C_t (from the accumulators of dC) and w_s = dt_s exp(cum_64 -
// cum_s) x_s . dS B_s (from those of dx). The first sum is that of E's row sums from t on less that of its
// column sums from t on, without the diagonal, which would only cancel; both come from the same fp32 values, so that
// what else cancels cancels (taken from dy . y and x . dx, which carry different roundings, d a_log was off by 3e-4).
// x . dx without the skip is the column sums of M o Z, the diagonal, and x . dS B.
//
// scan_grad_kernel: CTA (chunk, group, split of the group's heads), 16 warps, one head after another with the
// next head's tiles on the way (cp.async) and the last one's d dt behind (a warp without a part of Z). fp16 warp MMAs;
// x, dy, B and C are bf16 values under power-of-two scales (exact over 2^17 of range and more), M, W, S and dS two
// fp16 parts (2^-23; as bf16 parts, 2^-17, they were what short sequences' d a_log was off by, 8e-6, and the kernel
// 10% faster). Partial dB and dC of the splits and partial parameter sums per chunk are added in order by two
// small kernels.
//
// Measured (4 x 2,048 tokens, 64 heads): 394 to 406 us of the call's 651 (back to back from a graph), the states' kernel 240 to 250. Neither the tensor pipe nor
// shared memory is near its limit (36 and 52 %): a head's chain of products, exchanges and sums between two
// barriers bounds it, with one CTA per SM (228 KB); left out one at a time, Z and M cost 55 us, dC and dB 80, dx 45,
// the loads 28. The states alone are 1.1 GB of traffic, 166 us of the HBM's rate.
#include "ssm_scan.cuh"

namespace dfssm {
namespace scan {

namespace {

constexpr int kThreads = 512;

struct GradArgs {
    const uint16_t* dy;
    int64_t lddy;
    const uint16_t* s_in;      // [chunks][H][2][64][128] states in front of the chunks, fp16 high and low part
    const uint16_t* ds_out;    // the same: gradients behind them
    const float4* scale;       // [chunks][H] 2^-k of x, dy, the states, the gradients
    uint16_t* dx;
    int64_t lddx;
    uint16_t* ddt;
    int64_t ldddt;
    float* db_part;            // [splits][total][G 128]
    float* dc_part;
    float* sums;               // [chunks][H][4]: d dt_bias, d a_log, d d_skip
    int splits, per_split;     // heads per CTA
};

// one head's tiles
constexpr int kTx = 0, kTy = 8192, kTs = 16384, kTd = 16384 + 32768, kTile = 16384 + 2 * 32768;

// a head's decays, written one head ahead and read one head behind: three of them
struct HeadDecay {
    Decay d;
    float sig[kQ];             // d softplus
    float4 scale;              // 2^-k of x, dy, S, dS
};
// a head's partial sums, read one head behind: two of them
struct HeadSums {
    float wl[4][kQ];           // x . dx' of the four channel slices, of the part that leaves the chunk
    float z[4][kQ];            // C . (dy S) of the four state slices
    float row[4][kQ];          // sums of E over s < t, per block of 16 s
    float col[4][kQ];          // sums of M o Z over t > s, per block of 16 t
    float own[kQ];             // M o Z at t = s
    float skip[kQ];            // dy . x
    float dot[kThreads];       // <dS, S>
};
constexpr int kVecAt = 2 * 16384 + 2 * kTile + 2 * 8192;
constexpr int kGradSmem = kVecAt + 2 * (int)sizeof(HeadSums) + 3 * (int)sizeof(HeadDecay) + 128;
static_assert(kGradSmem <= 227 * 1024, "shared memory of one CTA");

// [64][128] bf16, contiguous in global memory, high then low part
__device__ __forceinline__ void load_state_tiles(uint32_t dst, const uint16_t* src, int tid) {
#pragma unroll
    for (int i = tid; i < 2 * kP * 16; i += kThreads) {
        const int part = i >> 10, row = (i >> 4) & 63, pc = i & 15;
        ptx::cp_async16_s(tile256(dst + part * 16384, row, pc), src + part * kStateElems + row * kN + 8 * pc);
    }
}

__global__ void __launch_bounds__(kThreads, 1) scan_grad_kernel(const Args a, const GradArgs o) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t wmax[kThreads / 32];
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    const uint32_t base = (ptx::smem_u32(smem_raw) + 127u) & ~127u;
    uint8_t* smem = smem_raw + (base - ptx::smem_u32(smem_raw));
    const uint32_t s_b = base, s_c = base + 16384, s_t = base + 32768, s_m = s_t + 2 * kTile;
    HeadSums* sums = reinterpret_cast<HeadSums*>(smem + kVecAt);
    HeadDecay* decays = reinterpret_cast<HeadDecay*>(smem + kVecAt + 2 * sizeof(HeadSums));
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int ngroups = a.nheads / a.per_group;
    const int sp = blockIdx.x % o.splits, g = blockIdx.x / o.splits % ngroups, ci = blockIdx.x / o.splits / ngroups;
    if (ci >= a.count[1]) return;
    const Chunk ch = a.chunks[ci];
    const int t0 = ch.t0, n = ch.n;
    const int h0 = g * a.per_group + sp * o.per_split;
    const int h1 = min(h0 + o.per_split, (g + 1) * a.per_group);

    auto fetch = [&](int h) {
        if (h < h1) {
            const uint32_t st = s_t + ((h - h0) & 1) * kTile;
            load_tile<64, kThreads>(st + kTx, a.x + (int64_t)h * kP, a.ldx, t0, n, tid);
            load_tile<64, kThreads>(st + kTy, o.dy + (int64_t)h * kP, o.lddy, t0, n, tid);
            const int64_t at = ((int64_t)ci * a.nheads + h) * 2 * kStateElems;
            load_state_tiles(st + kTs, o.s_in + at, tid);
            load_state_tiles(st + kTd, o.ds_out + at, tid);
        }
        ptx::cp_async_commit();
    };
    auto vectors = [&](int h) {                   // one warp
        if (h >= h1) return;
        HeadDecay& v = decays[(h - h0) % 3];
        const float bias = a.dt_bias[h], a2 = __fmul_rn(-expf(a.a_log[h]), kLog2e);
        const float r0 = raw_dt(a, t0, n, h, 2 * lane), r1 = raw_dt(a, t0, n, h, 2 * lane + 1);
        if (lane == 0) v.scale = o.scale[(int64_t)ci * a.nheads + h];
        chunk_decay(v.d, r0, r1, n, bias, a2, lane);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * lane + i;
            const float x = __fadd_rn(i ? r1 : r0, bias);
            v.sig[t] = x > 20.0f ? 1.0f : __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-x)));
        }
    };
    // d dt of a head whose sums are there; one warp, lane l has tokens 2 l, 2 l + 1
    auto finish = [&](int h) {
        const HeadDecay& d = decays[(h - h0) % 3];
        const HeadSums& v = sums[(h - h0) & 1];
        const float A = -expf(a.a_log[h]);
        float kp[2], q[2], wl[2], dot = 0.0f, sk = __fadd_rn(v.skip[2 * lane], v.skip[2 * lane + 1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * lane + i;
            const float leaves = __fadd_rn(__fadd_rn(v.wl[0][t], v.wl[1][t]), __fadd_rn(v.wl[2][t], v.wl[3][t]));
            const float col = __fadd_rn(__fadd_rn(v.col[0][t], v.col[1][t]), __fadd_rn(v.col[2][t], v.col[3][t]));
            kp[i] = __fadd_rn(__fadd_rn(leaves, col), v.own[t]);          // x . (dS B), all of it
            wl[i] = __fmul_rn(d.d.dt[t], leaves);
            const float z = __fmul_rn(d.d.done[t],
                                      __fadd_rn(__fadd_rn(v.z[0][t], v.z[1][t]), __fadd_rn(v.z[2][t], v.z[3][t])));
            const float row = __fadd_rn(__fadd_rn(v.row[0][t], v.row[1][t]), __fadd_rn(v.row[2][t], v.row[3][t]));
            q[i] = __fadd_rn(__fmaf_rn(-d.d.dt[t], col, row), z);
        }
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) dot = __fadd_rn(dot, v.dot[lane + 32 * i]);
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) {
            dot = __fadd_rn(dot, __shfl_xor_sync(0xffffffffu, dot, i));
            sk = __fadd_rn(sk, __shfl_xor_sync(0xffffffffu, sk, i));
        }
        // what enters at or after t and leaves it (from the right), what enters before t (from the left)
        float suf = __fadd_rn(q[0], q[1]), pre = __fadd_rn(wl[0], wl[1]);
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const float u = __shfl_down_sync(0xffffffffu, suf, s), x = __shfl_up_sync(0xffffffffu, pre, s);
            if (lane + s < 32) suf = __fadd_rn(suf, u);
            if (lane >= s) pre = __fadd_rn(pre, x);
        }
        float after = __shfl_down_sync(0xffffffffu, suf, 1), before = __shfl_up_sync(0xffffffffu, pre, 1);
        if (lane == 31) after = 0.0f;
        if (lane == 0) before = 0.0f;
        const float over = __fmul_rn(d.d.done[kQ - 1], dot);
        const float da[2] = {__fadd_rn(__fadd_rn(suf, before), over),
                             __fadd_rn(__fadd_rn(__fadd_rn(q[1], after), __fadd_rn(before, wl[0])), over)};
        float sb = 0.0f, sa = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * lane + i;
            if (t >= n) continue;
            const float dr = __fmul_rn(__fmaf_rn(A, da[i], kp[i]), d.sig[t]);
            o.ddt[(int64_t)(t0 + t) * o.ldddt + h] = f32_to_bf16_bits(dr);
            sb = __fadd_rn(sb, dr);
            sa = __fmaf_rn(da[i], __fmul_rn(d.d.dt[t], A), sa);
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) {
            sb = __fadd_rn(sb, __shfl_xor_sync(0xffffffffu, sb, s));
            sa = __fadd_rn(sa, __shfl_xor_sync(0xffffffffu, sa, s));
        }
        if (lane == 0)
            *reinterpret_cast<float4*>(o.sums + ((int64_t)ci * a.nheads + h) * 4) = make_float4(sb, sa, sk, 0.0f);
    };
    // x and dy of a head from bf16 to fp16 under their scales, in place
    auto convert = [&](int h) {
        const float4 sc = decays[(h - h0) % 3].scale;
        const uint32_t st = s_t + ((h - h0) & 1) * kTile;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t at = tile128(st + (i ? kTy : kTx), tid >> 3, tid & 7);
            const float up = __frcp_rn(i ? sc.y : sc.x);                  // a power of two: exact
            const uint4 v = ptx::lds128(at);
            const uint32_t q[4] = {bf16x2_to_f16x2(v.x, up), bf16x2_to_f16x2(v.y, up), bf16x2_to_f16x2(v.z, up),
                                   bf16x2_to_f16x2(v.w, up)};
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(q[0]), "r"(q[1]), "r"(q[2]), "r"(q[3]) : "memory");
        }
    };
    static_assert(kThreads == kQ * kP / 8, "a piece per thread and tile");
    const int64_t tl = (int64_t)ci * ngroups + g;
    load_tile<128, kThreads>(s_c, a.tiles + tl * 2 * (128 * kN), kN, 0, kQ, tid);
    load_tile<128, kThreads>(s_b, a.tiles + (tl * 2 + 1) * (128 * kN), kN, 0, kQ, tid);
    const float2 kcb = a.tile_scale[tl];              // 2^-k of C, of B
    const float kg = __fmul_rn(kcb.x, kcb.y);
    fetch(h0);
    if (w == 0) vectors(h0);
    ptx::cp_async_wait<0>();
    __syncthreads();
    convert(h0);
    __syncthreads();

    // G^T: warp (ws, wt) has rows s = 16 ws .., columns t = 16 wt ..; six of the sixteen have t < s everywhere
    const int ws = w & 3, wt = w >> 2;
    float G[2][4], W[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) G[j][i] = W[j][i] = 0.0f;
    if (wt >= ws) {
#pragma unroll 2
        for (int kk = 0; kk < kN; kk += 16) {
            uint32_t ba[4], cb[4];
            frag_a<256>(s_b, 16 * ws, kk, lane, ba);
            frag_b<256>(s_c, 16 * wt, kk, lane, cb);
            mma_h(G[0], ba, cb[0], cb[1]);
            mma_h(G[1], ba, cb[2], cb[3]);
        }
    }
    // warps 0 .. 7 have dC, rows t, the others dB, rows s: 32 (w & 1) + 16 i .., columns 32 (w / 2 % 4) + 8 j ..
    const bool side = w >= 8;
    const int rw = 32 * (w & 1), cw = 32 * ((w >> 1) & 3), pw = 16 * wt;
    float acc[2][4][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[i][j][q] = 0.0f;

    for (int h = h0; h < h1; ++h) {
        const uint32_t st = s_t + ((h - h0) & 1) * kTile;
        const uint32_t s_x = st + kTx, s_y = st + kTy, s_s = st + kTs, s_d = st + kTd;
        const Decay& dc = decays[(h - h0) % 3].d;
        const float4& sc = decays[(h - h0) % 3].scale;
        HeadSums& v = sums[(h - h0) & 1];
        const float skip = a.d_skip[h];
        fetch(h + 1);                             // over the tiles of the head before, which all warps have left
        // two of the warps without a part of Z
        if (w == 3 && h > h0) finish(h - 1);
        if (w == 2) vectors(h + 1);

        // ---- Z^T, then M^T to shared memory and W^T in registers
        if (wt >= ws) {
            float Z[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) Z[j][0] = Z[j][1] = Z[j][2] = Z[j][3] = 0.0f;
#pragma unroll
            for (int kk = 0; kk < kP; kk += 16) {
                uint32_t xa[4], yb[4];
                frag_a<128>(s_x, 16 * ws, kk, lane, xa);
                frag_b<128>(s_y, 16 * wt, kk, lane, yb);
                mma_h(Z[0], xa, yb[0], yb[1]);
                mma_h(Z[1], xa, yb[2], yb[3]);
            }
            const int s = 16 * ws + (lane >> 2);
            const float cs0 = dc.cum[s], cs1 = dc.cum[s + 8], ds0 = dc.dt[s], ds1 = dc.dt[s + 8];
            const float kz = __fmul_rn(sc.x, sc.y), w0 = __fmul_rn(ds0, kz), w1 = __fmul_rn(ds1, kz), km = __fmul_rn(kz, kg);
            float col0 = 0.0f, col1 = 0.0f;
            const int on = (lane >> 2) - 2 * (lane & 3);      // which of the thread's two columns is on the diagonal
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int t = 16 * wt + 8 * j + 2 * (lane & 3);
                const float2 ct = *reinterpret_cast<const float2*>(dc.cum + t);
                float l[4];
                l[0] = t >= s ? ex2(__fsub_rn(ct.x, cs0)) : 0.0f;
                l[1] = t + 1 >= s ? ex2(__fsub_rn(ct.y, cs0)) : 0.0f;
                l[2] = t >= s + 8 ? ex2(__fsub_rn(ct.x, cs1)) : 0.0f;
                l[3] = t + 1 >= s + 8 ? ex2(__fsub_rn(ct.y, cs1)) : 0.0f;
                const float m[4] = {__fmul_rn(G[j][0], l[0]), __fmul_rn(G[j][1], l[1]), __fmul_rn(G[j][2], l[2]),
                                    __fmul_rn(G[j][3], l[3])};
                // the sums of E over the warp's s for the thread's two t, and of M o Z over the thread's t
                float mz[4] = {__fmul_rn(m[0], Z[j][0]), __fmul_rn(m[1], Z[j][1]), __fmul_rn(m[2], Z[j][2]),
                                     __fmul_rn(m[3], Z[j][3])};
                // the diagonal (where L = 1), kept apart: what enters at t leaves before it could decay. It runs through
                // the first half of tile 0 and the second of tile 1.
                if (ws == wt && (unsigned)on < 2u) {
                    const int d = t + on;
                    v.skip[d] = __fmul_rn(on ? Z[j][2 * j + 1] : Z[j][2 * j], kz);
                    v.own[d] = __fmul_rn(on ? mz[2 * j + 1] : mz[2 * j], km);
                    if (on) mz[2 * j + 1] = 0.0f;
                    else mz[2 * j] = 0.0f;
                }
                col0 = __fadd_rn(col0, __fadd_rn(mz[0], mz[1]));
                col1 = __fadd_rn(col1, __fadd_rn(mz[2], mz[3]));
                float2 rs = make_float2(__fmaf_rn(mz[0], ds0, __fmul_rn(mz[2], ds1)), __fmaf_rn(mz[1], ds0, __fmul_rn(mz[3], ds1)));
#pragma unroll
                for (int q = 4; q < 32; q <<= 1) {
                    rs.x = __fadd_rn(rs.x, __shfl_xor_sync(0xffffffffu, rs.x, q));
                    rs.y = __fadd_rn(rs.y, __shfl_xor_sync(0xffffffffu, rs.y, q));
                }
                if (lane < 4) *reinterpret_cast<float2*>(v.row[ws] + t) = make_float2(__fmul_rn(rs.x, km), __fmul_rn(rs.y, km));
                const uint32_t p0 = tile128(s_m, s, 2 * wt + j) + 4 * (lane & 3);
                const uint32_t p1 = tile128(s_m, s + 8, 2 * wt + j) + 4 * (lane & 3);
                uint32_t m0, n0, m1, n1;
                split_f16x2(m[0], m[1], m0, n0);
                split_f16x2(m[2], m[3], m1, n1);
                ptx::sts32(p0, m0);
                ptx::sts32(p1, m1);
                ptx::sts32(p0 + 8192, n0);
                ptx::sts32(p1 + 8192, n1);
                W[j][0] = __fmaf_rn(Z[j][0], __fmul_rn(l[0], w0), W[j][0]);
                W[j][1] = __fmaf_rn(Z[j][1], __fmul_rn(l[1], w0), W[j][1]);
                W[j][2] = __fmaf_rn(Z[j][2], __fmul_rn(l[2], w1), W[j][2]);
                W[j][3] = __fmaf_rn(Z[j][3], __fmul_rn(l[3], w1), W[j][3]);
            }
#pragma unroll
            for (int q = 1; q < 4; q <<= 1) {
                col0 = __fadd_rn(col0, __shfl_xor_sync(0xffffffffu, col0, q));
                col1 = __fadd_rn(col1, __shfl_xor_sync(0xffffffffu, col1, q));
            }
            if ((lane & 3) == 0) {
                v.col[wt][s] = __fmul_rn(col0, km);
                v.col[wt][s + 8] = __fmul_rn(col1, km);
            }
        } else {
            if (lane < 8) *reinterpret_cast<float2*>(v.row[ws] + 16 * wt + 2 * lane) = make_float2(0.0f, 0.0f);
            else if (lane < 16) *reinterpret_cast<float2*>(v.col[wt] + 16 * ws + 2 * (lane - 8)) = make_float2(0.0f, 0.0f);
        }
        // ---- dC += exp(cum_t) dy S, dB += dt_s exp(cum_64 - cum_s) x dS
        {
            const uint32_t s_u = side ? s_x : s_y, s_v = side ? s_d : s_s;
            float e[2][2], z[2][2];
            const float kt = side ? __fmul_rn(sc.x, sc.w) : __fmul_rn(sc.y, sc.z);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int r = rw + 16 * i + 8 * hf + (lane >> 2);
                    e[i][hf] = __fmul_rn(side ? __fmul_rn(dc.dt[r], dc.left[r]) : dc.done[r], kt);
                    z[i][hf] = 0.0f;
                }
            float T[2][4][4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) T[i][j][0] = T[i][j][1] = T[i][j][2] = T[i][j][3] = 0.0f;
#pragma unroll 1
            for (int kk = 0; kk < kP; kk += 16) {
                uint32_t ua[2][4];
                frag_a<128>(s_u, rw, kk, lane, ua[0]);
                frag_a<128>(s_u, rw + 16, kk, lane, ua[1]);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t vh[4], vl[4];
                    frag_bt<256>(s_v, kk, cw + 16 * j, lane, vh);
                    frag_bt<256>(s_v + 16384, kk, cw + 16 * j, lane, vl);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        mma_h(T[i][2 * j], ua[i], vl[0], vl[1]);
                        mma_h(T[i][2 * j + 1], ua[i], vl[2], vl[3]);
                        mma_h(T[i][2 * j], ua[i], vh[0], vh[1]);
                        mma_h(T[i][2 * j + 1], ua[i], vh[2], vh[3]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = rw + 16 * i + (lane >> 2);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (!side) {                  // C_t . (dy S)_t over the warp's states
                        uint32_t c0, c1;
                        const uint32_t at = 4 * (lane & 3);
                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(c0) : "r"(tile256(s_c, r, (cw >> 3) + j) + at));
                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(c1) : "r"(tile256(s_c, r + 8, (cw >> 3) + j) + at));
                        const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&c0));
                        const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&c1));
                        z[i][0] = __fmaf_rn(T[i][j][0], f0.x, __fmaf_rn(T[i][j][1], f0.y, z[i][0]));
                        z[i][1] = __fmaf_rn(T[i][j][2], f1.x, __fmaf_rn(T[i][j][3], f1.y, z[i][1]));
                    }
                    float(&to)[4] = acc[i][j];
                    to[0] = __fmaf_rn(e[i][0], T[i][j][0], to[0]);
                    to[1] = __fmaf_rn(e[i][0], T[i][j][1], to[1]);
                    to[2] = __fmaf_rn(e[i][1], T[i][j][2], to[2]);
                    to[3] = __fmaf_rn(e[i][1], T[i][j][3], to[3]);
                }
            }
            if (!side) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        float t = z[i][hf];
                        t = __fadd_rn(t, __shfl_xor_sync(0xffffffffu, t, 1));
                        t = __fadd_rn(t, __shfl_xor_sync(0xffffffffu, t, 2));
                        if ((lane & 3) == 0) v.z[w >> 1][rw + 16 * i + 8 * hf + (lane >> 2)] = __fmul_rn(__fmul_rn(t, kt), kcb.x);
                    }
            }
        }
        // ---- <dS, S>: the diagonal of dS S^T, warp (ws, wt) the channels 16 ws .. and the states 32 wt ..
        {
            float D[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) D[j][0] = D[j][1] = D[j][2] = D[j][3] = 0.0f;
#pragma unroll
            for (int kk = 32 * wt; kk < 32 * wt + 32; kk += 16) {
                uint32_t dh[4], dl[4], sh[4], sl[4];
                frag_a<256>(s_d, 16 * ws, kk, lane, dh);
                frag_a<256>(s_d + 16384, 16 * ws, kk, lane, dl);
                frag_b<256>(s_s, 16 * ws, kk, lane, sh);
                frag_b<256>(s_s + 16384, 16 * ws, kk, lane, sl);
#pragma unroll
                for (int j = 0; j < 2; ++j) {        // low by low is below 2^-24 of the product
                    mma_h(D[j], dl, sh[2 * j], sh[2 * j + 1]);
                    mma_h(D[j], dh, sl[2 * j], sl[2 * j + 1]);
                    mma_h(D[j], dh, sh[2 * j], sh[2 * j + 1]);
                }
            }
            // rows lane / 4 (+ 8), columns 2 (lane % 4), + 1 of tile j: on the diagonal of tile 0 its first two, of 1 its last
            const int on = (lane >> 2) - 2 * (lane & 3);
            const float dot = on == 0 ? __fadd_rn(D[0][0], D[1][2]) : on == 1 ? __fadd_rn(D[0][1], D[1][3]) : 0.0f;
            v.dot[tid] = __fmul_rn(dot, __fmul_rn(sc.z, sc.w));
        }
        // ---- dx, rows s = 16 ws .., channels pw + 8 p ..
        {
            const float kx = __fmul_rn(kcb.y, sc.w);
            float X[2][4];
#pragma unroll
            for (int p = 0; p < 2; ++p) X[p][0] = X[p][1] = X[p][2] = X[p][3] = 0.0f;
#pragma unroll 4
            for (int kk = 0; kk < kN; kk += 16) {
                uint32_t dh[4], dl[4], ba[4];
                frag_b<256>(s_d, pw, kk, lane, dh);
                frag_b<256>(s_d + 16384, pw, kk, lane, dl);
                frag_a<256>(s_b, 16 * ws, kk, lane, ba);
                mma_h(X[0], ba, dl[0], dl[1]);
                mma_h(X[1], ba, dl[2], dl[3]);
                mma_h(X[0], ba, dh[0], dh[1]);
                mma_h(X[1], ba, dh[2], dh[3]);
            }
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int s = 16 * ws + 8 * hf + (lane >> 2);
                const float e = __fmul_rn(dc.left[s], kx);
                float wl = 0.0f;
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const uint32_t at = 4 * (lane & 3);
                    uint32_t xv;
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(xv) : "r"(tile128(s_x, s, (pw >> 3) + p) + at));
                    float& x0 = X[p][2 * hf];
                    float& x1 = X[p][2 * hf + 1];
                    x0 = __fmul_rn(x0, e);
                    x1 = __fmul_rn(x1, e);
                    const float2 xf = __half22float2(*reinterpret_cast<const __half2*>(&xv));
                    wl = __fmaf_rn(x0, xf.x, wl);
                    wl = __fmaf_rn(x1, xf.y, wl);
                }
                wl = __fadd_rn(wl, __shfl_xor_sync(0xffffffffu, wl, 1));
                wl = __fadd_rn(wl, __shfl_xor_sync(0xffffffffu, wl, 2));
                if ((lane & 3) == 0) v.wl[wt][s] = __fmul_rn(wl, sc.x);
            }
            ptx::cp_async_wait<0>();
            __syncthreads();                      // M^T is there, and the next head's tiles
            float Y[2][4];
#pragma unroll
            for (int p = 0; p < 2; ++p) Y[p][0] = Y[p][1] = Y[p][2] = Y[p][3] = 0.0f;
#pragma unroll
            for (int kt = 0; kt < 4; ++kt) {
                if (kt < ws) continue;            // t < s everywhere
                uint32_t yb[4], mh[4], ml[4];
                frag_bt<128>(s_y, 16 * kt, pw, lane, yb);
                frag_a<128>(s_m, 16 * ws, 16 * kt, lane, mh);
                frag_a<128>(s_m + 8192, 16 * ws, 16 * kt, lane, ml);
                mma_h(Y[0], ml, yb[0], yb[1]);
                mma_h(Y[1], ml, yb[2], yb[3]);
                mma_h(Y[0], mh, yb[0], yb[1]);
                mma_h(Y[1], mh, yb[2], yb[3]);
            }
            if (h + 1 < h1) convert(h + 1);
            const float ky = __fmul_rn(kg, sc.y), sky = __fmul_rn(skip, sc.y);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int s = 16 * ws + 8 * hf + (lane >> 2);
                const float dts = dc.dt[s];
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    uint32_t yv;
                    const uint32_t at = 4 * (lane & 3);
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(yv) : "r"(tile128(s_y, s, (pw >> 3) + p) + at));
                    const float2 yf = __half22float2(*reinterpret_cast<const __half2*>(&yv));
                    // over the x that the head is done with, to go out in whole 32-byte sectors
                    ptx::sts32(tile128(s_x, s, (pw >> 3) + p) + at,
                               bf16x2_of(make_float2(
                                   __fmaf_rn(dts, __fmaf_rn(Y[p][2 * hf], ky, X[p][2 * hf]), __fmul_rn(sky, yf.x)),
                                   __fmaf_rn(dts, __fmaf_rn(Y[p][2 * hf + 1], ky, X[p][2 * hf + 1]), __fmul_rn(sky, yf.y)))));
                }
            }
            __syncwarp();
            const int s = 16 * ws + (lane >> 1), pc = (pw >> 3) + (lane & 1);
            const uint4 row = ptx::lds128(tile128(s_x, s, pc));
            if (s < n) *reinterpret_cast<uint4*>(o.dx + (int64_t)(t0 + s) * o.lddx + h * kP + 8 * pc) = row;
        }
        __syncthreads();                          // the head's sums and the next one's fp16 tiles are there
    }
    if (w == 0) finish(h1 - 1);

    // ---- W^T as two fp16 parts under the scale of its largest value, then dB += W^T C, dC += W B
    {
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) m = fmaxf(m, fabsf(W[j][q]));
        const uint32_t mb = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
        if (lane == 0) wmax[w] = mb;
    }
    __syncthreads();
    uint32_t mb = 0u;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) mb = max(mb, wmax[i]);
    const float2 kw = pow2_scale(mb, 13);
    {
        const int s = 16 * ws + (lane >> 2);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t h0v, l0v, h1v, l1v;
            split_f16x2(__fmul_rn(W[j][0], kw.x), __fmul_rn(W[j][1], kw.x), h0v, l0v);
            split_f16x2(__fmul_rn(W[j][2], kw.x), __fmul_rn(W[j][3], kw.x), h1v, l1v);
            const uint32_t p0 = tile128(s_m, s, 2 * wt + j) + 4 * (lane & 3);
            const uint32_t p1 = tile128(s_m, s + 8, 2 * wt + j) + 4 * (lane & 3);
            ptx::sts32(p0, h0v);
            ptx::sts32(p1, h1v);
            ptx::sts32(p0 + 8192, l0v);
            ptx::sts32(p1 + 8192, l1v);
        }
    }
    __syncthreads();
    float T[2][4][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) T[i][j][0] = T[i][j][1] = T[i][j][2] = T[i][j][3] = 0.0f;
#pragma unroll 1
    for (int kk = 0; kk < kQ; kk += 16) {
        if (side ? kk + 15 < rw : kk > rw + 31) continue;      // dB: t >= s; dC: s <= t
        uint32_t vb[2][4];
        frag_bt<256>(side ? s_c : s_b, kk, cw, lane, vb[0]);
        frag_bt<256>(side ? s_c : s_b, kk, cw + 16, lane, vb[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int part = 1; part >= 0; --part) {
                uint32_t wa[4];
                if (side) frag_a<128>(s_m + part * 8192, rw + 16 * i, kk, lane, wa);
                else frag_at<128>(s_m + part * 8192, kk, rw + 16 * i, lane, wa);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    mma_h(T[i][2 * j], wa, vb[j][0], vb[j][1]);
                    mma_h(T[i][2 * j + 1], wa, vb[j][2], vb[j][3]);
                }
            }
        }
    }
    const float kwv = __fmul_rn(kw.y, side ? kcb.x : kcb.y);
    const int64_t ldp = (int64_t)ngroups * kN;
    float* part = side ? o.db_part : o.dc_part;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int r = rw + 16 * i + 8 * hf + (lane >> 2);
            if (r >= n) continue;
            const int64_t at = ((int64_t)sp * a.total + t0 + r) * ldp + g * kN + cw + 2 * (lane & 3);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<float2*>(part + at + 8 * j) =
                    make_float2(__fmaf_rn(T[i][j][2 * hf], kwv, acc[i][j][2 * hf]), __fmaf_rn(T[i][j][2 * hf + 1], kwv, acc[i][j][2 * hf + 1]));
        }
}

// dB and dC: the splits' parts added in order, 4 columns per thread; 8 CTAs per chunk (one: 24 us for 6 chunks of
// 16 parts, 8: 7), rows of no chunk stay
__global__ void __launch_bounds__(256) scan_sum_kernel(const Args a, const float* __restrict__ db_part,
                                                       const float* __restrict__ dc_part, int splits, uint16_t* db,
                                                       int64_t lddb, uint16_t* dc, int64_t lddc) {
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    if ((int)(blockIdx.x >> 3) >= a.count[1]) return;
    const Chunk ch = a.chunks[blockIdx.x >> 3];
    const int cols = a.nheads / a.per_group * kN, per = cols / 4;
    const float* part = blockIdx.y ? dc_part : db_part;
    uint16_t* out = blockIdx.y ? dc : db;
    const int64_t ld = blockIdx.y ? lddc : lddb;
    for (int i = (blockIdx.x & 7) * 256 + threadIdx.x; i < ch.n * per; i += 8 * 256) {
        const int r = i / per, c = 4 * (i - r * per);
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int k = 0; k < splits; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(part + ((int64_t)k * a.total + ch.t0 + r) * cols + c);
            s = make_float4(__fadd_rn(s.x, v.x), __fadd_rn(s.y, v.y), __fadd_rn(s.z, v.z), __fadd_rn(s.w, v.w));
        }
        *reinterpret_cast<uint2*>(out + (int64_t)(ch.t0 + r) * ld + c) =
            make_uint2(bf16x2_of(make_float2(s.x, s.y)), bf16x2_of(make_float2(s.z, s.w)));
    }
}

// the parameters' gradients: CTA per head over all chunks
__global__ void __launch_bounds__(256) scan_params_kernel(const Args a, const float* __restrict__ sums, float* ddt_bias,
                                                          float* da_log, float* dd_skip) {
    __shared__ float4 red[8];
    ptx::pdl_wait();
    const int h = blockIdx.x, n = a.count[1];
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i = threadIdx.x; i < n; i += 256) {
        const float4 v = *reinterpret_cast<const float4*>(sums + ((int64_t)i * a.nheads + h) * 4);
        s = make_float4(__fadd_rn(s.x, v.x), __fadd_rn(s.y, v.y), __fadd_rn(s.z, v.z), 0.0f);
    }
#pragma unroll
    for (int q = 16; q > 0; q >>= 1) {
        s.x = __fadd_rn(s.x, __shfl_xor_sync(0xffffffffu, s.x, q));
        s.y = __fadd_rn(s.y, __shfl_xor_sync(0xffffffffu, s.y, q));
        s.z = __fadd_rn(s.z, __shfl_xor_sync(0xffffffffu, s.z, q));
    }
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 8; ++w)
            s = make_float4(__fadd_rn(s.x, red[w].x), __fadd_rn(s.y, red[w].y), __fadd_rn(s.z, red[w].z), 0.0f);
        ddt_bias[h] = s.x;
        da_log[h] = s.y;
        dd_skip[h] = s.z;
    }
}

// Splits of a group's heads: the fewest waves of 148 CTAs, a CTA costing its heads and about one more; up to 32 (60
// tokens, 64 heads: 40 us, with 16 49, with 64 41)
struct Split {
    int splits, per;
};
Split choose_split(int cap_chunks, int ngroups, int per_group) {
    Split best{1, per_group};
    double cost = 1e30;
    for (int s = 1; s <= per_group && s <= 32; ++s) {
        const int per = (per_group + s - 1) / s;
        const int64_t ctas = (int64_t)cap_chunks * ngroups * s;
        const double c = (double)((ctas + 147) / 148) * (per + 1);
        if (c < cost) {
            cost = c;
            best = Split{(per_group + per - 1) / per, per};
        }
    }
    return best;
}

struct BwdWs {
    size_t s_in, ds, scale, db, dc, sums, total;
};
BwdWs bwd_ws(const dfssm_scan_dims* d, int total, int nseq, const Plan& p) {
    BwdWs w{};
    const size_t states = (size_t)p.cap_chunks * d->nheads * 2 * kStateElems * 2;
    const Split sp = choose_split(p.cap_chunks, d->ngroups, d->nheads / d->ngroups);
    size_t o = p.total;
    w.s_in = o;
    o = up256(o + states);
    w.ds = o;
    o = up256(o + states);
    w.scale = o;
    o = up256(o + (size_t)p.cap_chunks * d->nheads * sizeof(float4));
    w.db = o;
    o = up256(o + (size_t)sp.splits * total * d->ngroups * kN * 4);
    w.dc = o;
    o = up256(o + (size_t)sp.splits * total * d->ngroups * kN * 4);
    w.sums = o;
    o = up256(o + (size_t)p.cap_chunks * d->nheads * 16);
    w.total = o;
    return w;
}

}  // namespace

cudaError_t setup_bwd() {
    return cudaFuncSetAttribute(scan_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kGradSmem);
}

size_t bwd_workspace(const dfssm_scan_dims* d, int total, int nseq) {
    return bwd_ws(d, total, nseq, make_plan(d->nheads, d->ngroups, total, nseq, true)).total;
}

}  // namespace scan
}  // namespace dfssm

using namespace dfssm;
using namespace dfssm::scan;

extern "C" dfssm_status dfssm_ssm_scan_bwd(const dfssm_scan_dims* dims, const dfssm_scan_inputs* in, int32_t total,
                                           int32_t nseq, const void* dy, int64_t dy_stride, const float* dfinal_state,
                                           const dfssm_scan_grads* gr, void* workspace, size_t workspace_bytes,
                                           void* stream) {
    dfssm_status st = check_call(dims, in, total, nseq);
    if (st != DFSSM_OK) return st;
    if (!gr || !dy || !al16(dfinal_state) || !al16(gr->dinit_state)) return DFSSM_ERR_INVALID_ARG;
    const int64_t di = (int64_t)dims->nheads * kP, gn = (int64_t)dims->ngroups * kN, most = (int64_t)1 << 30;
    const void* rows[4] = {dy, gr->dx, gr->db, gr->dc};
    const int64_t ld[4] = {dy_stride, gr->dx_stride, gr->db_stride, gr->dc_stride}, least[4] = {di, di, gn, gn};
    for (int i = 0; i < 4; ++i)
        if (!rows[i] || !al16(rows[i]) || ld[i] < least[i] || ld[i] % 8 != 0 || ld[i] > most) return DFSSM_ERR_INVALID_ARG;
    if (!gr->ddt || (reinterpret_cast<uintptr_t>(gr->ddt) & 1u) || gr->ddt_stride < dims->nheads || gr->ddt_stride > most)
        return DFSSM_ERR_INVALID_ARG;
    const void* words[3] = {gr->ddt_bias, gr->da_log, gr->dd_skip};
    for (const void* p : words)
        if (!p || (reinterpret_cast<uintptr_t>(p) & 3u)) return DFSSM_ERR_INVALID_ARG;
    const Plan p = make_plan(dims->nheads, dims->ngroups, total, nseq, true);
    const BwdWs w = bwd_ws(dims, total, nseq, p);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < w.total)
        return DFSSM_ERR_INVALID_ARG;
    if ((st = setup()) != DFSSM_OK) return st;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const Args a = make_args(dims, in, total, nseq, p, ws);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    GradArgs o{};
    o.dy = static_cast<const uint16_t*>(dy);
    o.lddy = dy_stride;
    uint16_t* s_in = reinterpret_cast<uint16_t*>(ws + w.s_in);
    uint16_t* ds = reinterpret_cast<uint16_t*>(ws + w.ds);
    o.s_in = s_in;
    o.ds_out = ds;
    o.dx = static_cast<uint16_t*>(gr->dx);
    o.lddx = gr->dx_stride;
    o.ddt = static_cast<uint16_t*>(gr->ddt);
    o.ldddt = gr->ddt_stride;
    o.db_part = reinterpret_cast<float*>(ws + w.db);
    o.dc_part = reinterpret_cast<float*>(ws + w.dc);
    o.sums = reinterpret_cast<float*>(ws + w.sums);
    const Split sp = choose_split(p.cap_chunks, dims->ngroups, dims->nheads / dims->ngroups);
    o.splits = sp.splits;
    o.per_split = sp.per;
    float* scale = reinterpret_cast<float*>(ws + w.scale);
    o.scale = reinterpret_cast<const float4*>(scale);
    const StateArgs st_args{o.dy, dy_stride, dfinal_state, s_in, ds, scale, gr->dinit_state};
    if (launch_table(a, s) != cudaSuccess || launch_states(a, st_args, s) != cudaSuccess)
        return DFSSM_ERR_CUDA;
    if (launch_after(scan_grad_kernel, p.cap_chunks * dims->ngroups * sp.splits, kThreads, kGradSmem, s, a, o) != cudaSuccess ||
        launch_after(scan_sum_kernel, dim3(8 * p.cap_chunks, 2), 256, 0, s, a, o.db_part, o.dc_part, sp.splits,
                     static_cast<uint16_t*>(gr->db), gr->db_stride, static_cast<uint16_t*>(gr->dc), gr->dc_stride) != cudaSuccess ||
        launch_after(scan_params_kernel, dims->nheads, 256, 0, s, a, o.sums, gr->ddt_bias, gr->da_log, gr->dd_skip) != cudaSuccess)
        return DFSSM_ERR_CUDA;
    return DFSSM_OK;
}
