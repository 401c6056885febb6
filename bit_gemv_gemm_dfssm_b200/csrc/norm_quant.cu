// Residual add + RMS norm with an int8 output and one fp32 scale per token, and the norm's
// gradient.
//
// The forward is the block frame of block_norm.cu followed by the layer's own quantiser, in one
// pass over the data:
//   r' = r + delta;  f = 1 / sqrt(mean(r'^2) + eps);  o = (r' f) w      (fp32, not rounded)
//   amax = max |o|;  q = clamp(rint(o 127/amax), +-127);  s_x = amax/127
// and, if asked, val = bf16(s_x q): the values that the int8 product sees, as a bf16 operand.
// o goes into the quantiser unrounded (the separate calls round it to bf16 in between, which
// moves s_x by up to 2^-9).
//
// The gradient, straight through the quantiser (dout is the gradient with respect to o):
//   g = dout w;  c = sum(g r)/d;  dr = f g - (f^3 c) r (+ dstream);  dw = sum_t dout (r f)
//
// Both move a few bytes per element and compute little: bound by HBM for many tokens, by the
// launch for one. A row belongs to TPR threads (8 up to 64 channels, a warp up to 1024, a CTA above), each of
// which holds NV pieces of 8 columns in registers from the only load to the only store, so no
// byte moves twice; the row's sums go through shuffles and, for TPR = 256, one shared-memory
// step. The gradient's CTAs are persistent, so that dw accumulates in registers over a CTA's
// rows; one partial row per CTA goes to the workspace and a second kernel adds the partials.
// Every order of summation is fixed by m and d.
//
// Measured, 16,384 x 2048 with a bf16 delta: forward 72 us with the L2 flushed before it, 6.1 TB/s (66 back to back from a
// graph, where the next call overwrites what is still in the L2); gradient with dw 88 us, 5.3 TB/s (84). One token: the
// launch, 2.4 us in a graph, 5 us with the gradient's two.
#include <cmath>
#include <cstdint>

#include "dfssm_internal.cuh"
#include "epilogue.cuh"

namespace dfssm {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxD = 8192;
// CTAs of the gradient per SM: what the registers allow up to 256 and for 1,025 to 2,048 channels (80 to 89 of them). Where a
// thread holds more pieces of a row (124 to 254 registers) one or two CTAs fit, and the grid goes in two or three turns.
constexpr int kBwdCtasPerSm = 3;
constexpr int kBwdMaxCtas = 148 * kBwdCtasPerSm;   // partial rows of dw in the workspace

__device__ __forceinline__ void load8(const float* p, float v[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(float* p, const float v[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void load8_bf16(const void* base, int64_t i, float v[8]) {
    const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[2 * k] = bf16_lo(w[k]);
        v[2 * k + 1] = bf16_hi(w[k]);
    }
}

// Sum, or max of bit patterns of |x|, over the TPR threads of a row; every thread gets it. `red` holds one
// slot per warp; a second use needs another array (no barrier behind the read).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (TPR > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int w = 1; w < kThreads / 32; ++w) v = __fadd_rn(v, red[w]);
    }
    return v;
}
template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (TPR > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int w = 1; w < kThreads / 32; ++w) v = max(v, red[w]);
    }
    return v;
}

__device__ __forceinline__ float norm_factor(float ss, int d, float eps) {
    return __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)d), eps)));
}

// ------------------------------------------------------------------------------- forward

struct Q8Args {
    const float* w;
    const float* rin;
    const void* delta;
    float* rout;
    int8_t* q;
    float* sx;
    uint16_t* val;
    int d, m;
    float eps;
    int delta_bf16;
};

template <int TPR, int NV>
__global__ void __launch_bounds__(kThreads) add_rmsnorm_quant_kernel(const Q8Args a) {
    __shared__ float red[kThreads / 32];
    __shared__ uint32_t redm[kThreads / 32];
    const int sub = threadIdx.x % TPR;
    const int row = blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
    const bool live = row < a.m;
    const int64_t base = (int64_t)row * a.d;
    float v[NV][8];
    float ss = 0.0f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int c = 8 * (sub + TPR * n);
        if (live && c < a.d) {
            load8(a.rin + base + c, v[n]);
            if (a.delta) {
                float dv[8];
                if (a.delta_bf16) load8_bf16(a.delta, base + c, dv);
                else load8(static_cast<const float*>(a.delta) + base + c, dv);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[n][k] = __fadd_rn(v[n][k], dv[k]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[n][k] = 0.0f;
        }
    }
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int c = 8 * (sub + TPR * n);
        if (live && c < a.d) store8(a.rout + base + c, v[n]);
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = __fmaf_rn(v[n][k], v[n][k], ss);
    }
    const float f = norm_factor(row_sum<TPR>(ss, red), a.d, a.eps);
    uint32_t am = 0u;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int c = 8 * (sub + TPR * n);
        if (live && c < a.d) {
            float w[8];
            load8(a.w + c, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[n][k] = __fmul_rn(__fmul_rn(v[n][k], f), w[k]);
                am = max(am, __float_as_uint(v[n][k]) & 0x7FFFFFFFu);
            }
        }
    }
    const float amax = __uint_as_float(row_max<TPR>(am, redm));
    const bool zero = amax == 0.0f;
    const float inv = quant_inv(amax), sx = quant_sx(amax);
    if (live && sub == 0) a.sx[row] = sx;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int c = 8 * (sub + TPR * n);
        if (!live || c >= a.d) continue;
        int q[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) q[k] = quant1(v[n][k], inv, zero);
        uint2 p;
        p.x = (uint32_t)(q[0] & 0xFF) | ((uint32_t)(q[1] & 0xFF) << 8) | ((uint32_t)(q[2] & 0xFF) << 16) |
              ((uint32_t)(q[3] & 0xFF) << 24);
        p.y = (uint32_t)(q[4] & 0xFF) | ((uint32_t)(q[5] & 0xFF) << 8) | ((uint32_t)(q[6] & 0xFF) << 16) |
              ((uint32_t)(q[7] & 0xFF) << 24);
        *reinterpret_cast<uint2*>(a.q + base + c) = p;
        if (a.val) {
            uint32_t b[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                b[k] = bf16x2_of(make_float2(__fmul_rn(sx, small_int_to_float(q[2 * k])),
                                             __fmul_rn(sx, small_int_to_float(q[2 * k + 1]))));
            *reinterpret_cast<uint4*>(a.val + base + c) = make_uint4(b[0], b[1], b[2], b[3]);
        }
    }
}

// ------------------------------------------------------------------------------- gradient

struct BwdArgs {
    const float* w;
    const float* r;
    const void* dout;
    const float* dstream;
    float* dr;
    float* part;     // [gridDim.x][d] partial dw, or NULL
    int d, m;
    float eps;
    int dout_bf16;
};

// One row group's loads in flight: the next rows' while the current ones are reduced and stored
// (16,384 x 2048 with a bf16 gradient and a stream gradient, the call: 94 -> 88 us).
template <int NV, bool BF>
struct BwdRow {
    float r[NV][8];
    uint32_t g[NV][BF ? 4 : 8];
    float ds[NV][8];
};

template <int TPR, int NV, bool BF>
__device__ __forceinline__ void bwd_load(const BwdArgs& a, int row, int sub, BwdRow<NV, BF>& v) {
    const int64_t base = (int64_t)row * a.d;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int c = 8 * (sub + TPR * n);
        const bool in = row < a.m && c < a.d;
#pragma unroll
        for (int k = 0; k < 8; ++k) v.r[n][k] = v.ds[n][k] = 0.0f;
#pragma unroll
        for (int k = 0; k < (BF ? 4 : 8); ++k) v.g[n][k] = 0u;
        if (!in) continue;
        load8(a.r + base + c, v.r[n]);
        if (BF) {
            const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.dout) + base + c);
            v.g[n][0] = q.x; v.g[n][1] = q.y; v.g[n][2] = q.z; v.g[n][3] = q.w;
        } else {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(a.dout) + base + c);
            const uint4 x = p[0], y = p[1];
            v.g[n][0] = x.x; v.g[n][1] = x.y; v.g[n][2] = x.z; v.g[n][3] = x.w;
            v.g[n][BF ? 0 : 4] = y.x; v.g[n][BF ? 0 : 5] = y.y; v.g[n][BF ? 0 : 6] = y.z; v.g[n][BF ? 0 : 7] = y.w;
        }
        if (a.dstream) load8(a.dstream + base + c, v.ds[n]);
    }
}

template <int NV, bool BF>
__device__ __forceinline__ float bwd_g(const BwdRow<NV, BF>& v, int n, int k) {
    if (BF) return (k & 1) ? bf16_hi(v.g[n][k >> 1]) : bf16_lo(v.g[n][k >> 1]);
    return __uint_as_float(v.g[n][BF ? 0 : k]);
}

template <int TPR, int NV, bool BF>
__global__ void __launch_bounds__(kThreads) add_rmsnorm_bwd_kernel(const BwdArgs a) {
    constexpr int kRows = kThreads / TPR;
    __shared__ float2 red[2][kThreads / 32];     // [row parity]: a slot is reused two barriers later
    const int sub = threadIdx.x % TPR, in_row = threadIdx.x / TPR;
    float dw[NV][8];
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int k = 0; k < 8; ++k) dw[n][k] = 0.0f;
    int par = 0;
    BwdRow<NV, BF> cur, nxt;
    bwd_load<TPR, NV, BF>(a, blockIdx.x * kRows + in_row, sub, cur);
    for (int row0 = blockIdx.x * kRows; row0 < a.m; row0 += gridDim.x * kRows, par ^= 1) {
        const int row = row0 + in_row;
        const bool live = row < a.m;
        const int64_t base = (int64_t)row * a.d;
        bwd_load<TPR, NV, BF>(a, min(row + (int)gridDim.x * kRows, a.m), sub, nxt);
        float ss = 0.0f, gr = 0.0f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c = 8 * (sub + TPR * n);
            float w[8];
            if (c < a.d) load8(a.w + c, w);
            else
#pragma unroll
                for (int k = 0; k < 8; ++k) w[k] = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                ss = __fmaf_rn(cur.r[n][k], cur.r[n][k], ss);
                gr = __fmaf_rn(__fmul_rn(bwd_g(cur, n, k), w[k]), cur.r[n][k], gr);
            }
        }
#pragma unroll
        for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
            ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, o));
            gr = __fadd_rn(gr, __shfl_xor_sync(0xffffffffu, gr, o));
        }
        if (TPR > 32) {
            if ((threadIdx.x & 31) == 0) red[par][threadIdx.x >> 5] = make_float2(ss, gr);
            __syncthreads();
            ss = red[par][0].x;
            gr = red[par][0].y;
#pragma unroll
            for (int w = 1; w < kThreads / 32; ++w) {
                ss = __fadd_rn(ss, red[par][w].x);
                gr = __fadd_rn(gr, red[par][w].y);
            }
        }
        const float f = norm_factor(ss, a.d, a.eps);
        const float c3 = __fmul_rn(__fmul_rn(__fmul_rn(f, f), f), __fdiv_rn(gr, (float)a.d));
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c = 8 * (sub + TPR * n);
            if (!live || c >= a.d) continue;
            float w[8], o[8];
            load8(a.w + c, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float g = bwd_g(cur, n, k);
                o[k] = __fmaf_rn(-c3, cur.r[n][k], __fmul_rn(f, __fmul_rn(g, w[k])));
                if (a.dstream) o[k] = __fadd_rn(o[k], cur.ds[n][k]);
                dw[n][k] = __fmaf_rn(g, __fmul_rn(cur.r[n][k], f), dw[n][k]);
            }
            store8(a.dr + base + c, o);
        }
        cur = nxt;
    }
    if (!a.part) return;
    // the CTA's partial dw: its row groups added in order
    if (TPR == kThreads) {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c = 8 * (sub + TPR * n);
            if (c < a.d) store8(a.part + (int64_t)blockIdx.x * a.d + c, dw[n]);
        }
    } else {
        extern __shared__ float sdw[];                   // [kRows][TPR * NV * 8]
        constexpr int kCols = TPR * NV * 8;
#pragma unroll
        for (int n = 0; n < NV; ++n) store8(sdw + (threadIdx.x / TPR) * kCols + 8 * (sub + TPR * n), dw[n]);
        __syncthreads();
        for (int c = threadIdx.x; c < a.d; c += kThreads) {
            float s = sdw[c];
            for (int g = 1; g < kRows; ++g) s = __fadd_rn(s, sdw[g * kCols + c]);
            a.part[(int64_t)blockIdx.x * a.d + c] = s;
        }
    }
}

// dw[c] = sum over the partial rows: 32 columns per CTA, 32 row groups added in order
__global__ void __launch_bounds__(1024) dw_reduce_kernel(const float* __restrict__ part, int n, int d, float* dw) {
    __shared__ float s[32][33];
    const int cl = threadIdx.x & 31, g = threadIdx.x >> 5, c = blockIdx.x * 32 + cl;
    float acc = 0.0f;
    if (c < d) {
#pragma unroll 8
        for (int i = g; i < n; i += 32) acc = __fadd_rn(acc, part[(int64_t)i * d + c]);
    }
    s[g][cl] = acc;
    __syncthreads();
    if (g == 0 && c < d) {
#pragma unroll
        for (int k = 1; k < 32; ++k) acc = __fadd_rn(acc, s[k][cl]);
        dw[c] = acc;
    }
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int bwd_rows(int d) { return d <= 64 ? kThreads / 8 : d <= 1024 ? kThreads / 32 : 1; }
int bwd_ctas(int d, int m) {
    const int need = (m + bwd_rows(d) - 1) / bwd_rows(d);
    return need < kBwdMaxCtas ? need : kBwdMaxCtas;
}

template <int TPR, int NV>
cudaError_t launch_q8(const Q8Args& a, cudaStream_t s) {
    constexpr int rows = kThreads / TPR;
    add_rmsnorm_quant_kernel<TPR, NV><<<(a.m + rows - 1) / rows, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}
template <int TPR, int NV>
cudaError_t launch_bwd(const BwdArgs& a, cudaStream_t s) {
    constexpr int rows = kThreads / TPR;
    const size_t smem = TPR == kThreads ? 0 : sizeof(float) * rows * TPR * NV * 8;   // at most 32 KB
    if (a.dout_bf16) add_rmsnorm_bwd_kernel<TPR, NV, true><<<bwd_ctas(a.d, a.m), kThreads, smem, s>>>(a);
    else add_rmsnorm_bwd_kernel<TPR, NV, false><<<bwd_ctas(a.d, a.m), kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

}  // namespace dfssm

using namespace dfssm;

extern "C" dfssm_status dfssm_add_rmsnorm_quant(const float* norm_w, int32_t d, float eps, const float* resid_in,
                                             const void* delta, int32_t delta_dtype, int32_t m, float* resid_out,
                                             int8_t* q, float* sx, void* val, void* stream) {
    if (d < 8 || d > kMaxD || d % 8 != 0 || m < 1 || m > 65536) return DFSSM_ERR_UNSUPPORTED_SHAPE;
    if (!norm_w || !resid_in || !resid_out || !q || !sx || !al16(norm_w) || !al16(resid_in) || !al16(resid_out) ||
        !al16(q) || !al16(sx) || !al16(delta) || !al16(val))
        return DFSSM_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 0.0f) return DFSSM_ERR_INVALID_ARG;
    if (delta && delta_dtype != DFSSM_BF16 && delta_dtype != DFSSM_F32) return DFSSM_ERR_INVALID_ARG;
    const Q8Args a{norm_w, resid_in, delta, resid_out, q, sx, static_cast<uint16_t*>(val), d, m, eps,
                   delta_dtype == DFSSM_BF16 ? 1 : 0};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (d <= 64) e = launch_q8<8, 1>(a, s);
    else if (d <= 256) e = launch_q8<32, 1>(a, s);
    else if (d <= 512) e = launch_q8<32, 2>(a, s);
    else if (d <= 1024) e = launch_q8<32, 4>(a, s);
    else if (d <= 2048) e = launch_q8<256, 1>(a, s);
    else if (d <= 4096) e = launch_q8<256, 2>(a, s);
    else e = launch_q8<256, 4>(a, s);
    return e == cudaSuccess ? DFSSM_OK : DFSSM_ERR_CUDA;
}

extern "C" dfssm_status dfssm_add_rmsnorm_bwd_workspace_bytes(int32_t d, int32_t m, size_t* bytes) {
    if (d < 8 || d > kMaxD || d % 8 != 0 || m < 1 || m > 65536) return DFSSM_ERR_UNSUPPORTED_SHAPE;
    if (!bytes) return DFSSM_ERR_INVALID_ARG;
    *bytes = (size_t)bwd_ctas(d, m) * d * sizeof(float);
    return DFSSM_OK;
}

extern "C" dfssm_status dfssm_add_rmsnorm_bwd(const float* norm_w, int32_t d, float eps, const float* resid,
                                              const void* dout, int32_t dout_dtype, const float* dstream, int32_t m,
                                              float* dresid, float* dnorm_w, void* workspace, size_t workspace_bytes,
                                              void* stream) {
    size_t need = 0;
    const dfssm_status st = dfssm_add_rmsnorm_bwd_workspace_bytes(d, m, &need);
    if (st != DFSSM_OK) return st;
    if (!norm_w || !resid || !dout || !dresid || !al16(norm_w) || !al16(resid) || !al16(dout) || !al16(dstream) ||
        !al16(dresid) || !al16(dnorm_w))
        return DFSSM_ERR_INVALID_ARG;
    if (dnorm_w && (!workspace || !al16(workspace) || workspace_bytes < need)) return DFSSM_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 0.0f) return DFSSM_ERR_INVALID_ARG;
    if (dout_dtype != DFSSM_BF16 && dout_dtype != DFSSM_F32) return DFSSM_ERR_INVALID_ARG;
    const BwdArgs a{norm_w, resid, dout, dstream, dresid, dnorm_w ? static_cast<float*>(workspace) : nullptr, d, m, eps,
                    dout_dtype == DFSSM_BF16 ? 1 : 0};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (d <= 64) e = launch_bwd<8, 1>(a, s);
    else if (d <= 256) e = launch_bwd<32, 1>(a, s);
    else if (d <= 512) e = launch_bwd<32, 2>(a, s);
    else if (d <= 1024) e = launch_bwd<32, 4>(a, s);
    else if (d <= 2048) e = launch_bwd<256, 1>(a, s);
    else if (d <= 4096) e = launch_bwd<256, 2>(a, s);
    else e = launch_bwd<256, 4>(a, s);
    if (e == cudaSuccess && dnorm_w) {
        dw_reduce_kernel<<<(d + 31) / 32, 1024, 0, s>>>(a.part, bwd_ctas(d, m), d, dnorm_w);
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? DFSSM_OK : DFSSM_ERR_CUDA;
}
