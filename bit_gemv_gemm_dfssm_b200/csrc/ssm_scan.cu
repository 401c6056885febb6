// The state operations' recurrence over packed sequences of any length (dfssm_ssm_scan_fwd): what ssm_step.cu does for one
// token, for the tokens of a prompt or a training batch. This file has the work table, the forward kernel of short
// calls, the kernels that carry states alone through a sequence, and the call's plan; ssm_scan_tc.cu has the forward
// kernel of long calls, ssm_scan_bwd.cu the gradient.
//
// A CTA takes one head through one item (a sequence, or a segment of a long one), chunk by chunk (ssm_scan.cuh has the
// formulas), with the head's 64 x 128 state in fp32 registers. One CTA per (head, item) fills the GPU from two or three
// sequences of 64 heads on; with fewer, long sequences are cut into segments, whose start states come from two
// small kernels before (each segment's own contribution, state products only; then a carry over the segments).
// Items are handed out longest first.
//
// Operands are fp16 under power-of-two scales: x, B and C (bf16) enter exactly over 2^17 and more of range below their
// chunk's largest value; M = G exp(cum_t - cum_s) dt_s and the state as the readout's operand are one fp16 number
// each (2^-11 of the value, beside the output's own 2^-8); the weighted x that goes into the state is two (2^-23),
// so that the state, which goes on to the next tokens and is returned, keeps fp32's precision.
//
// Short calls (scan_fwd_kernel, warp MMAs, chunks of 64 tokens) are one launch that converts its tiles itself. What a
// call of a few tokens costs is one launch, one chunk's chain of loads, products and exchanges, and the
// states: 64 heads, 5.5 us for one sequence of 1 to 16 tokens, 8.8 for 64, 14 for 128.
#include <mutex>
#include <type_traits>

#include "ssm_scan.cuh"

namespace dfssm {
namespace scan {

namespace {

// ------------------------------------------------------------------------------- the work table

constexpr int kTableThreads = 1024;
constexpr int kMaxSorted = 1024;

// inclusive sum over the CTA; every thread gets its own and the total
__device__ __forceinline__ int block_scan(int v, int* red, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();
    if (lane == 31) red[warp] = v;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int w = 0; w < kTableThreads / 32; ++w) {
        if (w < warp) before += red[w];
        total += red[w];
    }
    return v + before;
}

// One CTA: validates the offsets, cuts the sequences, numbers items and chunks. A sequence whose offsets
// do not fit is left out (and reported).
__global__ void __launch_bounds__(kTableThreads) scan_table_kernel(const Args a) {
    __shared__ int red[kTableThreads / 32];
    __shared__ int lens[kMaxSorted];
    __shared__ int end[2];               // items and chunks in front of the first sequence that does not fit
    ptx::pdl_launch_dependents();
    if (threadIdx.x < 2) end[threadIdx.x] = 0x7FFFFFFF;
    int n_items = 0, n_chunks = 0, n_slots = 0;
    for (int s0 = 0; s0 < a.nseq; s0 += kTableThreads) {
        const int s = s0 + threadIdx.x;
        int t0 = 0, len = 0, nseg = 0, nch = 0;
        if (s < a.nseq) {
            t0 = a.cu[s];
            const int t1 = a.cu[s + 1];
            if (t0 < 0 || t1 < t0 || t1 > a.total) {
                atomicOr(a.err, DFSSM_DEVERR_SEQLENS);
            } else {
                len = t1 - t0;
                nseg = len <= a.cut_at ? 1 : (len + a.seg_len - 1) / a.seg_len;
                nch = (len + a.chunk - 1) / a.chunk;
            }
        }
        int ti = 0, tc = 0, ts = 0;
        const int cut = nseg > 1 ? nseg : 0;
        const int i1 = n_items + block_scan(nseg, red, ti);
        const int c1 = n_chunks + block_scan(nch, red, tc);
        const int s1 = n_slots + block_scan(cut, red, ts);
        // Overlapping offsets could ask for more than the workspace holds. From the first sequence on that does not fit
        // (the sums only grow) all are left out, so that every counted item and chunk is written below.
        const bool fits = i1 <= a.cap_items && c1 <= a.cap_chunks && s1 <= a.cap_slots && end[0] == 0x7FFFFFFF;
        __syncthreads();                // end[] of the sequences before is read
        if (s < a.nseq) {
            const int i0 = i1 - nseg, c0 = c1 - nch;
            a.seq_slots[s] = fits ? make_int2(s1 - cut, cut) : make_int2(0, 0);
            if (!fits) {
                atomicOr(a.err, DFSSM_DEVERR_SEQLENS);
                atomicMin(&end[0], i0);
                atomicMin(&end[1], c0);
            } else {
                for (int k = 0; k < nseg; ++k) {
                    const int at = k * a.seg_len;
                    a.seq_items[i0 + k] = Item{s, t0 + at, nseg == 1 ? len : min(a.seg_len, len - at), c0 + at / a.chunk, s1 - cut + k,
                                               (k == 0 ? kFirst : 0) | (k == nseg - 1 ? kLast : 0) | (nseg > 1 ? kCut : 0)};
                }
            }
        }
        n_items = min(n_items + ti, a.cap_items);
        n_chunks = min(n_chunks + tc, a.cap_chunks);
        n_slots = min(n_slots + ts, a.cap_slots);
        __syncthreads();                // end[] is written
    }
    n_items = min(n_items, end[0]);
    n_chunks = min(n_chunks, end[1]);
    __syncthreads();                    // the items of this CTA are visible to it
    if (threadIdx.x == 0) {
        a.count[0] = n_items;
        a.count[1] = n_chunks;
    }
    const bool sorted = n_items <= kMaxSorted;
    if (sorted)
        for (int i = threadIdx.x; i < n_items; i += kTableThreads) lens[i] = a.seq_items[i].len;
    __syncthreads();
    for (int i = threadIdx.x; i < n_items; i += kTableThreads) {
        int rank = i;
        if (sorted) {
            const int mine = lens[i];
            rank = 0;
            for (int j = 0; j < n_items; ++j) rank += lens[j] > mine || (lens[j] == mine && j < i);
        }
        a.items[rank] = a.seq_items[i];
    }
    for (int i = threadIdx.x >> 5; i < n_items; i += kTableThreads / 32) {
        const Item it = a.seq_items[i];
        for (int k = threadIdx.x & 31; a.chunk * k < it.len; k += 32)
            a.chunks[it.chunk0 + k] = Chunk{it.t0 + a.chunk * k, min(a.chunk, it.len - a.chunk * k)};
    }
}

// ------------------------------------------------------------------------------- forward

struct FwdOut {
    uint16_t* y;
    int64_t ldy;
    float* final_state;        // or NULL
};

// ---- B and C in fp16
// fp16 holds a bf16 value exactly over 2^-24 .. 2^15; a tile is scaled by a power of two that brings its
// largest magnitude to [2^3, 2^4), so that only values below 2^-17 of that lose bits, and G = C B^T stays below 2^15.

constexpr int kTileTop = 3;

// CTA (chunk, group, C or B): the tile, rows behind the chunk's tokens as zeros
__global__ void __launch_bounds__(512) scan_tiles_kernel(const Args a) {
    __shared__ uint32_t red[16];
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    const int ngroups = a.nheads / a.per_group;
    const int side = blockIdx.x & 1, g = (blockIdx.x >> 1) % ngroups, ci = (blockIdx.x >> 1) / ngroups;
    if (ci >= a.count[1]) return;
    const Chunk ch = a.chunks[ci];
    const uint16_t* src = (side ? a.b : a.c) + (int64_t)g * kN;
    const int64_t ld = side ? a.ldb : a.ldc;
    uint4 v[4];
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = (threadIdx.x >> 4) + 32 * i, pc = threadIdx.x & 15;
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (row < ch.n) v[i] = *reinterpret_cast<const uint4*>(src + (int64_t)(ch.t0 + row) * ld + 8 * pc);
        m = abs_max_bf16x2(abs_max_bf16x2(abs_max_bf16x2(abs_max_bf16x2(m, v[i].x), v[i].y), v[i].z), v[i].w);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 16; ++w) m = max(m, red[w]);
    const float2 sc = pow2_scale(m, kTileTop);
    uint16_t* dst = a.tiles + (((int64_t)ci * ngroups + g) * 2 + side) * (128 * kN);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(dst + 8 * (threadIdx.x + 512 * i)) =
            make_uint4(bf16x2_to_f16x2(v[i].x, sc.x), bf16x2_to_f16x2(v[i].y, sc.x), bf16x2_to_f16x2(v[i].z, sc.x),
                       bf16x2_to_f16x2(v[i].w, sc.x));
    if (threadIdx.x == 0) (side ? &a.tile_scale[(int64_t)ci * ngroups + g].y : &a.tile_scale[(int64_t)ci * ngroups + g].x)[0] = sc.y;
}

// ---- the forward kernel
constexpr int kFwdThreads = 256;
constexpr int kStage = 16384 + 16384 + 8192;          // C, B, X of one chunk
struct FwdDecay {
    float cum[kQ];       // log 2 units
    float dts[kQ];       // dt 2^kd, the largest in [1/2, 1)
    float wl[kQ];        // dts exp(cum_64 - cum_t)
    float done[kQ];      // exp(cum_t)
    float kd;            // 2^-kd
    float pad[3];
};
constexpr int kFwdX = 16384;                          // y's parts that a warp hands to its partner
constexpr int kFwdSmem = 2 * kStage + 8192 + kFwdX + 2 * (int)sizeof(FwdDecay) + 128 + 128;

__device__ __forceinline__ void fwd_decay(FwdDecay& f, Decay& d, float raw0, float raw1, int n, float bias, float a2,
                                          int lane) {
    chunk_decay(d, raw0, raw1, n, bias, a2, lane);
    __syncwarp();
    const float2 cum = reinterpret_cast<const float2*>(d.cum)[lane], dt = reinterpret_cast<const float2*>(d.dt)[lane];
    const float2 left = reinterpret_cast<const float2*>(d.left)[lane];
    const uint32_t m = __reduce_max_sync(0xffffffffu, max(__float_as_uint(dt.x), __float_as_uint(dt.y)));
    const float2 sc = pow2_scale(m, -1);
    const float2 ds = make_float2(__fmul_rn(dt.x, sc.x), __fmul_rn(dt.y, sc.x));
    reinterpret_cast<float2*>(f.cum)[lane] = cum;
    reinterpret_cast<float2*>(f.dts)[lane] = ds;
    reinterpret_cast<float2*>(f.wl)[lane] = make_float2(__fmul_rn(ds.x, left.x), __fmul_rn(ds.y, left.y));
    reinterpret_cast<float2*>(f.done)[lane] = reinterpret_cast<const float2*>(d.done)[lane];
    if (lane == 0) f.kd = sc.y;
}

// The kernel of short calls: it converts each chunk's tiles of B and C itself, so that a call is one launch.
__global__ void __launch_bounds__(kFwdThreads, 2) scan_fwd_kernel(const Args a, const FwdOut o) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ Decay scratch;                         // of warp 0
    const uint32_t base = (ptx::smem_u32(smem_raw) + 127u) & ~127u;
    uint8_t* smem = smem_raw + (base - ptx::smem_u32(smem_raw));
    const uint32_t s_m = base + 2 * kStage, s_ex = s_m + 8192;
    FwdDecay* dec = reinterpret_cast<FwdDecay*>(smem + 2 * kStage + 8192 + kFwdX);
    uint32_t* s_max = reinterpret_cast<uint32_t*>(dec + 2);                // [2][8]
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int pw = w & 3, hv = w >> 2;                // channels 16 pw ..; states 64 hv ..; tokens 32 hv .. of y
    const int h = blockIdx.x % a.nheads, g = h / a.per_group;
    Item it;
    if (!get_item(a, blockIdx.x / a.nheads, it) || it.len < 0) return;
    const int n_ch = (it.len + kQ - 1) / kQ;

    const uint16_t* x = a.x + (int64_t)h * kP;
    const uint16_t* b = a.b + (int64_t)g * kN;
    const uint16_t* c = a.c + (int64_t)g * kN;
    auto fetch = [&](int k) {
        if (k < n_ch) {
            const int t0 = it.t0 + k * kQ, n = min(kQ, it.len - k * kQ);
            const uint32_t st = base + (k & 1) * kStage;
            load_tile<128, kFwdThreads>(st, c, a.ldc, t0, n, tid);
            load_tile<128, kFwdThreads>(st + 16384, b, a.ldb, t0, n, tid);
            load_tile<64, kFwdThreads>(st + 32768, x, a.ldx, t0, n, tid);
        }
        ptx::cp_async_commit();
    };
    fetch(0);
    const float bias = a.dt_bias[h], a2 = __fmul_rn(-expf(a.a_log[h]), kLog2e), skip = a.d_skip[h];
    // the warp's part of the state: 16 channels x 64 states, 8 accumulator tiles
    float S[8][4];
    const int64_t sh = ((int64_t)it.seq * a.nheads + h) * kStateElems;
    const int s_at = (16 * pw + (lane >> 2)) * kN + 64 * hv + 2 * (lane & 3);
    {
        const float* src = a.init ? a.init + sh : nullptr;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float2 lo = make_float2(0.0f, 0.0f), hi = lo;
            if (src) {
                lo = *reinterpret_cast<const float2*>(src + s_at + 8 * j);
                hi = *reinterpret_cast<const float2*>(src + s_at + 8 * kN + 8 * j);
            }
            S[j][0] = lo.x; S[j][1] = lo.y; S[j][2] = hi.x; S[j][3] = hi.y;
        }
    }
    float raw0 = 0.0f, raw1 = 0.0f;
    auto raws = [&](int k) {
        if (w != 0 || k >= n_ch) return;
        const int t0 = it.t0 + k * kQ, n = min(kQ, it.len - k * kQ);
        raw0 = raw_dt(a, t0, n, h, 2 * lane);
        raw1 = raw_dt(a, t0, n, h, 2 * lane + 1);
    };
    auto decay = [&](int k) {
        if (w != 0 || k >= n_ch) return;
        fwd_decay(dec[k & 1], scratch, raw0, raw1, min(kQ, it.len - k * kQ), bias, a2, lane);
    };
    raws(0);
    decay(0);
    raws(1);
    // A chunk, of whose four blocks of 16 tokens the first `blocks` hold tokens; what lies behind is neither worked on nor
    // read. Short chunks (up to 16 and up to 32 tokens, a server's few at a time) have their own code: 64 sequences of
    // 8 tokens, 64 heads 153 -> 98 us, one of 1 token 8.6 -> 5.5 us, 16 of 32 40 -> 31 us; with the count at run time, full
    // chunks lost a quarter.
    auto chunk = [&](int k, auto blocks) {
        constexpr int nb = decltype(blocks)::value;
        const int t0 = it.t0 + k * kQ, n = min(kQ, it.len - k * kQ);
        const uint32_t st = base + (k & 1) * kStage;
        const uint32_t s_c = st, s_b = st + 16384, s_x = st + 32768;
        const FwdDecay& d = dec[k & 1];
        ptx::cp_async_wait<0>();
        __syncthreads();                 // this chunk's tiles and decays are there; the last one's are free
        fetch(k + 1);
        float2 tsc;                      // 2^-k of C and of B
        {
            uint4 v[2][4];
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                uint32_t m = 0u;
#pragma unroll
                for (int i = 0; i < 4; ++i) {     // 16 rows; the zeros behind the tokens are the same in fp16
                    if (i >= nb) break;
                    v[side][i] = ptx::lds128(st + 16384 * side + 16 * (tid + kFwdThreads * i));
                    m = abs_max_bf16x2(abs_max_bf16x2(abs_max_bf16x2(abs_max_bf16x2(m, v[side][i].x), v[side][i].y),
                                                      v[side][i].z), v[side][i].w);
                }
                m = __reduce_max_sync(0xffffffffu, m);
                if (lane == 0) s_max[8 * side + w] = m;
            }
            __syncthreads();
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                uint32_t m = 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = max(m, s_max[8 * side + i]);
                const float2 sc = pow2_scale(m, kTileTop);
                (side ? tsc.y : tsc.x) = sc.y;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i >= nb) break;
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};"
                                 ::"r"(st + 16384 * side + 16 * (tid + kFwdThreads * i)),
                                 "r"(bf16x2_to_f16x2(v[side][i].x, sc.x)), "r"(bf16x2_to_f16x2(v[side][i].y, sc.x)),
                                 "r"(bf16x2_to_f16x2(v[side][i].z, sc.x)), "r"(bf16x2_to_f16x2(v[side][i].w, sc.x)) : "memory");
                }
            }
            __syncthreads();
        }

        // ---- M in fp16, rows 16 pw + lane / 4 (+ 8), columns in blocks hv and hv + 2 of 16 up to the diagonal
        if (pw < nb) {
            float G[2][2][4];
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int j = 0; j < 2; ++j) G[q][j][0] = G[q][j][1] = G[q][j][2] = G[q][j][3] = 0.0f;
            if (hv <= pw) {
#pragma unroll
                for (int kk = 0; kk < kN; kk += 16) {
                    uint32_t ca[4];
                    frag_a<256>(s_c, 16 * pw, kk, lane, ca);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        if (hv + 2 * q > pw) break;
                        uint32_t bb[4];
                        frag_b<256>(s_b, 16 * (hv + 2 * q), kk, lane, bb);
                        mma_h(G[q][0], ca, bb[0], bb[1]);
                        mma_h(G[q][1], ca, bb[2], bb[3]);
                    }
                }
            }
            const int r = 16 * pw + (lane >> 2);
            const float c0 = d.cum[r], c1 = d.cum[r + 8];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int blk = hv + 2 * q;
                if (blk > pw) break;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int s = 16 * blk + 8 * j + 2 * (lane & 3);
                    const float2 cs = *reinterpret_cast<const float2*>(d.cum + s);
                    const float2 ds = *reinterpret_cast<const float2*>(d.dts + s);
                    float m[4];
                    m[0] = __fmul_rn(__fmul_rn(G[q][j][0], ds.x), ex2(__fsub_rn(c0, cs.x)));
                    m[1] = __fmul_rn(__fmul_rn(G[q][j][1], ds.y), ex2(__fsub_rn(c0, cs.y)));
                    m[2] = __fmul_rn(__fmul_rn(G[q][j][2], ds.x), ex2(__fsub_rn(c1, cs.x)));
                    m[3] = __fmul_rn(__fmul_rn(G[q][j][3], ds.y), ex2(__fsub_rn(c1, cs.y)));
                    if (blk == pw) {             // the diagonal
                        if (s > r) m[0] = 0.0f;
                        if (s + 1 > r) m[1] = 0.0f;
                        if (s > r + 8) m[2] = 0.0f;
                        if (s + 1 > r + 8) m[3] = 0.0f;
                    }
                    ptx::sts32(tile128(s_m, r, 2 * blk + j) + 4 * (lane & 3), f16x2_of(m[0], m[1]));
                    ptx::sts32(tile128(s_m, r + 8, 2 * blk + j) + 4 * (lane & 3), f16x2_of(m[2], m[3]));
                }
            }
        }
        decay(k + 1);                    // warp 0, which has the fewest blocks of M
        raws(k + 2);
        // ---- the state's readout over the warp's 64 states, for all 64 tokens
        float y[4][2][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int p = 0; p < 2; ++p) y[i][p][0] = y[i][p][1] = y[i][p][2] = y[i][p][3] = 0.0f;
        {
            uint32_t m = 0u;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) m = max(m, __float_as_uint(S[j][q]) & 0x7FFFFFFFu);
            m = __reduce_max_sync(0xffffffffu, m);
            const float2 ss = pow2_scale(m, 13);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                uint32_t sb[4];          // [2 * channel tile + k half]
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    sb[q] = f16x2_of(__fmul_rn(S[2 * kk + (q & 1)][q & 2], ss.x), __fmul_rn(S[2 * kk + (q & 1)][(q & 2) + 1], ss.x));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i >= nb) break;
                    uint32_t ca[4];
                    frag_a<256>(s_c, 16 * i, 64 * hv + 16 * kk, lane, ca);
                    mma_h(y[i][0], ca, sb[0], sb[1]);
                    mma_h(y[i][1], ca, sb[2], sb[3]);
                }
            }
            // the other half's tokens go to the warp that has the other 64 states of these channels
            const float back = __fmul_rn(ss.y, tsc.x);
            const uint32_t ex = s_ex + (uint32_t)((pw * 2 + (hv ^ 1)) * 2048 + lane * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i >= nb) break;
                const float e0 = __fmul_rn(d.done[16 * i + (lane >> 2)], back), e1 = __fmul_rn(d.done[16 * i + 8 + (lane >> 2)], back);
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    y[i][p][0] = __fmul_rn(y[i][p][0], e0);
                    y[i][p][1] = __fmul_rn(y[i][p][1], e0);
                    y[i][p][2] = __fmul_rn(y[i][p][2], e1);
                    y[i][p][3] = __fmul_rn(y[i][p][3], e1);
                    if ((i >> 1) != hv)
                        asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};"
                                     ::"r"(ex + (uint32_t)(((i & 1) * 2 + p) * 512)), "f"(y[i][p][0]), "f"(y[i][p][1]),
                                     "f"(y[i][p][2]), "f"(y[i][p][3]) : "memory");
                }
            }
        }
        // ---- the scale of x over the warp's channels
        uint32_t xm = 0u;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            if (ks >= nb) break;
            uint32_t xa[4];
            frag_at<128>(s_x, 16 * ks, 16 * pw, lane, xa);
#pragma unroll
            for (int q = 0; q < 4; ++q) xm = abs_max_bf16x2(xm, xa[q]);
        }
        const float2 xs = pow2_scale(__reduce_max_sync(0xffffffffu, xm), 13);
        __syncthreads();                 // M and the exchanged parts are there

        // ---- y of the warp's 32 tokens and 16 channels
        {
            float u[2][2][4];            // the chunk's own tokens
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int p = 0; p < 2; ++p) u[i][p][0] = u[i][p][1] = u[i][p][2] = u[i][p][3] = 0.0f;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                if (ks > 2 * hv + 1 || ks >= nb) break;
                uint32_t xb[4];
                frag_bt<128>(s_x, 16 * ks, 16 * pw, lane, xb);
#pragma unroll
                for (int q = 0; q < 4; ++q) xb[q] = bf16x2_to_f16x2(xb[q], xs.x);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (ks > 2 * hv + i || 2 * hv + i >= nb) continue;
                    uint32_t ma[4];
                    frag_a<128>(s_m, 32 * hv + 16 * i, 16 * ks, lane, ma);
                    mma_h(u[i][0], ma, xb[0], xb[1]);
                    mma_h(u[i][1], ma, xb[2], xb[3]);
                }
            }
            const float beta = __fmul_rn(__fmul_rn(tsc.x, tsc.y), __fmul_rn(d.kd, xs.y));
            const uint32_t ex = s_ex + (uint32_t)((pw * 2 + hv) * 2048 + lane * 16);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (2 * hv + i >= nb) break;
                uint32_t out[2][2];      // [row half][channel tile]
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const uint4 e4 = ptx::lds128(ex + (uint32_t)((i * 2 + p) * 512));
                    const float part[4] = {__uint_as_float(e4.x), __uint_as_float(e4.y), __uint_as_float(e4.z), __uint_as_float(e4.w)};
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const int t = 32 * hv + 16 * i + 8 * hf + (lane >> 2);
                        uint32_t xv;
                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(xv) : "r"(tile128(s_x, t, 2 * pw + p) + 4 * (lane & 3)));
                        float v[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float own = hv ? y[2 + i][p][2 * hf + e] : y[i][p][2 * hf + e];
                            // the two halves of the states in one order for both warps
                            const float in = hv ? __fadd_rn(part[2 * hf + e], own) : __fadd_rn(own, part[2 * hf + e]);
                            v[e] = __fmaf_rn(u[i][p][2 * hf + e], beta, in);
                        }
                        out[hf][p] = bf16x2_of(make_float2(__fmaf_rn(skip, bf16_lo(xv), v[0]), __fmaf_rn(skip, bf16_hi(xv), v[1])));
                    }
                }
                // a quad holds 16 channels of a row in pairs; lane q of it gathers channels 4 q .. 4 q + 3
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int from = (lane & ~3) | (2 * (lane & 1));
                    const uint32_t a0 = __shfl_sync(0xffffffffu, out[hf][0], from), a1 = __shfl_sync(0xffffffffu, out[hf][0], from + 1);
                    const uint32_t b0 = __shfl_sync(0xffffffffu, out[hf][1], from), b1 = __shfl_sync(0xffffffffu, out[hf][1], from + 1);
                    const int t = 32 * hv + 16 * i + 8 * hf + (lane >> 2);
                    if (t < n)
                        *reinterpret_cast<uint2*>(o.y + (int64_t)(t0 + t) * o.ldy + h * kP + 16 * pw + 4 * (lane & 3)) =
                            lane & 2 ? make_uint2(b0, b1) : make_uint2(a0, a1);
                }
            }
        }
        // ---- the state at the chunk's end: w x as two fp16 parts
        {
            float D[8][4];
#pragma unroll
            for (int j = 0; j < 8; ++j) D[j][0] = D[j][1] = D[j][2] = D[j][3] = 0.0f;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                if (ks >= nb) break;
                float2 w0 = *reinterpret_cast<const float2*>(d.wl + 16 * ks + 2 * (lane & 3));
                float2 w1 = *reinterpret_cast<const float2*>(d.wl + 16 * ks + 8 + 2 * (lane & 3));
                w0 = make_float2(__fmul_rn(w0.x, xs.x), __fmul_rn(w0.y, xs.x));
                w1 = make_float2(__fmul_rn(w1.x, xs.x), __fmul_rn(w1.y, xs.x));
                uint32_t xa[4], hi[4], lo[4];
                frag_at<128>(s_x, 16 * ks, 16 * pw, lane, xa);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float2 ww = q < 2 ? w0 : w1;
                    split_f16x2(__fmul_rn(bf16_lo(xa[q]), ww.x), __fmul_rn(bf16_hi(xa[q]), ww.y), hi[q], lo[q]);
                }
                uint32_t bb[4][4];
#pragma unroll
                for (int q = 0; q < 4; ++q) frag_bt<256>(s_b, 16 * ks, 64 * hv + 16 * q, lane, bb[q]);
#pragma unroll
                for (int q = 0; q < 8; ++q) mma_h(D[q], lo, bb[q >> 1][2 * (q & 1)], bb[q >> 1][2 * (q & 1) + 1]);
#pragma unroll
                for (int q = 0; q < 8; ++q) mma_h(D[q], hi, bb[q >> 1][2 * (q & 1)], bb[q >> 1][2 * (q & 1) + 1]);
            }
            const float keep = d.done[kQ - 1], back = __fmul_rn(__fmul_rn(tsc.y, d.kd), xs.y);
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) S[j][q] = __fmaf_rn(D[j][q], back, __fmul_rn(S[j][q], keep));
        }
    };
    for (int k = 0; k < n_ch; ++k) {
        const int left = it.len - k * kQ;
        if (left <= 16) chunk(k, std::integral_constant<int, 1>{});
        else if (left <= 32) chunk(k, std::integral_constant<int, 2>{});
        else chunk(k, std::integral_constant<int, 4>{});
    }
    ptx::cp_async_wait<0>();
    if (o.final_state) {
        float* dst = o.final_state + sh + s_at;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            *reinterpret_cast<float2*>(dst + 8 * j) = make_float2(S[j][0], S[j][1]);
            *reinterpret_cast<float2*>(dst + 8 * kN + 8 * j) = make_float2(S[j][2], S[j][3]);
        }
    }
}

}  // namespace

// ------------------------------------------------------------------------------- segments

// Starts of the segments of cut sequences, from the segments' own contributions, in place.
// CTA (sequence, head), y: 0 forward in time, 1 backward (from the last segment to the first).
__global__ void __launch_bounds__(256) scan_carry_kernel(const Args a, const float* __restrict__ init,
                                                         const float* __restrict__ dfinal) {
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    const int h = blockIdx.x % a.nheads, s = blockIdx.x / a.nheads, rev = blockIdx.y;
    const int i0 = a.seq_slots[s].x, i1 = i0 + a.seq_slots[s].y;
    if (i1 - i0 < 2) return;
    const float* start = rev ? dfinal : init;
    float4 v[8];
    const float4* src = reinterpret_cast<const float4*>(start + ((int64_t)s * a.nheads + h) * kStateElems);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = start ? src[threadIdx.x + 256 * k] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i = i0; i < i1; ++i) {
        const int64_t at = ((int64_t)rev * a.cap_slots + (rev ? i0 + i1 - 1 - i : i)) * a.nheads + h;
        float4* p = reinterpret_cast<float4*>(a.seg_state + at * kStateElems);
        const bool more = i + 1 < i1;
        const float keep = more ? a.seg_decay[at] : 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float4 own = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (more) own = p[threadIdx.x + 256 * k];
            p[threadIdx.x + 256 * k] = v[k];
            v[k] = make_float4(__fmaf_rn(keep, v[k].x, own.x), __fmaf_rn(keep, v[k].y, own.y),
                               __fmaf_rn(keep, v[k].z, own.z), __fmaf_rn(keep, v[k].w, own.w));
        }
    }
}

// The state alone through an item: blockIdx.y 0 forward in time (u = x, v = B), 1 backward (u = dy, v = C: the
// state's gradient). STORE: from its start, at every chunk to the workspace, with the scales of the gradient kernel;
// otherwise from zero, the item's own contribution and decay, for what starts behind it. Eight warps; warp (pw, hv) holds the channels
// 16 pw .. and the states 64 hv .. in fp32 accumulators. v comes in fp16 (scan_tiles_kernel), the weighted u enters
// as two fp16 parts under a power-of-two scale of the warp's channels (2^-23 of each, down to 2^-38 of the largest).
// Bound by a chunk's chain of steps between two barriers and their instructions (half of the issue slots) with two
// CTAs per SM, 4 us for a chunk of each: 4 x 2,048 tokens, 64 heads, both directions 250 us, 2.5 TB/s.
struct StateDecay {
    float wt[kQ];        // the weights of u, the largest in [1/2, 1)
    float keep;          // exp(cum_64)
    float cum;           // cum_64
    float kd;            // 2^-k of the weights
    float pad;
};
constexpr int kStTile = 16384 + 8192;                                    // v, u
constexpr int kStateSmem = 2 * kStTile + 8 * 2048 + 16 * (int)sizeof(StateDecay) + 128;

template <bool STORE>
__global__ void __launch_bounds__(256, 2) scan_state_kernel(const Args a, const StateArgs o) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ Decay scratch_of[8];
    __shared__ uint32_t s_max[2][8], u_max[2][8];    // the warps' largest |S| and |u|
    ptx::pdl_launch_dependents();
    const uint32_t base = (ptx::smem_u32(smem_raw) + 127u) & ~127u;
    uint8_t* smem = smem_raw + (base - ptx::smem_u32(smem_raw));
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, pw = w & 3, hv = w >> 2;
    const uint32_t stage = base + 2 * kStTile + 2048 * w;
    StateDecay* dec = reinterpret_cast<StateDecay*>(smem + 2 * kStTile + 8 * 2048);
    const bool rev = blockIdx.y != 0;
    const int ngroups = a.nheads / a.per_group;
    const int h = blockIdx.x % a.nheads, g = h / a.per_group;
    Item it;
    if (!get_item(a, blockIdx.x / a.nheads, it) || it.len < 0) return;
    if (!STORE && (!(it.flags & kCut) || (it.flags & (rev ? kFirst : kLast)))) return;     // nothing starts behind it
    const int n_ch = (it.len + kQ - 1) / kQ;
    const uint16_t* u = (rev ? o.dy : a.x) + (int64_t)h * kP;
    const int64_t ldu = rev ? o.lddy : a.ldx;
    auto chunk_of = [&](int k) { return rev ? n_ch - 1 - k : k; };
    // a chunk's tile and scale; the forward pass's table has chunks of 128 tokens
    auto tile_at = [&](int q) { return (int64_t)(it.chunk0 + (a.chunk == kQ ? q : q >> 1)) * ngroups + g; };
    auto fetch = [&](int k) {
        if (k < n_ch) {
            const int q = chunk_of(k), t0 = it.t0 + q * kQ, n = min(kQ, it.len - q * kQ);
            const uint32_t st = base + (k & 1) * kStTile;
            const uint16_t* tl = a.tiles + (tile_at(q) * 2 + (rev ? 0 : 1)) * (128 * kN) + (a.chunk == kQ ? 0 : (q & 1) * kQ * kN);
            load_tile<128, 256>(st, tl, kN, 0, kQ, tid);
            load_tile<64, 256>(st + 16384, u, ldu, t0, n, tid);
        }
        ptx::cp_async_commit();
    };
    fetch(0);
    const float bias = a.dt_bias[h], a2 = __fmul_rn(-expf(a.a_log[h]), kLog2e);
    float S[8][4];
    const int s_at = (16 * pw + (lane >> 2)) * kN + 64 * hv + 2 * (lane & 3);
    const int64_t sh = ((int64_t)it.seq * a.nheads + h) * kStateElems;
    const int64_t slot = ((int64_t)(rev ? a.cap_slots : 0) + it.slot) * a.nheads + h;
    {
        const float* start = rev ? o.dfinal : a.init;
        const float* src = !STORE ? nullptr : it.flags & kCut ? a.seg_state + slot * kStateElems : start ? start + sh : nullptr;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float2 lo = make_float2(0.0f, 0.0f), hi = lo;
            if (src) {
                lo = *reinterpret_cast<const float2*>(src + s_at + 8 * j);
                hi = *reinterpret_cast<const float2*>(src + s_at + 8 * kN + 8 * j);
            }
            S[j][0] = lo.x; S[j][1] = lo.y; S[j][2] = hi.x; S[j][3] = hi.y;
        }
    }
    // the decays of eight chunks at a time, one per warp, in a ring of sixteen (one warp doing each chunk's in turn kept
    // the others waiting at every chunk's barrier)
    float total = 0.0f, raw0 = 0.0f, raw1 = 0.0f;
    auto raws = [&](int k) {
        if (k >= n_ch) return;
        const int q = chunk_of(k), t0 = it.t0 + q * kQ, n = min(kQ, it.len - q * kQ);
        raw0 = raw_dt(a, t0, n, h, 2 * lane);
        raw1 = raw_dt(a, t0, n, h, 2 * lane + 1);
    };
    auto decay = [&](int k) {
        if (k >= n_ch) return;
        StateDecay& d = dec[k & 15];
        Decay& scratch = scratch_of[w];
        chunk_decay(scratch, raw0, raw1, min(kQ, it.len - chunk_of(k) * kQ), bias, a2, lane);
        __syncwarp();
        float2 wt = reinterpret_cast<const float2*>(rev ? scratch.done : scratch.left)[lane];
        if (!rev) {
            const float2 dt = reinterpret_cast<const float2*>(scratch.dt)[lane];
            wt = make_float2(__fmul_rn(wt.x, dt.x), __fmul_rn(wt.y, dt.y));
        }
        // the largest weight to [1/2, 1): what a fast decay leaves keeps its bits
        const float2 sc = pow2_scale(__reduce_max_sync(0xffffffffu, max(__float_as_uint(wt.x), __float_as_uint(wt.y))), -1);
        wt = make_float2(__fmul_rn(wt.x, sc.x), __fmul_rn(wt.y, sc.x));
        reinterpret_cast<float2*>(d.wt)[lane] = wt;
        if (lane == 0) {
            d.keep = scratch.done[kQ - 1];
            d.cum = scratch.cum[kQ - 1];
            d.kd = sc.y;
        }
    };
    raws(w);
    decay(w);
    auto largest = [&](int k) {                 // of S, for the chunk k behind it
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) m = fmaxf(m, fabsf(S[j][q]));
        const uint32_t mb = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
        if (lane == 0) s_max[k & 1][w] = mb;
    };
    auto all_max = [](const uint32_t* m) { return max(max(max(m[0], m[1]), max(m[2], m[3])), max(max(m[4], m[5]), max(m[6], m[7]))); };
    // the scales of the gradient kernel: its chunk of u (once all warps have seen it) and the state
    auto scale_of = [&](int k) { return o.scale + ((int64_t)(it.chunk0 + chunk_of(k)) * a.nheads + h) * 4 + (rev ? 1 : 0); };
    if (STORE) largest(0);
    for (int k = 0; k < n_ch; ++k) {
        const uint32_t s_v = base + (k & 1) * kStTile, s_u = s_v + 16384;
        const StateDecay& d = dec[k & 15];
        ptx::cp_async_wait<0>();
        __syncthreads();
        fetch(k + 1);
        if ((k & 7) == 2) raws((k & ~7) + 8 + w);
        if ((k & 7) == 4) decay((k & ~7) + 8 + w);
        const float2 tsc = a.tile_scale[tile_at(chunk_of(k))];
        if (STORE) {
            // the warp's 16 rows x 64 states as fp16 high and low parts (2^-23 of each value) under a power-of-two scale of
            // the whole state, staged so that whole 128-byte rows go out
            const float2 ss = pow2_scale(all_max(s_max[k & 1]), 13);
            if (tid == 0) {
                scale_of(k)[2] = ss.y;
                if (k > 0) scale_of(k - 1)[0] = pow2_scale(all_max(u_max[(k - 1) & 1]), 13).y;
            }
            uint16_t* dst = (rev ? o.dstates : o.states) +
                            ((int64_t)(it.chunk0 + chunk_of(k)) * a.nheads + h) * 2 * kStateElems + 16 * pw * kN + 64 * hv;
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    uint32_t q[4], lo;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        split_f16x2(__fmul_rn(S[j + (i >> 1)][2 * (i & 1)], ss.x), __fmul_rn(S[j + (i >> 1)][2 * (i & 1) + 1], ss.x), q[i], lo);
                        if (part) q[i] = lo;
                    }
                    const int mi = lane >> 3;    // rows 0..7 and 8..15 of tile j, then of tile j + 1
                    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};"
                                 ::"r"(tile128(stage, 8 * (mi & 1) + (lane & 7), j + (mi >> 1))), "r"(q[0]), "r"(q[1]),
                                 "r"(q[2]), "r"(q[3]) : "memory");
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 4 * i + (lane >> 3), pc = lane & 7;
                    *reinterpret_cast<uint4*>(dst + part * kStateElems + row * kN + 8 * pc) = ptx::lds128(tile128(stage, row, pc));
                }
            }
        }
        uint32_t um = 0u;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            uint32_t ua[4];
            frag_at<128>(s_u, 16 * ks, 16 * pw, lane, ua);
#pragma unroll
            for (int q = 0; q < 4; ++q) um = abs_max_bf16x2(um, ua[q]);
        }
        um = __reduce_max_sync(0xffffffffu, um);
        const float2 us = pow2_scale(um, 13);
        if (STORE && lane == 0) u_max[k & 1][w] = um;
        float D[8][4];
#pragma unroll
        for (int j = 0; j < 8; ++j) D[j][0] = D[j][1] = D[j][2] = D[j][3] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            float2 w0 = *reinterpret_cast<const float2*>(d.wt + 16 * ks + 2 * (lane & 3));
            float2 w1 = *reinterpret_cast<const float2*>(d.wt + 16 * ks + 8 + 2 * (lane & 3));
            w0 = make_float2(__fmul_rn(w0.x, us.x), __fmul_rn(w0.y, us.x));
            w1 = make_float2(__fmul_rn(w1.x, us.x), __fmul_rn(w1.y, us.x));
            uint32_t ua[4], hi[4], lo[4];
            frag_at<128>(s_u, 16 * ks, 16 * pw, lane, ua);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 ww = q < 2 ? w0 : w1;
                split_f16x2(__fmul_rn(bf16_lo(ua[q]), ww.x), __fmul_rn(bf16_hi(ua[q]), ww.y), hi[q], lo[q]);
            }
            uint32_t bb[4][4];
#pragma unroll
            for (int q = 0; q < 4; ++q) frag_bt<256>(s_v, 16 * ks, 64 * hv + 16 * q, lane, bb[q]);
#pragma unroll
            for (int q = 0; q < 8; ++q) mma_h(D[q], lo, bb[q >> 1][2 * (q & 1)], bb[q >> 1][2 * (q & 1) + 1]);
#pragma unroll
            for (int q = 0; q < 8; ++q) mma_h(D[q], hi, bb[q >> 1][2 * (q & 1)], bb[q >> 1][2 * (q & 1) + 1]);
        }
        total = __fadd_rn(total, d.cum);
        const float keep = d.keep, back = __fmul_rn(__fmul_rn(rev ? tsc.x : tsc.y, d.kd), us.y);
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) S[j][q] = __fmaf_rn(D[j][q], back, __fmul_rn(S[j][q], keep));
        if (STORE) largest(k + 1);
    }
    ptx::cp_async_wait<0>();
    if (STORE && n_ch > 0) {
        __syncthreads();
        if (tid == 0) scale_of(n_ch - 1)[0] = pow2_scale(all_max(u_max[(n_ch - 1) & 1]), 13).y;
    }
    float* dst = !STORE ? a.seg_state + slot * kStateElems : rev && o.dinit && (it.flags & kFirst) ? o.dinit + sh : nullptr;
    if (dst) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            *reinterpret_cast<float2*>(dst + s_at + 8 * j) = make_float2(S[j][0], S[j][1]);
            *reinterpret_cast<float2*>(dst + s_at + 8 * kN + 8 * j) = make_float2(S[j][2], S[j][3]);
        }
    }
    if (!STORE && tid == 0) a.seg_decay[slot] = exp2f(total);
}

// ------------------------------------------------------------------------------- host

// Forward calls whose sequences have at most kDirectMean tokens on average take the warp-MMA kernel in one launch, where
// even one sequence holding all the tokens is not long (kDirectTokens), or not long beside the work there is. Measured,
// sequences x tokens, 64 heads from states, calls back to back from a graph, one launch against tensor cores behind table
// and tiles (us): 1 x 1 5.5 / 16, 1 x 128 14 / 17, 1 x 256 25 / 20, 1 x 512 46 / 27, 2 x 256 25 / 20, 4 x 128 21 / 27, 4 x 256
// 36 / 32, 9 x 112 39 / 45, 16 x 64 41 / 73, 128 x 8 193 / 485, 128 x 31 244 / 526. The lengths are on the device, so the
// rule sees their mean: a long sequence beside short ones pays for what the usual calls of that mean gain, 1,000 tokens beside 8
// single ones 91 / 55, 700 beside 7 of 40 67 / 50, 500 beside 3 single ones 47 / 33 (3,900 beside 127 single ones: 398 / 574, in
// the last place 551 / 582).
constexpr int kDirectMean = 128;
constexpr int kDirectTokens = 1024;

Plan make_plan(int nheads, int ngroups, int total, int nseq, bool backward) {
    Plan p{};
    // A segment is a CTA's fair share of 148 CTAs (backward: 296, for two directions), 512 tokens at least. A sequence
    // is cut where that saves time: what is left of it after the first segment takes 34 ns a token, the cut
    // 16 ns a token of a segment (the states of all segments but one, beforehand) and about 20 us of launches.
    // Measured, uncut / cut, forward: 1 x 2,048 tokens, 64 heads 72 / 81 us, 1 x 1,500 54 / 62; 8 heads 72 / 49.
    int64_t share = ((int64_t)total * nheads + 147) / 148;
    if (share < 512) share = 512;
    p.seg_len = (int)((share + 127) / 128 * 128);
    if (p.seg_len > (total + 127) / 128 * 128) p.seg_len = (total + 127) / 128 * 128;
    p.cut_at = p.seg_len + p.seg_len / 4 * 3 + 640;
    // short calls save the launches of the table and of the tiles: every sequence is one item, in the order given
    p.direct = !backward && total <= (int64_t)kDirectMean * nseq &&
               (total <= kDirectTokens || total <= (int64_t)nseq * nheads / 2);
    p.chunk = backward ? kQ : 128;
    p.cap_items = total / p.seg_len + nseq;
    p.cap_chunks = total / p.chunk + nseq;
    p.cap_slots = 2 * (total / p.seg_len) + 1;             // a cut sequence of n tokens has at most 2 n / seg_len segments
    size_t o = 256;                                        // error word
    p.count = o;       o += 256;
    p.items = o;       o = up256(o + sizeof(Item) * (size_t)p.cap_items);
    p.seq_items = o;   o = up256(o + sizeof(Item) * (size_t)p.cap_items);
    p.seq_slots = o;   o = up256(o + sizeof(int2) * (size_t)nseq);
    p.chunks = o;      o = up256(o + sizeof(Chunk) * (size_t)p.cap_chunks);
    const size_t tiles = p.direct ? 0 : (size_t)p.cap_chunks * ngroups;
    p.tiles = o;       o = up256(o + tiles * 2 * 128 * kN * 2);
    p.tile_scale = o;  o = up256(o + tiles * sizeof(float2));
    const size_t slots = (backward ? 2 : 1) * (size_t)p.cap_slots * nheads;
    p.seg_decay = o;   o = up256(o + 4 * slots);
    p.seg_state = o;
    if (total > p.cut_at) o = up256(o + 4 * slots * kStateElems);
    p.total = o;
    return p;
}

Args make_args(const dfssm_scan_dims* dims, const dfssm_scan_inputs* in, int total, int nseq, const Plan& p, uint8_t* ws) {
    Args a{};
    a.x = static_cast<const uint16_t*>(in->x);
    a.b = static_cast<const uint16_t*>(in->b);
    a.c = static_cast<const uint16_t*>(in->c);
    a.dt = static_cast<const uint16_t*>(in->dt);
    a.ldx = in->x_stride;
    a.ldb = in->b_stride;
    a.ldc = in->c_stride;
    a.lddt = in->dt_stride;
    a.dt_bias = in->dt_bias;
    a.a_log = in->a_log;
    a.d_skip = in->d_skip;
    a.init = in->init_state;
    a.cu = in->cu_seqlens;
    a.nheads = dims->nheads;
    a.per_group = dims->nheads / dims->ngroups;
    a.total = total;
    a.nseq = nseq;
    a.seg_len = p.seg_len;
    a.cut_at = p.cut_at;
    a.direct = p.direct;
    a.chunk = p.chunk;
    a.cap_items = p.cap_items;
    a.cap_chunks = p.cap_chunks;
    a.cap_slots = p.cap_slots;
    a.err = reinterpret_cast<uint32_t*>(ws);
    a.count = reinterpret_cast<int32_t*>(ws + p.count);
    a.items = reinterpret_cast<Item*>(ws + p.items);
    a.seq_items = reinterpret_cast<Item*>(ws + p.seq_items);
    a.seq_slots = reinterpret_cast<int2*>(ws + p.seq_slots);
    a.chunks = reinterpret_cast<Chunk*>(ws + p.chunks);
    a.tiles = reinterpret_cast<uint16_t*>(ws + p.tiles);
    a.tile_scale = reinterpret_cast<float2*>(ws + p.tile_scale);
    a.seg_state = reinterpret_cast<float*>(ws + p.seg_state);
    a.seg_decay = reinterpret_cast<float*>(ws + p.seg_decay);
    return a;
}

dfssm_status check_dims(const dfssm_scan_dims* d, int total, int nseq) {
    if (!d) return DFSSM_ERR_INVALID_ARG;
    if (d->headdim != kP || d->d_state != kN) return DFSSM_ERR_UNSUPPORTED_SHAPE;
    if (d->nheads < 1 || d->nheads > 1024 || d->ngroups < 1 || d->nheads % d->ngroups != 0)
        return DFSSM_ERR_UNSUPPORTED_SHAPE;
    if (total < 1 || total > (1 << 22) || nseq < 1 || nseq > 65536) return DFSSM_ERR_UNSUPPORTED_SHAPE;
    // rows of the tiles of B and C, which the tensor map counts in 32 bits
    if (((int64_t)total / 128 + nseq) * d->ngroups * 256 > INT32_MAX) return DFSSM_ERR_UNSUPPORTED_SHAPE;
    return DFSSM_OK;
}

dfssm_status check_call(const dfssm_scan_dims* d, const dfssm_scan_inputs* in, int total, int nseq) {
    const dfssm_status st = check_dims(d, total, nseq);
    if (st != DFSSM_OK) return st;
    if (!in) return DFSSM_ERR_INVALID_ARG;
    const int64_t di = (int64_t)d->nheads * kP, gn = (int64_t)d->ngroups * kN, most = (int64_t)1 << 30;
    const void* rows[3] = {in->x, in->b, in->c};
    const int64_t ld[3] = {in->x_stride, in->b_stride, in->c_stride}, least[3] = {di, gn, gn};
    for (int i = 0; i < 3; ++i)
        if (!rows[i] || !al16(rows[i]) || ld[i] < least[i] || ld[i] % 8 != 0 || ld[i] > most) return DFSSM_ERR_INVALID_ARG;
    if (!in->dt || (reinterpret_cast<uintptr_t>(in->dt) & 1u) || in->dt_stride < d->nheads || in->dt_stride > most)
        return DFSSM_ERR_INVALID_ARG;
    const void* words[4] = {in->dt_bias, in->a_log, in->d_skip, in->cu_seqlens};
    for (const void* p : words)
        if (!p || (reinterpret_cast<uintptr_t>(p) & 3u)) return DFSSM_ERR_INVALID_ARG;
    if (!al16(in->init_state)) return DFSSM_ERR_INVALID_ARG;
    return DFSSM_OK;
}

namespace {
bool g_ready[64];
std::mutex g_mu;
}  // namespace

dfssm_status setup() {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DFSSM_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_mu);
    if (!g_ready[dev]) {
        const cudaFuncAttribute at = cudaFuncAttributeMaxDynamicSharedMemorySize;
        if (cudaFuncSetAttribute(scan_fwd_kernel, at, kFwdSmem) != cudaSuccess || setup_tc() != cudaSuccess ||
            cudaFuncSetAttribute(scan_state_kernel<false>, at, kStateSmem) != cudaSuccess ||
            cudaFuncSetAttribute(scan_state_kernel<true>, at, kStateSmem) != cudaSuccess ||
            setup_bwd() != cudaSuccess)
            return DFSSM_ERR_CUDA;
        g_ready[dev] = true;
    }
    return DFSSM_OK;
}

cudaError_t launch_table(const Args& a, cudaStream_t s) {
    scan_table_kernel<<<1, kTableThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_after(scan_tiles_kernel, 2 * a.cap_chunks * (a.nheads / a.per_group), 512, 0, s, a);
}

cudaError_t launch_segment_starts(const Args& a, const StateArgs& o, int directions, cudaStream_t s) {
    if (a.total <= a.cut_at) return cudaSuccess;           // no sequence can be cut
    // not launch_after: CTAs that come in beside the tiles' are packed two to an SM where one to an SM would do
    // (16,384 tokens, 64 heads: 477 us, with it 597)
    scan_state_kernel<false><<<dim3(a.cap_items * a.nheads, directions), 256, kStateSmem, s>>>(a, o);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_after(scan_carry_kernel, dim3(a.nseq * a.nheads, directions), 256, 0, s, a, a.init, o.dfinal);
}

cudaError_t launch_states(const Args& a, const StateArgs& o, cudaStream_t s) {
    const cudaError_t e = launch_segment_starts(a, o, 2, s);
    if (e != cudaSuccess) return e;
    scan_state_kernel<true><<<dim3(a.cap_items * a.nheads, 2), 256, kStateSmem, s>>>(a, o);
    return cudaGetLastError();
}

}  // namespace scan
}  // namespace dfssm

using namespace dfssm;
using namespace dfssm::scan;

extern "C" dfssm_status dfssm_ssm_scan_workspace_bytes(const dfssm_scan_dims* dims, int32_t total, int32_t nseq,
                                                       int32_t backward, size_t* bytes) {
    const dfssm_status st = check_dims(dims, total, nseq);
    if (st != DFSSM_OK) return st;
    if (!bytes) return DFSSM_ERR_INVALID_ARG;
    *bytes = backward ? bwd_workspace(dims, total, nseq) : make_plan(dims->nheads, dims->ngroups, total, nseq, false).total;
    return DFSSM_OK;
}

extern "C" dfssm_status dfssm_ssm_scan_fwd(const dfssm_scan_dims* dims, const dfssm_scan_inputs* in, int32_t total,
                                           int32_t nseq, void* y, int64_t y_stride, float* final_state, void* workspace,
                                           size_t workspace_bytes, void* stream) {
    dfssm_status st = check_call(dims, in, total, nseq);
    if (st != DFSSM_OK) return st;
    if (!y || !al16(y) || y_stride < (int64_t)dims->nheads * kP || y_stride % 8 != 0 || y_stride > ((int64_t)1 << 30) ||
        !al16(final_state))
        return DFSSM_ERR_INVALID_ARG;
    const Plan p = make_plan(dims->nheads, dims->ngroups, total, nseq, false);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < p.total)
        return DFSSM_ERR_INVALID_ARG;
    if ((st = setup()) != DFSSM_OK) return st;
    const Args a = make_args(dims, in, total, nseq, p, static_cast<uint8_t*>(workspace));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a.direct) {
        const FwdOut o{static_cast<uint16_t*>(y), y_stride, final_state};
        scan_fwd_kernel<<<nseq * a.nheads, kFwdThreads, kFwdSmem, s>>>(a, o);
    } else {
        if (launch_table(a, s) != cudaSuccess || launch_segment_starts(a, StateArgs{}, 1, s) != cudaSuccess)
            return DFSSM_ERR_CUDA;
        if (launch_tc(a, static_cast<uint16_t*>(y), y_stride, final_state, s) != cudaSuccess) return DFSSM_ERR_CUDA;
    }
    return cudaGetLastError() == cudaSuccess ? DFSSM_OK : DFSSM_ERR_CUDA;
}
