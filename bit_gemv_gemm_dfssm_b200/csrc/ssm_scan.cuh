// Shared parts of the state scan over packed sequences (ssm_scan.cu, ssm_scan_tc.cu, ssm_scan_bwd.cu): the work
// table, the decays of a chunk, shared-memory tiles and warp-MMA fragments.
//
// The recurrence of one head h (64 channels p, 128 states n; B and C shared by a group of heads):
//   dt_t = softplus(dt_raw + dt_bias) (the argument itself above 20), a_t = -exp(a_log) dt_t
//   S_t  = exp(a_t) S_{t-1} + dt_t x_t B_t^T,      y_t = S_t C_t + d_skip x_t
// is worked on in chunks of 64 tokens, 128 in ssm_scan_tc.cu (cum_t = a_1 + ... + a_t inside the chunk):
//   y_t   = sum_{s <= t} (C_t . B_s) exp(cum_t - cum_s) dt_s x_s + exp(cum_t) S_0 C_t + d_skip x_t
//   S_end = exp(cum_64) S_0 + sum_s exp(cum_64 - cum_s) dt_s x_s B_s^T
// All exponents are <= 0. Decays are kept in units of log 2.
#pragma once

#include <cstdint>

#include <cuda_fp16.h>

#include "dfssm_internal.cuh"
#include "epilogue.cuh"
#include "ptx.cuh"

namespace dfssm {
namespace scan {

constexpr int kP = 64;           // channels per head
constexpr int kN = 128;          // states per channel
constexpr int kQ = 64;           // tokens per chunk
constexpr int kStateElems = kP * kN;
constexpr float kLog2e = 1.4426950408889634f;

// One run of tokens that a CTA takes through the recurrence: a sequence, or a segment of one.
struct Item {
    int32_t seq;
    int32_t t0;        // first token row
    int32_t len;       // tokens (0: an empty sequence)
    int32_t chunk0;    // index of its first chunk
    int32_t slot;      // cut sequences: its place among the segments of all of them
    int32_t flags;
};
enum { kFirst = 1, kLast = 2, kCut = 4 };   // first / last segment of its sequence; the sequence has several

struct Chunk {
    int32_t t0;
    int32_t n;         // 1 .. 64 (128) tokens
};

// What every kernel of a call gets.
struct Args {
    const uint16_t* x;
    const uint16_t* b;
    const uint16_t* c;
    const uint16_t* dt;
    int64_t ldx, ldb, ldc, lddt;       // row strides in elements
    const float* dt_bias;
    const float* a_log;
    const float* d_skip;
    const float* init;                 // [nseq][H][64][128] or NULL
    const int32_t* cu;
    int nheads, per_group;             // heads; heads per group
    int total, nseq;
    int seg_len;                       // tokens of a segment (a multiple of the chunk)
    int cut_at;                        // sequences longer than this are cut into segments
    int chunk;                         // tokens per chunk of the table: 64, or 128 for the tensor-core forward
    int direct;                        // 1: no table, item i is sequence i
    int cap_items, cap_chunks, cap_slots;
    uint32_t* err;
    int32_t* count;                    // [0] items, [1] chunks
    Item* items;                       // longest first
    Item* seq_items;                   // the same in sequence order
    int2* seq_slots;                   // [nseq] first slot and segments of a cut sequence (0 segments: not cut)
    Chunk* chunks;
    uint16_t* tiles;                   // [chunks][groups][C, B][128][128] fp16, scaled (scan_tiles_kernel)
    float2* tile_scale;                // [chunks][groups] 2^-k of C and of B
    float* seg_state;                  // [1 or 2][cap_slots][H][64][128]: what a cut sequence's segments start from
    float* seg_decay;                  // [1 or 2][cap_slots][H] (1: the gradient's, backward in time)
};

__device__ __forceinline__ bool get_item(const Args& a, int i, Item& it) {
    if (!a.direct) {
        if (i >= a.count[0]) return false;
        it = a.items[i];
        return true;
    }
    if (i >= a.nseq) return false;
    const int t0 = a.cu[i], t1 = a.cu[i + 1];
    if (t0 < 0 || t1 < t0 || t1 > a.total) {
        if (threadIdx.x == 0) atomicOr(a.err, DFSSM_DEVERR_SEQLENS);
        return false;
    }
    it = Item{i, t0, t1 - t0, 0, i, kFirst | kLast};
    return true;
}

// ---- shared-memory tiles: rows of 128 or 256 bytes, 16-byte pieces swizzled by the row, so that
// ldmatrix (8 rows, one piece each) hits 8 bank groups
__device__ __forceinline__ uint32_t tile128(uint32_t base, int row, int piece) {
    return base + (uint32_t)(row * 128 + 16 * (piece ^ (row & 7)));
}
__device__ __forceinline__ uint32_t tile256(uint32_t base, int row, int piece) {
    return base + (uint32_t)(row * 256 + 16 * (piece ^ (row & 7)));
}

// 64 rows x 64 (COLS = 64) or x 128 bf16 by cp.async; rows from n on are filled with zeros
template <int COLS, int THREADS>
__device__ __forceinline__ void load_tile(uint32_t dst, const uint16_t* src, int64_t ld, int t0, int n, int tid) {
    constexpr int kPieces = COLS / 8;
#pragma unroll
    for (int i = tid; i < kQ * kPieces; i += THREADS) {
        const int row = i / kPieces, pc = i % kPieces;
        const bool in = row < n;
        const uint16_t* p = src + (int64_t)(t0 + (in ? row : 0)) * ld + 8 * pc;
        ptx::cp_async16_zfill_s(COLS == 64 ? tile128(dst, row, pc) : tile256(dst, row, pc), p, in ? 16u : 0u);
    }
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t saddr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(saddr));
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t saddr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(saddr));
}

// D(16x8 fp32) += A(16x16 fp16) B(16x8 fp16)
__device__ __forceinline__ void mma_h(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The power of two 2^k that brings m (a largest magnitude, as bits) to [2^top, 2^(top + 1)), and 2^-k. k is kept
// within +-100 (a zero maximum: the largest). An infinity or NaN among the values gives NaN: scaled by it, the finite ones
// would go down to nothing unseen.
__device__ __forceinline__ float2 pow2_scale(uint32_t m_bits, int top) {
    if (m_bits >= 0x7F800000u) return make_float2(__int_as_float(0x7FC00000), __int_as_float(0x7FC00000));
    const int k = max(-100, min(100, top + 127 - (int)(m_bits >> 23)));
    return make_float2(__int_as_float((127 + k) << 23), __int_as_float((127 - k) << 23));
}

// the larger of m and the magnitudes of two bf16 values, as fp32 bits
__device__ __forceinline__ uint32_t abs_max_bf16x2(uint32_t m, uint32_t v) {
    return max(m, max((v << 16) & 0x7FFF0000u, v & 0x7FFF0000u));
}
__device__ __forceinline__ uint32_t f16x2_of(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t v, float scale) {
    return f16x2_of(__fmul_rn(bf16_lo(v), scale), __fmul_rn(bf16_hi(v), scale));
}
// (a, b) as two fp16 pairs whose sum is (a, b) to 2^-23 of each (or to 2^-25 below fp16's normal range)
__device__ __forceinline__ void split_f16x2(float a, float b, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __floats2half2_rn(a, b);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    const float2 f = __half22float2(h);
    lo = f16x2_of(__fsub_rn(a, f.x), __fsub_rn(b, f.y));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Fragments of a tile stored [row][col] (32-lane addresses; see the m16n8k16 register layout):
//  frag_a:  A operand rows x k, rows r0.., k from column k0       (tile rows = A rows)
//  frag_at: A operand from the transposed tile (tile rows = k)    rows = tile columns
//  frag_b:  B operand for two 8-wide n tiles, tile rows = n, columns = k   -> {b0,b1} of tile 0, tile 1
//  frag_bt: the same from the transposed tile (tile rows = k, columns = n)
template <int W>
__device__ __forceinline__ uint32_t tile_at(uint32_t base, int row, int piece) {
    return W == 128 ? tile128(base, row, piece) : tile256(base, row, piece);
}
template <int W>
__device__ __forceinline__ void frag_a(uint32_t base, int r0, int k0, int lane, uint32_t (&r)[4]) {
    const int mi = lane >> 3;
    ldmatrix_x4(tile_at<W>(base, r0 + 8 * (mi & 1) + (lane & 7), (k0 >> 3) + (mi >> 1)), r);
}
template <int W>
__device__ __forceinline__ void frag_at(uint32_t base, int k0, int c0, int lane, uint32_t (&r)[4]) {
    const int mi = lane >> 3;
    ldmatrix_x4_trans(tile_at<W>(base, k0 + 8 * (mi >> 1) + (lane & 7), (c0 >> 3) + (mi & 1)), r);
}
template <int W>
__device__ __forceinline__ void frag_b(uint32_t base, int n0, int k0, int lane, uint32_t (&r)[4]) {
    const int mi = lane >> 3;
    ldmatrix_x4(tile_at<W>(base, n0 + 8 * (mi >> 1) + (lane & 7), (k0 >> 3) + (mi & 1)), r);
}
template <int W>
__device__ __forceinline__ void frag_bt(uint32_t base, int k0, int n0, int lane, uint32_t (&r)[4]) {
    const int mi = lane >> 3;
    ldmatrix_x4_trans(tile_at<W>(base, k0 + 8 * (mi & 1) + (lane & 7), (n0 >> 3) + (mi >> 1)), r);
}

__device__ __forceinline__ float softplus_dt(float v) { return v > 20.0f ? v : log1pf(expf(v)); }
__device__ __forceinline__ float bf16f(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// Decays of a chunk for one head, in shared memory
struct Decay {
    float cum[kQ];      // a_1 + ... + a_t, log 2 units
    float dt[kQ];
    float left[kQ];     // exp(cum_64 - cum_t), from the sum a_{t+1} + ... + a_64
    float done[kQ];     // exp(cum_t)
};

// One warp: lane l takes tokens 2 l and 2 l + 1. raw0, raw1: dt_raw of the two (any value where t >= n).
__device__ __forceinline__ void chunk_decay(Decay& d, float raw0, float raw1, int n, float bias, float a2, int lane) {
    const float dt0 = 2 * lane < n ? softplus_dt(__fadd_rn(raw0, bias)) : 0.0f;
    const float dt1 = 2 * lane + 1 < n ? softplus_dt(__fadd_rn(raw1, bias)) : 0.0f;
    const float v0 = __fmul_rn(dt0, a2), v1 = __fmul_rn(dt1, a2);
    float up = __fadd_rn(v0, v1), down = up;        // inclusive sums over the lanes, from the left and from the right
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float u = __shfl_up_sync(0xffffffffu, up, o), w = __shfl_down_sync(0xffffffffu, down, o);
        if (lane >= o) up = __fadd_rn(up, u);
        if (lane + o < 32) down = __fadd_rn(down, w);
    }
    float before = __shfl_up_sync(0xffffffffu, up, 1), after = __shfl_down_sync(0xffffffffu, down, 1);
    if (lane == 0) before = 0.0f;
    if (lane == 31) after = 0.0f;
    const float c0 = __fadd_rn(before, v0);
    const float r0 = __fadd_rn(v1, after);
    reinterpret_cast<float2*>(d.cum)[lane] = make_float2(c0, up);
    reinterpret_cast<float2*>(d.dt)[lane] = make_float2(dt0, dt1);
    reinterpret_cast<float2*>(d.left)[lane] = make_float2(exp2f(r0), exp2f(after));
    reinterpret_cast<float2*>(d.done)[lane] = make_float2(exp2f(c0), exp2f(up));
}

__device__ __forceinline__ float raw_dt(const Args& a, int t0, int n, int h, int i) {
    return i < n ? bf16f(a.dt[(int64_t)(t0 + i) * a.lddt + h]) : 0.0f;
}

// ---- host side: the call's plan and workspace
struct Plan {
    int seg_len, cut_at, chunk, direct, cap_items, cap_chunks, cap_slots;
    size_t count, items, seq_items, seq_slots, chunks, tiles, tile_scale, seg_state, seg_decay, total;
};
Plan make_plan(int nheads, int ngroups, int total, int nseq, bool backward);
dfssm_status check_call(const dfssm_scan_dims* dims, const dfssm_scan_inputs* in, int total, int nseq);
dfssm_status setup();
Args make_args(const dfssm_scan_dims* dims, const dfssm_scan_inputs* in, int total, int nseq, const Plan& p, uint8_t* ws);
// the work table, and B and C in fp16
cudaError_t launch_table(const Args& a, cudaStream_t s);
struct StateArgs {
    const uint16_t* dy;
    int64_t lddy;
    const float* dfinal;       // [nseq][H][64][128] gradient of the final states, or NULL
    uint16_t* states;          // [chunks][H][2][64][128]: the state in front of every chunk
    uint16_t* dstates;         // the same: the gradient of the state behind it
    float* scale;              // [chunks][H][4] 2^-k of x, dy, the states, their gradients
    float* dinit;              // [nseq][H][64][128] gradient of the initial states, or NULL
};
// the start states of the segments of cut sequences (nothing to do when none can be cut); directions 2: of their
// gradients too
cudaError_t launch_segment_starts(const Args& a, const StateArgs& o, int directions, cudaStream_t s);
// the states and, backward in time, their gradients at every chunk
cudaError_t launch_states(const Args& a, const StateArgs& o, cudaStream_t s);
// the forward kernel of long calls (ssm_scan_tc.cu)
cudaError_t setup_tc();
cudaError_t launch_tc(const Args& a, uint16_t* y, int64_t ldy, float* final_state, cudaStream_t s);
cudaError_t setup_bwd();
size_t bwd_workspace(const dfssm_scan_dims* dims, int total, int nseq);

inline size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }
inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace scan
}  // namespace dfssm
