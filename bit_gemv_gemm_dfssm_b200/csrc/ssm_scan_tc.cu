// The scan's forward pass for long calls on the 5th-generation tensor cores (ssm_scan.cuh has the formulas, with chunks
// of 128 tokens here).
//
// A persistent-in-time CTA takes one head through one item, chunk by chunk. Per chunk four products, all fp16
// operands with fp32 accumulators in tensor memory:
//   G  = C B^T          128 x 128 x 128   both tiles as scan_tiles_kernel left them
//   Yi = C S^T          128 x  64 x 128   S (the state, scaled, one fp16 part) stored [state][channel]
//   Ya = M X            128 x  64 x 128   M = G exp(cum_t - cum_s) dt_s, causal, from tensor memory
//   D  = B^T (w X)      128 x  64 x 128   twice: w x as two fp16 parts
// and y = exp(cum_t) Yi + Ya + d_skip x, S = exp(cum_128) S + D. The state itself stays in fp32 registers; every
// scale is a power of two. B^T, X, S and w X are read along their rows (M- or N-major operands), so nothing is
// transposed.
//
// Roles (20 warps): TMA; MMA issue; decays (two warps in turn); and four groups of four warps, one thread per row:
//   M group: G from tensor memory -> M back into tensor memory;
//   X group: x -> fp16 in place, w x -> two tiles;
//   S group: thread n holds S[0..63][n]: S -> fp16 tile, then S = keep S + D;
//   Y group: Yi, Ya, x -> y in bf16 over the x tile, out as whole rows.
// They meet in mbarriers only, so that the products of one chunk run beside the conversions of the next. Every
// wait is bounded.
//
// Measured (8 sequences, 16,384 tokens, 64 heads): the call 269 us back to back from a graph, 4.5 us per chunk and SM, where the products take 20 % of the
// tensor pipe and 250 MB 12 % of the HBM's rate: the chain G -> M -> Ya -> y and S -> D -> S of one chunk, each step
// a hand-over between roles, bounds it. Chunks of 64 tokens on warp MMAs took 440 us; one role's loops unrolled
// further, or twice the warps per role, were slower (instruction fetches; 290 to 320 us).
#include <cstddef>

#include "ssm_scan.cuh"

namespace dfssm {
namespace scan {

namespace {

constexpr int kT = 128;                          // tokens per chunk
constexpr int kDec = 4;                          // chunks whose decays are kept
constexpr int kTcThreads = 20 * 32;
constexpr int kTile = 16384;                     // 128 rows of 128 bytes
constexpr int kStageTc = 5 * kTile;              // C (2 column blocks), B (2), X
constexpr int kCB = 4 * kTile;
struct alignas(16) TcDecay {
    float cum[kT];       // log 2 units
    float dts[kT];       // dt 2^kd
    float wl[kT];        // dts exp(cum_128 - cum_t)
    float done[kT];      // exp(cum_t)
    float kd, kc, kb;    // 2^-kd, 2^-k of C, of B
    float pad;
    float off[3][96];    // rows 32 (r + 1) .. of M: dts_s exp(cum_{32 (r + 1)} - cum_s) for the columns s in front
};
struct alignas(16) TcShared {
    TcDecay dec[kDec];
    float kx[kDec];      // 2^-k of the x tile; goes back with the decays
    float ks[2];         // of the state tile; goes back with Yi
    alignas(16) uint32_t red[2][2][4];  // [X, S group][chunk parity] maxima of the warps
    uint64_t cb_full[2], cb_empty[2], xt_full[2], xt_empty[2], g_full[2], g_empty[2];
    uint64_t dec_full[kDec], dec_empty[kDec];
    uint64_t m_full, m_empty, x_full, wx_empty, d_full, d_empty, s_full, s_empty, y_full, y_empty, drain;
    uint32_t tmem, abort;
};
constexpr int kTcSmem = 2 * kStageTc + 3 * kTile + (int)sizeof(TcShared) + 1024;
static_assert(kTcSmem <= 232448, "shared memory");
static_assert(offsetof(TcShared, red) % 16 == 0 && offsetof(TcDecay, off) % 16 == 0 && sizeof(TcDecay) % 16 == 0 &&
              offsetof(TcDecay, dts) % 16 == 0 && offsetof(TcShared, cb_full) % 8 == 0, "vector accesses");

// tensor memory columns
constexpr uint32_t kColG = 0, kColM = 256, kColYi = 320, kColYa = 384, kColD = 448;

struct TcArgs {
    Args a;
    uint16_t* y;
    int64_t ldy;
    float* final_state;
};

constexpr uint32_t kIdescBase = (1u << 4) | ((uint32_t)(128 >> 4) << 24);       // D fp32, A and B fp16, M 128
constexpr uint32_t kIdescG = kIdescBase | ((uint32_t)(128 >> 3) << 17);
constexpr uint32_t kIdescY = kIdescBase | ((uint32_t)(64 >> 3) << 17) | (1u << 16);               // B along N
constexpr uint32_t kIdescD = kIdescBase | ((uint32_t)(64 >> 3) << 17) | (1u << 16) | (1u << 15);  // A along M, B along N

__global__ void __launch_bounds__(kTcThreads, 1)
scan_tc_kernel(const __grid_constant__ CUtensorMap map_t, const __grid_constant__ CUtensorMap map_x, const TcArgs p) {
    extern __shared__ uint8_t smem_raw[];
    ptx::pdl_wait();                                 // the work table, the tiles, the segments' starts
    const Args& a = p.a;
    const int ngroups = a.nheads / a.per_group;
    const int h = blockIdx.x % a.nheads, g = h / a.per_group;
    Item it;
    if (!get_item(a, blockIdx.x / a.nheads, it) || it.len < 0) return;
    uint8_t* smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = ptx::smem_u32(smem);
    const uint32_t s_wx = base + 2 * kStageTc, s_st = s_wx + 2 * kTile;
    TcShared& sh = *reinterpret_cast<TcShared*>(smem + 2 * kStageTc + 3 * kTile);
    volatile uint32_t* abort_flag = &sh.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_ch = (it.len + kT - 1) / kT;

    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(&sh.cb_full[s], 1);
            ptx::mbar_init(&sh.cb_empty[s], 1);       // the MMAs
            ptx::mbar_init(&sh.xt_full[s], 1);
            ptx::mbar_init(&sh.xt_empty[s], 4);       // the Y warps (behind the MMAs)
            ptx::mbar_init(&sh.g_full[s], 1);
            ptx::mbar_init(&sh.g_empty[s], 4);
        }
        for (int s = 0; s < kDec; ++s) {
            ptx::mbar_init(&sh.dec_full[s], 1);
            ptx::mbar_init(&sh.dec_empty[s], 16);     // every warp of the groups
        }
        ptx::mbar_init(&sh.m_full, 4);
        ptx::mbar_init(&sh.m_empty, 1);
        ptx::mbar_init(&sh.x_full, 4);
        ptx::mbar_init(&sh.wx_empty, 1);
        ptx::mbar_init(&sh.d_full, 1);
        ptx::mbar_init(&sh.d_empty, 4);
        ptx::mbar_init(&sh.s_full, 4);
        ptx::mbar_init(&sh.s_empty, 1);
        ptx::mbar_init(&sh.y_full, 1);
        ptx::mbar_init(&sh.y_empty, 4);
        ptx::mbar_init(&sh.drain, 1);
        sh.abort = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(&sh.tmem, 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = sh.tmem;

    // a bounded wait; a role that gives up takes all others along
    auto wait1 = [&](uint64_t* bar, uint32_t parity) -> bool {
        if (ptx::mbar_wait(bar, parity) && !*abort_flag) return true;
        atomicOr(a.err, DFSSM_DEVERR_TIMEOUT);
        *abort_flag = 1;
        return false;
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {       // the whole warp, through lane 0
        bool ok = true;
        if (lane == 0) ok = wait1(bar, parity);
        return __shfl_sync(0xffffffffu, ok, 0) != 0;
    };
    auto arrive = [&](uint64_t* bar) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar);
    };
    const int row = 32 * (warp & 3) + lane;          // of the groups' threads
    const uint32_t t_lane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    auto piece = [](uint32_t tile, int r, int pc) { return tile + (uint32_t)(r * 128 + 16 * (pc ^ (r & 7))); };
    auto sts128 = [](uint32_t at, const uint32_t* v) {
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
    };

    if (warp == 0) {
        if (lane == 0) {
            int k = 0;
            for (; k < n_ch; ++k) {
                const int s = k & 1;
                const uint32_t ph = ((uint32_t)(k >> 1) & 1u) ^ 1u;
                uint8_t* st = smem + s * kStageTc;
                const int trow = ((it.chunk0 + k) * ngroups + g) * 2 * kT;
                if (!wait1(&sh.cb_empty[s], ph)) break;
                ptx::mbar_arrive_expect_tx(&sh.cb_full[s], kCB);
                ptx::tma_load_2d(st, &map_t, 0, trow, &sh.cb_full[s]);
                ptx::tma_load_2d(st + kTile, &map_t, 64, trow, &sh.cb_full[s]);
                ptx::tma_load_2d(st + 2 * kTile, &map_t, 0, trow + kT, &sh.cb_full[s]);
                ptx::tma_load_2d(st + 3 * kTile, &map_t, 64, trow + kT, &sh.cb_full[s]);
                const bool ok = wait1(&sh.xt_empty[s], ph);
                ptx::mbar_arrive_expect_tx(&sh.xt_full[s], kTile);
                ptx::tma_load_2d(st + kCB, &map_x, h * kP, it.t0 + k * kT, &sh.xt_full[s]);
                if (!ok) {
                    ++k;
                    break;
                }
            }
            if (*abort_flag)                           // the copies still in flight land before the CTA ends
                for (int i = max(0, k - 2); i < k; ++i) {
                    ptx::mbar_wait(&sh.cb_full[i & 1], (uint32_t)(i >> 1) & 1u);
                    ptx::mbar_wait(&sh.xt_full[i & 1], (uint32_t)(i >> 1) & 1u);
                }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // Each product is issued as soon as what it reads is there and what it writes is free, whichever comes
            // first; in a fixed order G of the next chunk held up the readouts until that chunk's tiles had come.
            int kg = 0, kd = 0, ki = 0, ka = 0;        // chunks whose G, D, Yi, Ya are issued
            int freed = 0;                             // chunks whose C and B tiles are released
            uint32_t idle = 0;
            uint64_t since = 0;
            bool ok = true;
            auto ready = [&](uint64_t* bar, int phases) { return ptx::mbar_test(bar, (uint32_t)phases & 1u); };
            while (ok && (kg < n_ch || kd < n_ch || ki < n_ch || ka < n_ch)) {
                bool moved = false;
                if (kg < n_ch && ready(&sh.cb_full[kg & 1], kg >> 1) && ready(&sh.g_empty[kg & 1], (kg >> 1) ^ 1)) {
                    const uint32_t st = base + (kg & 1) * kStageTc;
                    ptx::tc_fence_after();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        ptx::mma_f16(tmem + kColG + 128u * (kg & 1), ptx::kmajor_sw128_desc(st + (j >> 2) * kTile) + 2 * (j & 3),
                                     ptx::kmajor_sw128_desc(st + (2 + (j >> 2)) * kTile) + 2 * (j & 3), kIdescG, j > 0);
                    ptx::mma_commit(&sh.g_full[kg & 1]);
                    ++kg;
                    moved = true;
                }
                if (kd < kg && ready(&sh.x_full, kd) && ready(&sh.d_empty, kd ^ 1)) {
                    // D = B^T (w X): lo, then hi
                    const uint32_t st = base + (kd & 1) * kStageTc;
                    ptx::tc_fence_after();
#pragma unroll
                    for (int part = 1; part >= 0; --part)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            ptx::mma_f16(tmem + kColD, ptx::mnmajor_sw128_desc(st + 2 * kTile + j * 2048, kTile),
                                         ptx::mnmajor_sw128_desc(s_wx + part * kTile + j * 2048, 1024), kIdescD,
                                         part == 0 || j > 0);
                    ptx::mma_commit(&sh.d_full);
                    ptx::mma_commit(&sh.wx_empty);
                    ++kd;
                    moved = true;
                }
                if (ki < kg && ki <= ka && ready(&sh.s_full, ki) && ready(&sh.y_empty, ki ^ 1)) {
                    // Yi = C S^T
                    const uint32_t st = base + (ki & 1) * kStageTc;
                    ptx::tc_fence_after();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        ptx::mma_f16(tmem + kColYi, ptx::kmajor_sw128_desc(st + (j >> 2) * kTile) + 2 * (j & 3),
                                     ptx::mnmajor_sw128_desc(s_st + j * 2048, 1024), kIdescY, j > 0);
                    ptx::mma_commit(&sh.s_empty);
                    ++ki;
                    moved = true;
                }
                if (ka < ki && ka < kd && ready(&sh.m_full, ka)) {
                    // Ya = M X (x is there: D of the chunk is issued)
                    const uint32_t st = base + (ka & 1) * kStageTc;
                    ptx::tc_fence_after();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        ptx::mma_f16_ts(tmem + kColYa, tmem + kColM + 8 * j, ptx::mnmajor_sw128_desc(st + kCB + j * 2048, 1024),
                                        kIdescY, j > 0);
                    ptx::mma_commit(&sh.m_empty);
                    ptx::mma_commit(&sh.y_full);
                    ++ka;
                    moved = true;
                }
                if (freed < min(kd, ki)) {             // G came before both
                    ptx::mma_commit(&sh.cb_empty[freed & 1]);
                    ++freed;
                }
                if (moved) {
                    idle = 0;
                    since = 0;
                } else if ((++idle & 255u) == 0u) {
                    const uint64_t t = ptx::globaltimer();
                    if (since == 0) since = t;
                    if (*abort_flag || t - since > 1000000000ull) {
                        atomicOr(a.err, DFSSM_DEVERR_TIMEOUT);
                        *abort_flag = 1;
                        ok = false;
                    }
                }
            }
            if (!ok) {                                 // the MMAs issued so far end before tensor memory is given back
                ptx::mma_commit(&sh.drain);
                ptx::mbar_wait(&sh.drain, 0u);
            }
        }
    } else if (warp < 4) {
        // ---- decays, two warps in turn: lane l has tokens 4 l .. 4 l + 3
        const float bias = a.dt_bias[h], a2 = __fmul_rn(-expf(a.a_log[h]), kLog2e);
        float raw[4], nxt[4];
        auto load = [&](int k, float* r) {
            const int t0 = it.t0 + k * kT, n = min(kT, it.len - k * kT);
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = k < n_ch ? raw_dt(a, t0, n, h, 4 * lane + i) : 0.0f;
        };
        load(warp - 2, raw);
        for (int k = warp - 2; k < n_ch; k += 2) {
            load(k + 2, nxt);
            const float2 tsc = a.tile_scale[(int64_t)(it.chunk0 + k) * ngroups + g];
            const int n = min(kT, it.len - k * kT);
            float dt[4], v[4], up = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dt[i] = 4 * lane + i < n ? softplus_dt(__fadd_rn(raw[i], bias)) : 0.0f;
                v[i] = __fmul_rn(dt[i], a2);
                up = __fadd_rn(up, v[i]);
            }
            float down = up;
            const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(fmaxf(dt[0], dt[1]), fmaxf(dt[2], dt[3]))));
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float u = __shfl_up_sync(0xffffffffu, up, o), w = __shfl_down_sync(0xffffffffu, down, o);
                if (lane >= o) up = __fadd_rn(up, u);
                if (lane + o < 32) down = __fadd_rn(down, w);
            }
            float before = __shfl_up_sync(0xffffffffu, up, 1), after = __shfl_down_sync(0xffffffffu, down, 1);
            if (lane == 0) before = 0.0f;
            if (lane == 31) after = 0.0f;
            const float2 sc = pow2_scale(m, -1);
            float cum[4], left[4], dts[4];
            cum[0] = __fadd_rn(before, v[0]);
            left[3] = after;
#pragma unroll
            for (int i = 1; i < 4; ++i) cum[i] = __fadd_rn(cum[i - 1], v[i]);
#pragma unroll
            for (int i = 2; i >= 0; --i) left[i] = __fadd_rn(left[i + 1], v[i + 1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) dts[i] = __fmul_rn(dt[i], sc.x);
            if (!wait(&sh.dec_empty[k % kDec], ((uint32_t)(k / kDec) & 1u) ^ 1u)) break;
            TcDecay& d = sh.dec[k % kDec];
            reinterpret_cast<float4*>(d.cum)[lane] = make_float4(cum[0], cum[1], cum[2], cum[3]);
            reinterpret_cast<float4*>(d.dts)[lane] = make_float4(dts[0], dts[1], dts[2], dts[3]);
            reinterpret_cast<float4*>(d.wl)[lane] =
                make_float4(__fmul_rn(dts[0], exp2f(left[0])), __fmul_rn(dts[1], exp2f(left[1])),
                            __fmul_rn(dts[2], exp2f(left[2])), __fmul_rn(dts[3], exp2f(left[3])));
            reinterpret_cast<float4*>(d.done)[lane] = make_float4(exp2f(cum[0]), exp2f(cum[1]), exp2f(cum[2]), exp2f(cum[3]));
#pragma unroll
            for (int r = 0; r < 3; ++r) {
                const float c0 = __shfl_sync(0xffffffffu, cum[0], 8 * (r + 1));
                if (lane < 8 * (r + 1))
                    reinterpret_cast<float4*>(d.off[r])[lane] =
                        make_float4(__fmul_rn(dts[0], ex2(__fsub_rn(c0, cum[0]))), __fmul_rn(dts[1], ex2(__fsub_rn(c0, cum[1]))),
                                    __fmul_rn(dts[2], ex2(__fsub_rn(c0, cum[2]))), __fmul_rn(dts[3], ex2(__fsub_rn(c0, cum[3]))));
            }
            if (lane == 0) {
                d.kd = sc.y;
                d.kc = tsc.x;
                d.kb = tsc.y;
            }
            arrive(&sh.dec_full[k % kDec]);
#pragma unroll
            for (int i = 0; i < 4; ++i) raw[i] = nxt[i];
        }
    } else if (warp >= 4 && warp < 8) {
        // ---- M: row t of G, columns s up to the row's block of 32
        const int q4 = warp & 3;
        for (int k = 0; k < n_ch; ++k) {
            const int s2 = k & 1;
            const uint32_t ph2 = (uint32_t)(k >> 1) & 1u;
            const TcDecay& d = sh.dec[k % kDec];
            if (!wait(&sh.dec_full[k % kDec], (uint32_t)(k / kDec) & 1u) || !wait(&sh.g_full[s2], ph2) || !wait(&sh.m_empty, ((uint32_t)k & 1u) ^ 1u)) break;
            ptx::tc_fence_after();
            const float ct = d.cum[row];
            // In front of the row's block the decay is a product: of the row (from the block's first token) and of the
            // column (up to it, with dt, from the decays' warp). Both are <= 1.
            const float at = ex2(__fsub_rn(ct, d.cum[32 * q4]));
            const float2 at2 = make_float2(at, at);
#pragma unroll 1
            for (int cb = 0; cb < 2 * q4; ++cb) {
                uint32_t r[16], o[8];
                ptx::tmem_ld_32x32b_x16(t_lane + kColG + 128u * s2 + 16u * cb, r);
                ptx::tmem_ld_wait(r);
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 b = *reinterpret_cast<const float4*>(d.off[q4 - 1] + 16 * cb + i);
                    const float2 m0 = fmul2(fmul2(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), at2), make_float2(b.x, b.y));
                    const float2 m1 = fmul2(fmul2(make_float2(__uint_as_float(r[i + 2]), __uint_as_float(r[i + 3])), at2), make_float2(b.z, b.w));
                    o[i / 2] = f16x2_of(m0.x, m0.y);
                    o[i / 2 + 1] = f16x2_of(m1.x, m1.y);
                }
                ptx::tmem_st_32x32b_x8(t_lane + kColM + 8u * cb, o);
            }
#pragma unroll 1
            for (int cb = 2 * q4; cb < 2 * q4 + 2; ++cb) {         // the row's own block
                uint32_t r[16], o[8];
                ptx::tmem_ld_32x32b_x16(t_lane + kColG + 128u * s2 + 16u * cb, r);
                ptx::tmem_ld_wait(r);
                const int dg = lane - 16 * (cb & 1);               // columns of the piece up to the diagonal
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 cs = *reinterpret_cast<const float4*>(d.cum + 16 * cb + i);
                    const float4 ds = *reinterpret_cast<const float4*>(d.dts + 16 * cb + i);
                    const float m0 = i <= dg ? __fmul_rn(__fmul_rn(__uint_as_float(r[i]), ds.x), ex2(__fsub_rn(ct, cs.x))) : 0.0f;
                    const float m1 = i + 1 <= dg ? __fmul_rn(__fmul_rn(__uint_as_float(r[i + 1]), ds.y), ex2(__fsub_rn(ct, cs.y))) : 0.0f;
                    const float m2 = i + 2 <= dg ? __fmul_rn(__fmul_rn(__uint_as_float(r[i + 2]), ds.z), ex2(__fsub_rn(ct, cs.z))) : 0.0f;
                    const float m3 = i + 3 <= dg ? __fmul_rn(__fmul_rn(__uint_as_float(r[i + 3]), ds.w), ex2(__fsub_rn(ct, cs.w))) : 0.0f;
                    o[i / 2] = f16x2_of(m0, m1);
                    o[i / 2 + 1] = f16x2_of(m2, m3);
                }
                ptx::tmem_st_32x32b_x8(t_lane + kColM + 8u * cb, o);
            }
            if (k == 0) {                                          // what lies behind it is never written again
                uint32_t o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = 0u;
#pragma unroll 1
                for (int cb = 2 * q4 + 2; cb < 8; ++cb) ptx::tmem_st_32x32b_x8(t_lane + kColM + 8u * cb, o);
            }
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            arrive(&sh.m_full);
            if (lane == 0) {
                ptx::mbar_arrive(&sh.g_empty[s2]);
                ptx::mbar_arrive(&sh.dec_empty[k % kDec]);
            }
        }
    } else if (warp >= 8 && warp < 12) {
        // ---- X: row t of x
        bool ok = true;
        for (int k = 0; k < n_ch; ++k) {
            const int s2 = k & 1;
            const uint32_t ph2 = (uint32_t)(k >> 1) & 1u;
            const TcDecay& d = sh.dec[k % kDec];
            const uint32_t s_x = base + s2 * kStageTc + 4 * kTile;
            ok = ok && wait(&sh.xt_full[s2], ph2);
            const bool live = row < it.len - k * kT;
            uint32_t m = 0u;
#pragma unroll 2
            for (int i = 0; i < 8; ++i) {
                const uint4 v = ptx::lds128(piece(s_x, row, i));
                const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) m = max(m, max((w4[q] << 16) & 0x7FFF0000u, w4[q] & 0x7FFF0000u));
            }
            if (!live) m = 0u;
            m = __reduce_max_sync(0xffffffffu, m);
            uint32_t* red = sh.red[0][s2];
            if (lane == 0) red[warp & 3] = m;
            ok = ok && wait(&sh.dec_full[k % kDec], (uint32_t)(k / kDec) & 1u) && wait(&sh.wx_empty, ((uint32_t)k & 1u) ^ 1u);
            if (ptx::named_barrier_or(1, 128, !ok)) break;
            const float2 xs = pow2_scale(max(max(red[0], red[1]), max(red[2], red[3])), 13);
            const float w = __fmul_rn(d.wl[row], xs.x);
            const float2 xs2 = make_float2(xs.x, xs.x), w2 = make_float2(w, w);
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
                uint4 v = ptx::lds128(piece(s_x, row, i));
                if (!live) v = make_uint4(0u, 0u, 0u, 0u);
                const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
                uint32_t o[4], hi[4], lo[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float2 x2 = make_float2(bf16_lo(w4[q]), bf16_hi(w4[q]));
                    const float2 a2 = fmul2(x2, xs2), b2 = fmul2(x2, w2);
                    o[q] = f16x2_of(a2.x, a2.y);
                    const __half2 hh = __floats2half2_rn(b2.x, b2.y);
                    hi[q] = *reinterpret_cast<const uint32_t*>(&hh);
                    const float2 f = __half22float2(hh);
                    lo[q] = f16x2_of(__fsub_rn(b2.x, f.x), __fsub_rn(b2.y, f.y));
                }
                sts128(piece(s_x, row, i), o);
                sts128(piece(s_wx, row, i), hi);
                sts128(piece(s_wx + kTile, row, i), lo);
            }
            if (row == 0) sh.kx[k % kDec] = xs.y;
            ptx::fence_proxy_async_smem();
            arrive(&sh.x_full);
            if (lane == 0) ptx::mbar_arrive(&sh.dec_empty[k % kDec]);
        }
    } else if (warp >= 12 && warp < 16) {
        // ---- S: thread n holds the head's 64 channels of state n
        float2 S[kP / 2];
        const int64_t at = ((int64_t)it.seq * a.nheads + h) * kStateElems + row;
        const float* src = it.flags & kCut ? a.seg_state + ((int64_t)it.slot * a.nheads + h) * kStateElems + row
                                           : a.init ? a.init + at : nullptr;
#pragma unroll
        for (int i = 0; i < kP / 2; ++i)
            S[i] = src ? make_float2(src[(int64_t)(2 * i) * kN], src[(int64_t)(2 * i + 1) * kN]) : make_float2(0.0f, 0.0f);
        bool ok = true;
        for (int k = 0; k < n_ch; ++k) {
            const int s2 = k & 1;
            const uint32_t ph = (uint32_t)k & 1u;
            const TcDecay& d = sh.dec[k % kDec];
            float f0 = 0.0f, f1 = 0.0f;
#pragma unroll
            for (int i = 0; i < kP / 2; ++i) {
                f0 = fmaxf(f0, fabsf(S[i].x));
                f1 = fmaxf(f1, fabsf(S[i].y));
            }
            const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(f0, f1)));
            uint32_t* red = sh.red[1][s2];
            if (lane == 0) red[warp & 3] = m;
            ok = ok && wait(&sh.s_empty, ph ^ 1u);
            if (ptx::named_barrier_or(2, 128, !ok)) break;
            const float2 ss = pow2_scale(max(max(red[0], red[1]), max(red[2], red[3])), 13);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t o[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float2 v = fmul2(S[4 * i + q], make_float2(ss.x, ss.x));
                    o[q] = f16x2_of(v.x, v.y);
                }
                sts128(piece(s_st, row, i), o);
            }
            if (row == 0) sh.ks[s2] = ss.y;
            ptx::fence_proxy_async_smem();
            arrive(&sh.s_full);
            ok = wait(&sh.dec_full[k % kDec], (uint32_t)(k / kDec) & 1u) && wait(&sh.d_full, ph);
            if (!ok) continue;                         // the next barrier ends the group
            ptx::tc_fence_after();
            const float keep = d.done[kT - 1], back = __fmul_rn(__fmul_rn(d.kb, d.kd), *(volatile float*)&sh.kx[k % kDec]);
#pragma unroll
            for (int c = 0; c < kP; c += 16) {
                uint32_t r[16];
                ptx::tmem_ld_32x32b_x16(t_lane + kColD + c, r);
                ptx::tmem_ld_wait(r);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    S[c / 2 + i] = ffma2(make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), make_float2(back, back),
                                         fmul2(S[c / 2 + i], make_float2(keep, keep)));
            }
            ptx::tc_fence_before();
            arrive(&sh.d_empty);
            if (lane == 0) ptx::mbar_arrive(&sh.dec_empty[k % kDec]);
        }
        if (ok && p.final_state && (it.flags & kLast)) {
#pragma unroll
            for (int i = 0; i < kP / 2; ++i) {
                p.final_state[at + (int64_t)(2 * i) * kN] = S[i].x;
                p.final_state[at + (int64_t)(2 * i + 1) * kN] = S[i].y;
            }
        }
    } else if (warp >= 16) {
        // ---- Y: row t of y
        const float skip = a.d_skip[h];
        for (int k = 0; k < n_ch; ++k) {
            const int s2 = k & 1;
            const uint32_t ph = (uint32_t)k & 1u;
            const TcDecay& d = sh.dec[k % kDec];
            const uint32_t s_x = base + s2 * kStageTc + 4 * kTile;
            if (!wait(&sh.dec_full[k % kDec], (uint32_t)(k / kDec) & 1u) || !wait(&sh.y_full, ph)) break;
            ptx::tc_fence_after();
            const float kx = *(volatile float*)&sh.kx[k % kDec];
            const float alpha = __fmul_rn(d.done[row], __fmul_rn(*(volatile float*)&sh.ks[s2], d.kc));
            const float beta = __fmul_rn(__fmul_rn(d.kc, d.kb), __fmul_rn(d.kd, kx)), sx = __fmul_rn(skip, kx);
#pragma unroll 2
            for (int c = 0; c < kP; c += 16) {
                uint32_t yi[16], ya[16], o[8];
                ptx::tmem_ld_32x32b_x16(t_lane + kColYi + c, yi);
                ptx::tmem_ld_32x32b_x16(t_lane + kColYa + c, ya);
                ptx::tmem_ld_wait(yi);
                ptx::reg_fence(ya);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 x4 = ptx::lds128(piece(s_x, row, (c >> 3) + i));
                    const uint32_t w4[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float2 xf = __half22float2(*reinterpret_cast<const __half2*>(&w4[q]));
                        const int e = 8 * i + 2 * q;
                        const float2 in = fmul2(make_float2(__uint_as_float(yi[e]), __uint_as_float(yi[e + 1])), make_float2(alpha, alpha));
                        const float2 v = ffma2(make_float2(__uint_as_float(ya[e]), __uint_as_float(ya[e + 1])), make_float2(beta, beta), in);
                        o[4 * i + q] = bf16x2_of(ffma2(xf, make_float2(sx, sx), v));
                    }
                    sts128(piece(s_x, row, (c >> 3) + i), o + 4 * i);       // y over the x that only this thread still reads
                }
            }
            ptx::tc_fence_before();
            arrive(&sh.y_empty);                       // the row stores of the warp are also visible to it behind this
            const int n = min(kT, it.len - k * kT), t0 = it.t0 + k * kT;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = 32 * (warp & 3) + 4 * i + (lane >> 3), pc = lane & 7;
                const uint4 v = ptx::lds128(piece(s_x, r, pc));
                if (r < n) *reinterpret_cast<uint4*>(p.y + (int64_t)(t0 + r) * p.ldy + h * kP + 8 * pc) = v;
            }
            ptx::fence_proxy_async_smem();             // the tile's next contents come by TMA
            arrive(&sh.xt_empty[s2]);
            if (lane == 0) ptx::mbar_arrive(&sh.dec_empty[k % kDec]);
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

bool encode(CUtensorMap* map, CUtensorMapDataType type, const void* p, int64_t cols, int64_t rows, int64_t ld) {
    EncodeTiledFn enc = get_encode_fn();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)(2 * ld)};
    cuuint32_t box[2] = {64, kT}, estr[2] = {1, 1};
    return enc(map, type, 2, const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t setup_tc() {
    return cudaFuncSetAttribute(scan_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmem);
}

cudaError_t launch_tc(const Args& a, uint16_t* y, int64_t ldy, float* final_state, cudaStream_t s) {
    const int ngroups = a.nheads / a.per_group;
    CUtensorMap mt, mx;
    if (!encode(&mt, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a.tiles, kN, (int64_t)a.cap_chunks * ngroups * 2 * kT, kN) ||
        !encode(&mx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.x, (int64_t)a.nheads * kP, a.total, a.ldx))
        return cudaErrorInvalidValue;
    TcArgs p{a, y, ldy, final_state};
    return launch_after(scan_tc_kernel, a.cap_items * a.nheads, kTcThreads, kTcSmem, s, mt, mx, p);
}

}  // namespace scan
}  // namespace dfssm
