// sink_dkv.cu -- dk, dv of the base stream's window (row t, keys t - window < j <= t) in fp32, for the gradient with
// sinks (sink_bwd.cu), on the 5th-generation tensor cores.  Without sinks in the window's part it is the gradient of
// Eq. (4): the log-sum-exp and D = dO . o of the joint softmax are given.
//
// A CTA owns 128 keys of one (sequence, KV head): the MMA's M side, K and V resident in shared memory.  The query rows
// that can see them stream through a ring in rounds of 64 (64/G tokens x G heads): q's bf16 high part and residual
// and dO.  Per round
//   S^T = K q^T (both parts), dP^T = V dO^T                      fp32 in tensor memory, two buffers each
//   P^T = exp2(S^T c - lse), dS^T = P^T (dP^T - D)               as a bf16 high part and residual each, over S^T, dP^T
//   dV += P^T dO (two products), dK += dS^T q (three: the residuals' product is below fp32's rounding here)
// The MMA's fp32 accumulators are truncated at every step, not rounded: dk of 4800 rows a key (1284 steps) came out
// 1.9e-5 off.  So every 24 rounds (1536 rows, 288 steps) dV and dK are added to memory and begin anew.
// Four warpgroups take 16 rows (columns) of the round each: a warp's chain of loads, exponentials and stores is what a
// round waits for beside the MMAs.  4 x 16384 tokens of 32/8 heads, window 128: some 1000 us; 1 x 16384 280.
// Bound by a round's chain, MMAs and exponentials by turns: the 44 MMAs of 16 x (64 or 128) x 128 occupy the pipe for
// some 2050 of its 4200 cycles at d = 128, and without the residuals' products, or without the exponentials, a round
// would take 1.6 us instead of 2.2 either way.
// Roles (640 threads, one CTA an SM): warp 0 TMA producer; warp 1 tensor memory and the issue of S^T, dP^T; warp 3 that of
// dV, dK (one thread for both spends some 90 cycles an MMA, as long as a round takes); warp 2 the rows' log-sum-exp
// and D; warps 4-19 P^T, dS^T (lane = key), 16 columns a warpgroup, and at the end dK, dV.
// Tensor memory: S^T at 64 u, dP^T at 128 + 64 u (buffer u), dK at 256, dV at 256 + D.  Every wait is bounded.
#include "bwd_util.cuh"
#include "kernels.cuh"
#include "serve.cuh"
#include "tc.cuh"
#include "xattn.cuh"

namespace orthros {

namespace {

template <int D>
struct SdCfg {
    static constexpr int KEYS = 128, RB = 64;
    static constexpr int SLABS = D / 64;
    static constexpr int STG = 3;
    static constexpr int RUN = 24;            // rounds that dK, dV are summed over in tensor memory
    static constexpr int KSLAB = KEYS * 128;  // one 64-wide slab of the K (or V) tile
    static constexpr int RSLAB = RB * 128;    // one 64-wide slab of a row tile
    static constexpr int TILE = SLABS * RSLAB;
    static constexpr int K_OFF = 0;
    static constexpr int V_OFF = K_OFF + SLABS * KSLAB;
    static constexpr int ST_OFF = V_OFF + SLABS * KSLAB;  // [STG]: q high part, q residual, dO
    static constexpr int ST_BYTES = 3 * TILE;
    static constexpr int META_OFF = ST_OFF + STG * ST_BYTES;  // [STG][2][RB]: -lse, -D
    static constexpr int BAR_OFF = META_OFF + STG * 2 * RB * 4;
    static_assert(META_OFF % 16 == 0, "read 16 bytes at a time");
    static constexpr int NBARS = 1 + 3 * STG + 3 * 2 + 2;
    static constexpr int HOLD_OFF = BAR_OFF + NBARS * 8;
    static constexpr int USED = HOLD_OFF + 16 + 1024;
    static constexpr int SMEM = USED > 120 * 1024 ? USED : 120 * 1024;  // one CTA an SM: it takes all of tensor memory
    static_assert(SMEM <= 232448, "shared memory budget");
    static constexpr uint32_t TM_S = 0, TM_DP = 128, TM_DK = 256, TM_DV = 256 + D;
    static constexpr int THREADS = 640;
};

template <int D, int G>
__global__ void __launch_bounds__(640, 1) sink_dkv_tc_kernel(const __grid_constant__ SinkBwdMaps maps, const SinkBwdParams p)
{
    using C = SdCfg<D>;
    constexpr int TOK = C::RB / G;  // tokens of a round
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align1024(smem_raw);
    const uint32_t sbase = smem_u32(smem);
    uint64_t *kv_full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);  // K, V landed
    uint64_t *st_full = kv_full + 1;              // [STG] row tiles landed
    uint64_t *meta_full = st_full + C::STG;       // [STG] the rows' numbers staged
    uint64_t *st_empty = meta_full + C::STG;      // [STG] round's MMAs done with the stage
    uint64_t *s_full = st_empty + C::STG;         // [2] S^T, dP^T of a round complete
    uint64_t *p_full = s_full + 2;                // [2] P^T, dS^T written
    uint64_t *pv_done = s_full + 4;               // [2] dV, dK of a round complete
    uint64_t *acc_final = s_full + 6;             // of a run's last round
    uint64_t *acc_free = s_full + 7;              // a run's dK, dV read out of tensor memory
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + C::HOLD_OFF);
    float *meta = reinterpret_cast<float *>(smem + C::META_OFF);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kt0 = blockIdx.x * C::KEYS, bh = blockIdx.y, b = bh / p.Hkv, g = bh % p.Hkv;
    // rounds r: tokens r TOK ..; from the first that sees the tile to the last
    const int r0 = kt0 / TOK;
    const long long end = static_cast<long long>(kt0) + C::KEYS - 1 + p.window;  // tokens below this one
    const int r1 = static_cast<int>(((end < p.T ? end : p.T) + TOK - 1) / TOK);
    const int rounds = r1 - r0;  // at least 1

    __shared__ volatile int s_abort;  // a wait has given up
    if (threadIdx.x == 0) {
        s_abort = 0;
        mbar_init(kv_full, 1);
        for (int s = 0; s < C::STG; ++s) {
            mbar_init(&st_full[s], 1);
            mbar_init(&meta_full[s], 1);
            mbar_init(&st_empty[s], 1);
        }
        for (int u = 0; u < 2; ++u) {
            mbar_init(&s_full[u], 1);
            mbar_init(&p_full[u], 16);
            mbar_init(&pv_done[u], 1);
        }
        mbar_init(acc_final, 1);
        mbar_init(acc_free, 16);
        fence_barrier_init();
    }
    if (warp == 1)
        tmem_alloc(tmem_holder, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_holder;
    bool ok = true;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == 0) {
        // ------------------------------------------------------------------ producer
        if (lane == 0) {
            mbar_arrive_expect_tx(kv_full, 2 * C::SLABS * C::KSLAB);
#pragma unroll
            for (int sl = 0; sl < C::SLABS; ++sl) {
                tma_load_4d(smem + C::K_OFF + sl * C::KSLAB, &maps.k, kv_full, sl * 64, g, kt0, b);
                tma_load_4d(smem + C::V_OFF + sl * C::KSLAB, &maps.v, kv_full, sl * 64, g, kt0, b);
            }
            for (int i = 0; i < rounds; ++i) {
                const int s = i % C::STG, t0 = (r0 + i) * TOK;
                if ((i >= C::STG && !mbar_wait(&st_empty[s], static_cast<uint32_t>((i / C::STG - 1) & 1))) || s_abort) {
                    ok = false;
                    break;
                }
                uint8_t *st = smem + C::ST_OFF + s * C::ST_BYTES;
                mbar_arrive_expect_tx(&st_full[s], C::ST_BYTES);
#pragma unroll
                for (int sl = 0; sl < C::SLABS; ++sl) {
                    tma_load_4d(st + sl * C::RSLAB, &maps.q_hi, &st_full[s], sl * 64, g * G, t0, b);
                    tma_load_4d(st + C::TILE + sl * C::RSLAB, &maps.q_lo, &st_full[s], sl * 64, g * G, t0, b);
                    tma_load_4d(st + 2 * C::TILE + sl * C::RSLAB, &maps.dO, &st_full[s], sl * 64, g * G, t0, b);
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------------ S^T, dP^T
        if (elect_one()) {
            constexpr uint32_t IDESC_S = umma_idesc(128, C::RB, true, false);
            const uint64_t kdesc = umma_desc_sw128(sbase + C::K_OFF, 16, 1024);
            const uint64_t vdesc = umma_desc_sw128(sbase + C::V_OFF, 16, 1024);
            ok = mbar_wait(kv_full, 0);
            for (int i = 0; ok && i < rounds; ++i) {
                const int s = i % C::STG, u = i & 1;
                // S^T / dP^T buffer u is free once dV, dK of round i - 2 have read P^T, dS^T from it
                if (!(ok = mbar_wait(&st_full[s], static_cast<uint32_t>((i / C::STG) & 1)) &&
                           (i < 2 || mbar_wait(&pv_done[u], static_cast<uint32_t>(((i - 2) >> 1) & 1)))))
                    break;
                tc_fence_after();
                const uint32_t st = sbase + C::ST_OFF + s * C::ST_BYTES;
                const uint64_t hdesc = umma_desc_sw128(st, 16, 1024), ldesc = umma_desc_sw128(st + C::TILE, 16, 1024);
                const uint64_t odesc = umma_desc_sw128(st + 2 * C::TILE, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t ko = static_cast<uint32_t>((kk >> 2) * C::KSLAB + (kk & 3) * 32) >> 4;
                    const uint32_t ro = static_cast<uint32_t>((kk >> 2) * C::RSLAB + (kk & 3) * 32) >> 4;
                    umma_ss(tbase + C::TM_S + 64 * u, kdesc + ko, hdesc + ro, IDESC_S, kk != 0);
                    umma_ss(tbase + C::TM_S + 64 * u, kdesc + ko, ldesc + ro, IDESC_S, 1);
                    umma_ss(tbase + C::TM_DP + 64 * u, vdesc + ko, odesc + ro, IDESC_S, kk != 0);
                }
                umma_commit(&s_full[u]);
            }
        }
    } else if (warp == 3) {
        // ------------------------------------------------------------------ dV += P^T dO, dK += dS^T q
        if (elect_one()) {
            constexpr uint32_t IDESC_D = umma_idesc(128, D, true, true);
            for (int j = 0; ok && j < rounds; ++j) {
                const int u = j & 1, s = j % C::STG;
                if (!(ok = mbar_wait(&p_full[u], static_cast<uint32_t>((j >> 1) & 1)) &&
                           (j == 0 || j % C::RUN != 0 || mbar_wait(acc_free, static_cast<uint32_t>((j / C::RUN - 1) & 1)))))
                    break;
                tc_fence_after();
                const uint32_t st = sbase + C::ST_OFF + s * C::ST_BYTES;
                const uint64_t hdesc = umma_desc_sw128(st, C::RSLAB, 1024);
                const uint64_t ldesc = umma_desc_sw128(st + C::TILE, C::RSLAB, 1024);
                const uint64_t odesc = umma_desc_sw128(st + 2 * C::TILE, C::RSLAB, 1024);
                // 16 rows of P^T (dS^T) are 8 columns of high parts and 8 of residuals
#pragma unroll
                for (int kk = 0; kk < C::RB / 16; ++kk) {
                    const uint32_t acc = (j % C::RUN > 0 || kk > 0) ? 1u : 0u;
                    const uint64_t at = static_cast<uint64_t>(kk * (2048 >> 4));
                    const uint32_t ph = tbase + C::TM_S + 64 * u + 16 * kk;
                    const uint32_t sh = ph + (C::TM_DP - C::TM_S);
                    umma_ts(tbase + C::TM_DV, ph, odesc + at, IDESC_D, acc);
                    umma_ts(tbase + C::TM_DV, ph + 8, odesc + at, IDESC_D, 1);
                    umma_ts(tbase + C::TM_DK, sh, hdesc + at, IDESC_D, acc);
                    umma_ts(tbase + C::TM_DK, sh + 8, hdesc + at, IDESC_D, 1);
                    umma_ts(tbase + C::TM_DK, sh, ldesc + at, IDESC_D, 1);
                }
                // no commit that nothing waits for: round j + 2 waits for pv_done
                if (j == rounds - 1 || j % C::RUN == C::RUN - 1)
                    umma_commit(acc_final);
                if (j + 2 < rounds)
                    umma_commit(&pv_done[u]);
                if (j + C::STG < rounds)  // the producer waits for it
                    umma_commit(&st_empty[s]);
            }
            ok = ok && mbar_wait(acc_final, static_cast<uint32_t>(((rounds - 1) / C::RUN) & 1));
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------------ the rows' numbers
        for (int i = 0; ok && i < rounds; ++i) {
            const int s = i % C::STG;
            float m_lse[2], m_d[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int ct = lane + 32 * h, t = (r0 + i) * TOK + ct / G;
                m_lse[h] = -__int_as_float(0x7f800000);  // behind the last token: weights of zero
                m_d[h] = 0.f;
                if (t < p.T) {
                    const long long ri = (static_cast<long long>(b) * p.T + t) * p.Hq + g * G + ct % G;
                    m_lse[h] = -p.lse[ri];
                    m_d[h] = -p.Drow[ri];
                }
            }
            // the place is free once the stage of this round has landed: its producer waited for the MMAs of round
            // i - STG, which waited for that round's softmax
            if (!(ok = warp_wait(&st_full[s], static_cast<uint32_t>((i / C::STG) & 1))))
                break;
            float *m = meta + s * 2 * C::RB;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                m[lane + 32 * h] = m_lse[h];
                m[C::RB + lane + 32 * h] = m_d[h];
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&meta_full[s]);
        }
    } else {
        // ------------------------------------------------------------------ P^T, dS^T, then dK, dV
        const int rw = warp & 3, part = (warp - 4) >> 2;  // columns 16 part .. of a round
        const int key = kt0 + rw * 32 + lane;
        const uint32_t tl = tbase + (static_cast<uint32_t>(rw * 32) << 16);
        const float2 c22 = make_float2(p.scale * kLog2eF, p.scale * kLog2eF);
        for (int i = 0; i < rounds; ++i) {
            const int s = i % C::STG, u = i & 1;
            if (!(ok = warp_wait(&s_full[u], static_cast<uint32_t>((i >> 1) & 1)) &&
                       warp_wait(&meta_full[s], static_cast<uint32_t>((i / C::STG) & 1))))
                break;
            tc_fence_after();
            const float *m = meta + s * 2 * C::RB + 16 * part;
            const uint32_t s_at = tl + C::TM_S + 64 * u + 16 * part, d_at = tl + C::TM_DP + 64 * u + 16 * part;
            // what the warp's 32 keys are to the 16 rows: seen by all of them, by none, or by some
            const int t0 = (r0 + i) * TOK + 16 * part / G, t1 = (r0 + i) * TOK + (16 * part + 15) / G;
            const int k0 = kt0 + rw * 32;
            if (t1 < k0 || k0 + 31 <= t0 - p.window) {
                const uint32_t zero[16] = {};
                tmem_st16(s_at, zero);
                tmem_st16(d_at, zero);
            } else {
                const bool whole = k0 + 31 <= t0 && k0 > t1 - p.window;
                uint32_t sv[16], dv[16];
                tmem_ld16(s_at, sv);
                tmem_ld16(d_at, dv);
                tmem_wait_ld();
                uint32_t ph[8], pl[8], sh[8], sl[8];
#pragma unroll
                for (int e4 = 0; e4 < 4; ++e4) {
                    const float4 nl = *reinterpret_cast<const float4 *>(m + 4 * e4);
                    const float4 nd = *reinterpret_cast<const float4 *>(m + C::RB + 4 * e4);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int c = 4 * e4 + 2 * y, e = 2 * e4 + y;
                        float2 pr = ffma2(make_float2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), c22,
                                          y ? make_float2(nl.z, nl.w) : make_float2(nl.x, nl.y));
                        pr = make_float2(fast_exp2(pr.x), fast_exp2(pr.y));
                        float2 ds = fmul2(pr, fadd2(make_float2(__uint_as_float(dv[c]), __uint_as_float(dv[c + 1])),
                                                    y ? make_float2(nd.z, nd.w) : make_float2(nd.x, nd.y)));
                        if (!whole) {
                            const int ta = (r0 + i) * TOK + (16 * part + c) / G, tb = (r0 + i) * TOK + (16 * part + c + 1) / G;
                            const bool sa = key <= ta && key > ta - p.window, sb = key <= tb && key > tb - p.window;
                            pr = make_float2(sa ? pr.x : 0.f, sb ? pr.y : 0.f);
                            ds = make_float2(sa ? ds.x : 0.f, sb ? ds.y : 0.f);
                        }
                        split_pair2(pr, ph[e], pl[e]);
                        split_pair2(ds, sh[e], sl[e]);
                    }
                }
                tmem_st8(s_at, ph);
                tmem_st8(s_at + 8, pl);
                tmem_st8(d_at, sh);
                tmem_st8(d_at + 8, sl);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&p_full[u]);
            if (i < rounds - 1 && i % C::RUN < C::RUN - 1)
                continue;
            // a run's end: dK (scaled) by the first two groups, dV by the others, half of the columns each
            if (!(ok = warp_wait(acc_final, static_cast<uint32_t>((i / C::RUN) & 1))))
                break;
            tc_fence_after();
            const bool val = part >= 2;
            const float f = val ? 1.f : p.scale;
            float *dst = (val ? p.dv : p.dk) + ((static_cast<long long>(b) * p.T + key) * p.Hkv + g) * D;
#pragma unroll 1
            for (int c = D / 2 * (part & 1); c < D / 2 * (part & 1) + D / 2; c += 32) {
                uint32_t w[32];
                tmem_ld32(tl + (val ? C::TM_DV : C::TM_DK) + c, w);
                tmem_wait_ld();
                if (key < p.T) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (i >= C::RUN)
                            y = *reinterpret_cast<const float4 *>(dst + c + e);
                        y.x = fmaf(__uint_as_float(w[e]), f, y.x);
                        y.y = fmaf(__uint_as_float(w[e + 1]), f, y.y);
                        y.z = fmaf(__uint_as_float(w[e + 2]), f, y.z);
                        y.w = fmaf(__uint_as_float(w[e + 3]), f, y.w);
                        *reinterpret_cast<float4 *>(dst + c + e) = y;
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && i < rounds - 1)
                mbar_arrive(acc_free);
        }
    }
    if (!ok) {  // of an issuing warp its elected lane alone
        s_abort = 1;
        if (lane == 0 || warp == 1 || warp == 3)
            record_error(p.dev_err, ORTHROS_DEVERR_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    if (s_abort) {
        drain_in_flight();
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
    // This grid starts once every CTA of dq's has seen the prepared rows complete, and uses nothing of dq's: the two
    // run side by side where SMs are left.  What comes after this grid comes after dq's too.
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int D, int G>
cudaError_t launch_dkv(const SinkBwdMaps &maps, const SinkBwdParams &p, cudaStream_t stream)
{
    using C = SdCfg<D>;
    auto kern = sink_dkv_tc_kernel<D, G>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess)
        return e;
    return launch_dependent(kern, dim3((p.T + C::KEYS - 1) / C::KEYS, p.B * p.Hkv), C::THREADS, C::SMEM, stream, maps, p);
}

}  // namespace

cudaError_t launch_sink_dkv(int D, const SinkBwdMaps &maps, const SinkBwdParams &p, cudaStream_t stream)
{
    const int G = p.Hq / p.Hkv;
#define ORTHROS_DKV_CASE(DD, GG) \
    if (D == DD && G == GG)      \
        return launch_dkv<DD, GG>(maps, p, stream);
    ORTHROS_DKV_CASE(128, 1)
    ORTHROS_DKV_CASE(128, 2)
    ORTHROS_DKV_CASE(128, 4)
    ORTHROS_DKV_CASE(128, 8)
    ORTHROS_DKV_CASE(128, 16)
    ORTHROS_DKV_CASE(64, 1)
    ORTHROS_DKV_CASE(64, 2)
    ORTHROS_DKV_CASE(64, 4)
    ORTHROS_DKV_CASE(64, 8)
    ORTHROS_DKV_CASE(64, 16)
#undef ORTHROS_DKV_CASE
    return cudaErrorInvalidValue;
}

}  // namespace orthros
