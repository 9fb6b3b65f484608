// sink_dq.cu -- dq, dalpha and dbeta of the base stream with attention sinks (sink_bwd.cu) on the 5th-generation tensor
// cores: dq_t = scale sum_j dS_tj k_j over row t's window and the sinks, dq_raw = dq alpha, dalpha = sum_t x_t dq_t,
// dbeta = sum_t dq_t.
//
// A tile is 128 query rows (128/G tokens x G heads of a KV head): the MMA's M side, q's two bf16 parts and dO resident in
// shared memory.  Its keys stream through a ring in rounds of 64 (for tiles that have left key 0 behind, first a round
// of 32 with the sinks, from a tensor map that ends with them).  Per round
//   S = q K^T (both parts), dP = dO V^T            fp32 in tensor memory, two buffers each
//   dS = P (dP - D), P = exp2(S c - lse)           as a bf16 high part and residual over dP
//   dQ += dS K (two products)                      fp32 in tensor memory, two buffers
// A persistent CTA an SM walks consecutive tiles; while a tile's last dS, dQ and results are on their way the next
// one's rows arrive.  The MMA's accumulators are truncated at every step: every 32 rounds (2048 keys) dQ is added to
// memory and begins anew.
// Bound by a tile's chain: 96 KB of rows in, 5 rounds of 40 MMAs at window 128, 64 KB of fp32 out (d = 128); 1 x 16384
// tokens of 32/8 heads take 277 us, and 120 less without the results' work.
// Roles (512 threads): warps 0, 2 TMA producers of rows, of keys; warp 1 tensor memory and the issue of S, dP; warp 3 that
// of dQ; warps 4-7, 8-11 dS of
// a round's columns 0-31, 32-63 (lane = row); warps 12-15 dq_raw and the sums over a tile's rows, 16 columns at a
// time: up to four heads by shuffles that halve a lane's columns as they double its rows; more heads, whose sums
// would take too many registers, through a transposing buffer, where a thread sums one column of one head over its
// rows (the buffer for four heads, with its two barriers a step, bound the kernel: 10 us a tile).  Every wait is
// bounded.
#include "bwd_util.cuh"
#include "kernels.cuh"
#include "serve.cuh"
#include "tc.cuh"
#include "xattn.cuh"

namespace orthros {

namespace {

template <int D>
struct SqCfg {
    static constexpr int ROWS = 128, KB = 64;
    static constexpr int SLABS = D / 64;
    static constexpr int STG = 3;
    static constexpr int RUN = 32;            // rounds that dQ is summed over in tensor memory
    static constexpr int QSLAB = ROWS * 128;  // one 64-wide slab of a row tile
    static constexpr int QTILE = SLABS * QSLAB;
    static constexpr int KSLAB = KB * 128;
    static constexpr int KTILE = SLABS * KSLAB;
    static constexpr int Q_OFF = 0;  // q high part, q residual, dO
    static constexpr int ST_OFF = 3 * QTILE;  // [STG]: K, V
    static constexpr int TP_OFF = ST_OFF + STG * 2 * KTILE;  // float [2][128][17]: x dq and dq of 16 columns
    static constexpr int BAR_OFF = TP_OFF + 2 * ROWS * 17 * 4;
    static constexpr int NBARS = 2 + 2 * STG + 3 * 2 + 2 * 2;
    static constexpr int HOLD_OFF = BAR_OFF + NBARS * 8;
    static constexpr int USED = HOLD_OFF + 16 + 1024;
    static constexpr int SMEM = USED > 120 * 1024 ? USED : 120 * 1024;  // one CTA an SM: it takes all of tensor memory
    static_assert(SMEM <= 232448 && BAR_OFF % 8 == 0, "shared memory budget");
    static constexpr uint32_t TM_S = 0, TM_DP = 128, TM_DQ = 256;
    static constexpr int THREADS = 512;
};

// tile tau of the stream: which rows, which key blocks
struct SqTile {
    int bh, u0, lo, far, rounds;
};

template <int D, int G>
__device__ __forceinline__ SqTile sq_tile(const SinkBwdParams &p, long long tau, int per_stream)
{
    constexpr int TOK = SqCfg<D>::ROWS / G;
    SqTile t;
    t.bh = static_cast<int>(tau / per_stream);
    t.u0 = static_cast<int>(tau % per_stream) * TOK;
    t.lo = max(0, t.u0 - p.window + 1) / 64;
    t.far = p.sinks > 0 && t.lo > 0;
    t.rounds = t.far + (min(p.T, t.u0 + TOK) - 1) / 64 - t.lo + 1;
    return t;
}

template <int D, int G>
__global__ void __launch_bounds__(512, 1) sink_dq_tc_kernel(const __grid_constant__ SinkDqMaps maps, const SinkBwdParams p)
{
    using C = SqCfg<D>;
    constexpr int TOK = C::ROWS / G;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align1024(smem_raw);
    const uint32_t sbase = smem_u32(smem);
    uint64_t *q_full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);  // a tile's rows landed
    uint64_t *q_free = q_full + 1;             // a tile's S, dP complete
    uint64_t *kv_full = q_full + 2;            // [STG] round's keys landed
    uint64_t *kv_empty = kv_full + C::STG;     // [STG] its MMAs done
    uint64_t *s_full = kv_empty + C::STG;      // [2] S, dP of a round complete
    uint64_t *p_full = s_full + 2;             // [2] dS written
    uint64_t *ds_free = s_full + 4;            // [2] dQ of a round complete
    uint64_t *dq_full = s_full + 6;            // [2] dQ of a run complete
    uint64_t *dq_free = s_full + 8;            // [2] and read
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + C::HOLD_OFF);
    __shared__ volatile int s_abort;  // a wait has given up

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per_stream = (p.T + TOK - 1) / TOK;
    const long long tiles = static_cast<long long>(p.B) * p.Hkv * per_stream;
    const long long t_begin = tiles * blockIdx.x / gridDim.x, t_end = tiles * (blockIdx.x + 1) / gridDim.x;

    if (threadIdx.x == 0) {
        s_abort = 0;
        mbar_init(q_full, 1);
        mbar_init(q_free, 1);
        for (int s = 0; s < C::STG; ++s) {
            mbar_init(&kv_full[s], 1);
            mbar_init(&kv_empty[s], 1);
        }
        for (int u = 0; u < 2; ++u) {
            mbar_init(&s_full[u], 1);
            mbar_init(&p_full[u], 8);
            mbar_init(&ds_free[u], 1);
            mbar_init(&dq_full[u], 1);
            mbar_init(&dq_free[u], 4);
        }
        fence_barrier_init();
    }
    if (warp == 1)
        tmem_alloc(tmem_holder, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_holder;
    bool ok = true;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // for the prepared rows
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == 0) {
        // ------------------------------------------------------------------ rows
        if (lane == 0) {
            int j = 0;
            for (long long tau = t_begin; tau < t_end; ++tau, ++j) {
                const SqTile tl = sq_tile<D, G>(p, tau, per_stream);
                const int b = tl.bh / p.Hkv, g = tl.bh % p.Hkv;
                if ((j > 0 && !mbar_wait(q_free, static_cast<uint32_t>((j - 1) & 1))) || s_abort) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(q_full, 3 * C::QTILE);
#pragma unroll
                for (int sl = 0; sl < C::SLABS; ++sl) {
                    uint8_t *dst = smem + C::Q_OFF + sl * C::QSLAB;
                    tma_load_4d(dst, &maps.q_hi, q_full, sl * 64, g * G, tl.u0, b);
                    tma_load_4d(dst + C::QTILE, &maps.q_lo, q_full, sl * 64, g * G, tl.u0, b);
                    tma_load_4d(dst + 2 * C::QTILE, &maps.dO, q_full, sl * 64, g * G, tl.u0, b);
                }
                if (tau + 1 < t_end) {  // the next tile's rows on their way to L2: there is one buffer for them here
                    const SqTile nx = sq_tile<D, G>(p, tau + 1, per_stream);
#pragma unroll
                    for (int sl = 0; sl < C::SLABS; ++sl) {
                        tma_prefetch_4d(&maps.q_hi, sl * 64, nx.bh % p.Hkv * G, nx.u0, nx.bh / p.Hkv);
                        tma_prefetch_4d(&maps.q_lo, sl * 64, nx.bh % p.Hkv * G, nx.u0, nx.bh / p.Hkv);
                        tma_prefetch_4d(&maps.dO, sl * 64, nx.bh % p.Hkv * G, nx.u0, nx.bh / p.Hkv);
                    }
                }
            }
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------------ keys
        if (lane == 0) {
            long long i = 0;
            for (long long tau = t_begin; ok && tau < t_end; ++tau) {
                const SqTile tl = sq_tile<D, G>(p, tau, per_stream);
                const int b = tl.bh / p.Hkv, g = tl.bh % p.Hkv;
                for (int r = 0; r < tl.rounds; ++r, ++i) {
                    const int s = static_cast<int>(i % C::STG);
                    if ((i >= C::STG && !mbar_wait(&kv_empty[s], static_cast<uint32_t>((i / C::STG - 1) & 1))) || s_abort) {
                        ok = false;
                        break;
                    }
                    const bool sink = r < tl.far;
                    const CUtensorMap *mk = sink ? &maps.ks : &maps.k, *mv = sink ? &maps.vs : &maps.v;
                    const int row = sink ? 0 : (tl.lo + r - tl.far) * C::KB;
                    uint8_t *dst = smem + C::ST_OFF + s * 2 * C::KTILE;
                    mbar_arrive_expect_tx(&kv_full[s], (sink ? 1 : 2) * C::KTILE);  // 32 keys or 64, of K and of V
#pragma unroll
                    for (int sl = 0; sl < C::SLABS; ++sl) {
                        tma_load_4d(dst + sl * C::KSLAB, mk, &kv_full[s], sl * 64, g, row, b);
                        tma_load_4d(dst + C::KTILE + sl * C::KSLAB, mv, &kv_full[s], sl * 64, g, row, b);
                    }
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------------ S, dP
        if (elect_one()) {
            constexpr uint32_t IDESC_S = umma_idesc(128, C::KB, true, false), IDESC_S32 = umma_idesc(128, 32, true, false);
            const uint64_t hdesc = umma_desc_sw128(sbase + C::Q_OFF, 16, 1024);
            const uint64_t ldesc = umma_desc_sw128(sbase + C::Q_OFF + C::QTILE, 16, 1024);
            const uint64_t odesc = umma_desc_sw128(sbase + C::Q_OFF + 2 * C::QTILE, 16, 1024);
            long long i = 0;
            int j = 0;
            for (long long tau = t_begin; ok && tau < t_end; ++tau, ++j) {
                const SqTile tl = sq_tile<D, G>(p, tau, per_stream);
                if (!(ok = mbar_wait(q_full, static_cast<uint32_t>(j & 1))))
                    break;
                for (int r = 0; ok && r < tl.rounds; ++r, ++i) {
                    const int s = static_cast<int>(i % C::STG), u = static_cast<int>(i & 1);
                    // S / dP buffer u is free once dQ of round i - 2 has read dS from it
                    if (!(ok = mbar_wait(&kv_full[s], static_cast<uint32_t>((i / C::STG) & 1)) &&
                               (i < 2 || mbar_wait(&ds_free[u], static_cast<uint32_t>(((i - 2) >> 1) & 1)))))
                        break;
                    tc_fence_after();
                    const uint32_t st = sbase + C::ST_OFF + s * 2 * C::KTILE;
                    const uint64_t kdesc = umma_desc_sw128(st, 16, 1024), vdesc = umma_desc_sw128(st + C::KTILE, 16, 1024);
                    const uint32_t idesc = r < tl.far ? IDESC_S32 : IDESC_S;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t qo = static_cast<uint32_t>((kk >> 2) * C::QSLAB + (kk & 3) * 32) >> 4;
                        const uint32_t ko = static_cast<uint32_t>((kk >> 2) * C::KSLAB + (kk & 3) * 32) >> 4;
                        umma_ss(tbase + C::TM_S + 64 * u, hdesc + qo, kdesc + ko, idesc, kk != 0);
                        umma_ss(tbase + C::TM_S + 64 * u, ldesc + qo, kdesc + ko, idesc, 1);
                        umma_ss(tbase + C::TM_DP + 64 * u, odesc + qo, vdesc + ko, idesc, kk != 0);
                    }
                    umma_commit(&s_full[u]);
                    if (r == tl.rounds - 1)
                        umma_commit(q_free);
                }
            }
            // no commit is in flight when the CTA ends
            if (ok && j > 0)
                ok = mbar_wait(q_free, static_cast<uint32_t>((j - 1) & 1));
        }
    } else if (warp == 3) {
        // ------------------------------------------------------------------ dQ += dS K
        if (elect_one()) {
            constexpr uint32_t IDESC_Q = umma_idesc(128, D, true, true);
            long long i = 0;
            int run = 0;
            for (long long tau = t_begin; ok && tau < t_end; ++tau) {
                const SqTile tl = sq_tile<D, G>(p, tau, per_stream);
                for (int r = 0; ok && r < tl.rounds; ++r, ++i) {
                    const int s = static_cast<int>(i % C::STG), u = static_cast<int>(i & 1), buf = run & 1;
                    const bool begin = r % C::RUN == 0, end = r == tl.rounds - 1 || r % C::RUN == C::RUN - 1;
                    if (!(ok = mbar_wait(&p_full[u], static_cast<uint32_t>((i >> 1) & 1)) &&
                               (!begin || run < 2 || mbar_wait(&dq_free[buf], static_cast<uint32_t>((run / 2 - 1) & 1)))))
                        break;
                    tc_fence_after();
                    const uint64_t kdesc = umma_desc_sw128(sbase + C::ST_OFF + s * 2 * C::KTILE, C::KSLAB, 1024);
                    const uint32_t to = tbase + C::TM_DQ + D * buf;
                    const int steps = r < tl.far ? 2 : 4;  // 16 keys each
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        if (kk < steps) {
                            const uint32_t a = tbase + C::TM_DP + 64 * u + 32 * (kk >> 1) + 8 * (kk & 1);
                            const uint64_t bd = kdesc + static_cast<uint64_t>(kk * (2048 >> 4));
                            umma_ts(to, a, bd, IDESC_Q, begin && kk == 0 ? 0u : 1u);
                            umma_ts(to, a + 16, bd, IDESC_Q, 1);
                        }
                    umma_commit(&ds_free[u]);
                    umma_commit(&kv_empty[s]);
                    if (end) {
                        umma_commit(&dq_full[buf]);
                        ++run;
                    }
                }
            }
            // no commit is in flight when the CTA ends
            for (long long k = i > 2 ? i - 2 : 0; ok && k < i; ++k)
                ok = mbar_wait(&ds_free[k & 1], static_cast<uint32_t>((k >> 1) & 1));
            for (long long k = i > C::STG ? i - C::STG : 0; ok && k < i; ++k)
                ok = mbar_wait(&kv_empty[k % C::STG], static_cast<uint32_t>((k / C::STG) & 1));
        }
    } else if (warp >= 4 && warp < 12) {
        // ------------------------------------------------------------------ dS (lane = row)
        const int rw = warp & 3, half = (warp - 4) >> 2, row = rw * 32 + lane;
        const uint32_t tl_at = tbase + (static_cast<uint32_t>(rw * 32) << 16);
        const float2 c22 = make_float2(p.scale * kLog2eF, p.scale * kLog2eF);
        long long i = 0;
        for (long long tau = t_begin; ok && tau < t_end; ++tau) {
            const SqTile tl = sq_tile<D, G>(p, tau, per_stream);
            const int b = tl.bh / p.Hkv, g = tl.bh % p.Hkv;
            const int t = tl.u0 + row / G;
            float lse = __int_as_float(0x7f800000), Drow = 0.f;  // behind the last token: weights of zero
            if (t < p.T) {
                const long long ri = (static_cast<long long>(b) * p.T + t) * p.Hq + g * G + row % G;
                lse = p.lse[ri];
                Drow = p.Drow[ri];
            }
            const int klo = t - p.window, ksink = p.sinks, khi = t;  // keys klo + 1 .. t, and the sinks
            const int t_lo = tl.u0 + rw * 32 / G, t_hi = tl.u0 + (rw * 32 + 31) / G;  // the warp's tokens
            const float2 nlse2 = make_float2(-lse, -lse), nd2 = make_float2(-Drow, -Drow);
            for (int r = 0; r < tl.rounds; ++r, ++i) {
                const int u = static_cast<int>(i & 1);
                const bool sink = r < tl.far;
                if (!(ok = warp_wait(&s_full[u], static_cast<uint32_t>((i >> 1) & 1))))
                    break;
                if (!sink || half == 0) {
                    tc_fence_after();
                    const int key0 = (sink ? 0 : (tl.lo + r - tl.far) * C::KB) + 32 * half;
                    const uint32_t s_at = tl_at + C::TM_S + 64 * u + 32 * half, d_at = tl_at + C::TM_DP + 64 * u + 32 * half;
                    // what the warp's rows see of the 32 keys: all of them, none, or some
                    const bool whole = key0 + 31 <= t_lo && (key0 > t_hi - p.window || key0 + 31 < p.sinks);
                    const bool none = key0 > t_hi || (key0 + 31 <= t_lo - p.window && key0 >= p.sinks);
                    if (none) {
                        const uint32_t zero[16] = {};
                        tmem_st16(d_at, zero);
                        tmem_st16(d_at + 16, zero);
                    } else {
                        uint32_t sv[2][16], dv[2][16];
                        tmem_ld16(s_at, sv[0]);
                        tmem_ld16(d_at, dv[0]);
                        tmem_ld16(s_at + 16, sv[1]);
                        tmem_ld16(d_at + 16, dv[1]);
                        tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            uint32_t hi[8], lo[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const int c = 2 * e, key = key0 + 16 * x + c;
                                float2 y = ffma2(make_float2(__uint_as_float(sv[x][c]), __uint_as_float(sv[x][c + 1])), c22, nlse2);
                                y = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                                y = fmul2(y, fadd2(make_float2(__uint_as_float(dv[x][c]), __uint_as_float(dv[x][c + 1])), nd2));
                                if (!whole) {
                                    y.x = key <= khi && (key > klo || key < ksink) ? y.x : 0.f;
                                    y.y = key < khi && (key >= klo || key + 1 < ksink) ? y.y : 0.f;
                                }
                                split_pair2(y, hi[e], lo[e]);
                            }
                            tmem_st8(d_at + 8 * x, hi);
                            tmem_st8(d_at + 16 + 8 * x, lo);
                        }
                    }
                    tmem_wait_st();
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&p_full[u]);
            }
        }
    } else if (warp >= 12) {
        // ------------------------------------------------------------------ dq_raw and the sums
        const int rw = warp & 3, row = rw * 32 + lane, tid = threadIdx.x - 384;
        float *tp = reinterpret_cast<float *>(smem + C::TP_OFF);
        const bool v8 = (reinterpret_cast<uintptr_t>(p.dq) & 31) == 0;
        // Without shuffles a thread sums column tid % 16 of each 16 over a head's rows, or over those of two heads
        constexpr bool FOLD = G <= 4;  // by shuffles; PER: sums of 16 columns that a thread has in the end
        constexpr int PER = G == 16 || G == 4 ? 2 : 1;
        float sa[D / 16][PER], sb[D / 16][PER];
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
            for (int e = 0; e < PER; ++e)
                sa[c][e] = sb[c][e] = 0.f;
        const int grp = tid >> 4, col = tid & 15, h0 = G == 16 ? 2 * grp : grp % G;
        // sum of t[16] over the warp's rows of this lane's head: PER columns from fold_col on, a lane
        const int fold_col = (lane & 16) / 2 + (G <= 8 ? (lane & 8) / 2 : 0) + (G <= 4 ? (lane & 4) / 2 : 0) + (G <= 2 ? (lane & 2) / 2 : 0);
        auto fold = [&](float(&t)[16]) {
#pragma unroll
            for (int bit = 16, n = 8; bit >= G; bit >>= 1, n >>= 1) {
                if (n == 0) {
                    t[0] += __shfl_xor_sync(0xffffffffu, t[0], bit);
                } else {
#pragma unroll
                    for (int i = 0; i < n; ++i) {
                        const float give = lane & bit ? t[i] : t[i + n];
                        t[i] = (lane & bit ? t[i + n] : t[i]) + __shfl_xor_sync(0xffffffffu, give, bit);
                    }
                }
            }
        };
        auto flush = [&](int g) {
            if (FOLD && G == 1 && (lane & 1))  // the last of five steps left both lanes the same sum
                return;
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
#pragma unroll
                for (int e = 0; e < PER; ++e) {
                    const int at = FOLD ? (g * G + lane % G) * D + 16 * c + fold_col + e : (g * G + h0 + e) * D + 16 * c + col;
                    atomicAdd(p.dalpha + at, sa[c][e]);
                    atomicAdd(p.dbeta + at, sb[c][e]);
                    sa[c][e] = sb[c][e] = 0.f;
                }
        };
        int run = 0, cur_g = -1;
        for (long long tau = t_begin; ok && tau < t_end; ++tau) {
            const SqTile tl = sq_tile<D, G>(p, tau, per_stream);
            const int b = tl.bh / p.Hkv, g = tl.bh % p.Hkv;
            if (g != cur_g) {
                if (cur_g >= 0)
                    flush(cur_g);
                cur_g = g;
            }
            const int t = tl.u0 + row / G, h = g * G + row % G;
            const bool live = t < p.T;
            const long long at0 = ((static_cast<long long>(b) * p.T + (live ? t : 0)) * p.Hq + h) * D;
            float *dst = p.dq + at0;
            const uint4 *xrow = reinterpret_cast<const uint4 *>(p.q + at0);
            for (int r0 = 0; r0 < tl.rounds; r0 += C::RUN, ++run) {
                const bool last = r0 + C::RUN >= tl.rounds;
                const int buf = run & 1;
                uint4 xa = __ldg(xrow), xb = __ldg(xrow + 1);  // 16 values of x, a step ahead
                const bool got = warp_wait(&dq_full[buf], static_cast<uint32_t>((run >> 1) & 1));
                if (!(ok = FOLD ? got : bar_red_and(1, 128, got)))
                    break;
                tc_fence_after();
                const uint32_t at = tbase + (static_cast<uint32_t>(rw * 32) << 16) + C::TM_DQ + D * buf;
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t w[16];
                    tmem_ld16(at + 16 * c, w);
                    const uint32_t xw[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};
                    if (c + 1 < D / 16) {
                        xa = __ldg(xrow + 2 * c + 2);
                        xb = __ldg(xrow + 2 * c + 3);
                    }
                    tmem_wait_ld();
                    if (c == D / 16 - 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(&dq_free[buf]);
                    }
                    if (r0 > 0 && live)
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            const float4 y = *reinterpret_cast<const float4 *>(dst + 16 * c + e);
                            w[e] = __float_as_uint(__uint_as_float(w[e]) + y.x);
                            w[e + 1] = __float_as_uint(__uint_as_float(w[e + 1]) + y.y);
                            w[e + 2] = __float_as_uint(__uint_as_float(w[e + 2]) + y.z);
                            w[e + 3] = __float_as_uint(__uint_as_float(w[e + 3]) + y.w);
                        }
                    if (last) {
                        float ta[16], tb[16];
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            const float4 a = __ldg(reinterpret_cast<const float4 *>(p.alpha + h * D + 16 * c + e));
                            const float2 x0 = unpack_bf16x2(xw[e / 2]), x1 = unpack_bf16x2(xw[e / 2 + 1]);
                            const float xv[4] = {x0.x, x0.y, x1.x, x1.y}, av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const float y = live ? __uint_as_float(w[e + q]) * p.scale : 0.f;
                                ta[e + q] = live ? xv[q] * y : 0.f;
                                tb[e + q] = y;
                                w[e + q] = __float_as_uint(y * av[q]);
                            }
                        }
                        if (FOLD) {
                            fold(ta);
                            fold(tb);
#pragma unroll
                            for (int e = 0; e < PER; ++e) {
                                sa[c][e] += ta[e];
                                sb[c][e] += tb[e];
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                tp[row * 17 + e] = ta[e];
                                tp[(C::ROWS + row) * 17 + e] = tb[e];
                            }
                        }
                    }
                    if (live) {
#pragma unroll
                        for (int e = 0; e < 16; e += 8) {
                            const uint4 y = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
                            const uint4 z = make_uint4(w[e + 4], w[e + 5], w[e + 6], w[e + 7]);
                            if (v8) {
                                st_global_v8(dst + 16 * c + e, y, z);
                            } else {
                                *reinterpret_cast<uint4 *>(dst + 16 * c + e) = y;
                                *reinterpret_cast<uint4 *>(dst + 16 * c + e + 4) = z;
                            }
                        }
                    }
                    if (last && !FOLD) {
                        named_barrier(2, 128);
#pragma unroll
                        for (int e = 0; e < PER; ++e) {
                            float ya = 0.f, yb = 0.f;
#pragma unroll
                            for (int k = 0; k < TOK; ++k) {
                                const int r = k * G + h0 + e;
                                ya += tp[r * 17 + col];
                                yb += tp[(C::ROWS + r) * 17 + col];
                            }
                            sa[c][e] += ya;
                            sb[c][e] += yb;
                        }
                        named_barrier(2, 128);  // the buffer may be written again
                    }
                }
            }
        }
        if (ok && cur_g >= 0)
            flush(cur_g);
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
}

template <int D, int G>
cudaError_t launch_dq(const SinkDqMaps &maps, const SinkBwdParams &p, cudaStream_t stream)
{
    using C = SqCfg<D>;
    auto kern = sink_dq_tc_kernel<D, G>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess)
        return e;
    constexpr int TOK = C::ROWS / G;
    const long long tiles = static_cast<long long>(p.B) * p.Hkv * ((p.T + TOK - 1) / TOK);
    return launch_dependent(kern, dim3(static_cast<unsigned>(tiles < 152 ? tiles : 152)), C::THREADS, C::SMEM, stream, maps, p);
}

}  // namespace

cudaError_t launch_sink_dq(int D, const SinkDqMaps &maps, const SinkBwdParams &p, cudaStream_t stream)
{
    const int G = p.Hq / p.Hkv;
#define ORTHROS_DQ_CASE(DD, GG) \
    if (D == DD && G == GG)     \
        return launch_dq<DD, GG>(maps, p, stream);
    ORTHROS_DQ_CASE(128, 1)
    ORTHROS_DQ_CASE(128, 2)
    ORTHROS_DQ_CASE(128, 4)
    ORTHROS_DQ_CASE(128, 8)
    ORTHROS_DQ_CASE(128, 16)
    ORTHROS_DQ_CASE(64, 1)
    ORTHROS_DQ_CASE(64, 2)
    ORTHROS_DQ_CASE(64, 4)
    ORTHROS_DQ_CASE(64, 8)
    ORTHROS_DQ_CASE(64, 16)
#undef ORTHROS_DQ_CASE
    return cudaErrorInvalidValue;
}

}  // namespace orthros
