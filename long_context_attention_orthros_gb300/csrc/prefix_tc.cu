// prefix_tc.cu -- attention of every query row of a batch over one shared prompt prefix on the
// 5th-generation tensor cores (tcgen05 + tensor memory): the form of prefix_attn.cu for more rows
// than its warp MMAs keep up with.  Rows, partials and slots are those of prefix_attn.cu.
//
// A CTA takes a range of the prefix's keys and runs two softmax streams over it, so that one
// stream's MMAs run while the other's exponentials do:
//   ROWS2: tiles of 128 rows each, A and B; every pair of 64-key blocks serves both (R > 128);
//   KEYS2: one tile of 128 rows; the streams take pairs of key blocks in turn, each with its own
//          maximum, sum and O (its own partial), and the ring is one pair deeper;
//   DIRECT: as ROWS2 on two tiles of one sequence's rows, over the whole prefix and then the
//          sequence's own rows up to each copy's position, and o' leaves rounded to bf16.
// Per pair of blocks (128 keys) and stream:
//   S = q K^T   one N = 128 product per 16 of d, fp16, fp32 accumulators in tensor memory.  A q row is
//               scaled by a power of two to a largest value in [2^14, 2^15) before it is rounded (the
//               factor comes back in the exponent's FMA); K is converted from bf16 in shared memory,
//               a key row whose largest |k| reaches 65520, or lies below 2^-9, by an exact 2^-e
//               first and its logits multiplied back by 2^e;
//   softmax     a thread a row; the running maximum is raised only when it grows by more than 8
//               (log2 units); P <= 256 as bf16 over S;
//   O += P V    bf16, fp32 accumulators in tensor memory.
// At the end (but for DIRECT) O, the maximum and the sum leave as the stream's partial, unnormalised.
//
// Bound by HBM where the rows are few (8 sequences over 131072 rows, 32/8 heads, d = 128: 85 us, 6.3 TB/s,
// and 14 for its start and the own rows), by a stream's chain of S, softmax and P V where they fill
// the tile (4 x 256 copies: 308 us, 920 TFLOP/s; 305 without the look for small key rows).
//
// Roles (512 threads, one CTA an SM):
//   warps 0, 3    TMA producers of K and of V
//   warps 1, 2    lane 0 issues every tcgen05.mma of stream 0, of stream 1; warp 1 allocates tensor
//                 memory.  One thread for both streams spends 2850 cycles a pair of blocks issuing and
//                 1000 on waits that are over, more than the MMAs take
//   warps 12-15   convert each landed K block to fp16
//   warps 4-7     queries from global memory to fp16 tiles (with warps 8-11), then softmax and
//                 partial of stream 0; a warp without a row only keeps step
//   warps 8-11    the same for stream 1.  The streams' softmaxes take turns, warp by warp: left alone
//                 they run side by side, at half the rate, and the MMAs of both wait for them
// 4 x 256 copies of 32 heads over 16384 keys (d = 128): one issuer 328 us, two 393, two and turns 305; P V
// in two halves, the first beside the second half's exponentials: 309 (not kept).
// Tensor memory: S of stream t at 128 t; O at 256 + D t.  Every mbarrier wait is bounded; a timeout
// records ORTHROS_DEVERR_TIMEOUT and all roles drain to the common exit.
#include <cuda_fp16.h>

#include "prefix_rows.cuh"
#include "serve.cuh"
#include "tc.cuh"

namespace orthros {

enum { PT_KEYS2 = 0, PT_ROWS2 = 1, PT_DIRECT = 2 };

template <int D, int MODE>
struct PtCfg {
    static constexpr bool ROWS2 = MODE != PT_KEYS2;
    static constexpr int KB = 64;
    static constexpr int SLABS = D / 64;
    static constexpr int TILES = ROWS2 ? 2 : 1;
    static constexpr int Q_SLAB = 128 * 128;
    static constexpr int Q_BYTES = SLABS * Q_SLAB;
    static constexpr int PAIR_SLAB = 128 * 128;             // 128 keys of one 64-wide slab
    static constexpr int PAIR_BYTES = SLABS * PAIR_SLAB;    // K, or V, of a pair
    static constexpr int PAIRS = ROWS2 ? 2 : 3;
    static constexpr int SLOTS = 2 * PAIRS;                 // 64-key blocks of the ring
    static constexpr int K_OFF = 0;
    static constexpr int V_OFF = PAIRS * PAIR_BYTES;
    static constexpr int Q_OFF = 2 * PAIRS * PAIR_BYTES;
    // Marks of a block's conversion live two rounds of the ring: K is released when its S are complete,
    // before the softmax has read them, and the block two rounds later is converted after it has.
    static constexpr int MARKS = 2 * SLOTS;
    static constexpr int KEXP_OFF = Q_OFF + TILES * Q_BYTES;   // int8 [MARKS][KB]: key row shift
    static constexpr int KFLAG_OFF = KEXP_OFF + MARKS * KB;    // uint8 [MARKS][8]
    static constexpr int QSC_OFF = KFLAG_OFF + MARKS * 8;      // int8 [TILES][128]: query row shift
    static constexpr int BAR_OFF = QSC_OFF + TILES * 128;
    static constexpr int MPAIRS = 2 * PAIRS;  // an even number: a mark of a pair belongs to one stream for good
    static constexpr int NBARS = SLOTS + MARKS + MPAIRS + 2 * PAIRS + 18;
    static constexpr int HOLD_OFF = BAR_OFF + NBARS * 8;
    static constexpr int USED = HOLD_OFF + 16 + 1024;
    static constexpr int SMEM = USED > 120 * 1024 ? USED : 120 * 1024;  // one CTA an SM: it takes all of tensor memory
    static_assert(SMEM <= 232448, "shared memory budget");
    static constexpr uint32_t TM_S = 0, TM_O = 256;
    static constexpr int CPR = D / 8;       // 16-byte chunks of a query row
    static constexpr int RPP = 256 / CPR;   // rows one pass of the softmax warps' 256 threads covers
    static constexpr int CONV_THREADS = 128;
};

template <int D, int G, int MODE>
__global__ void __launch_bounds__(512, 1)
    prefix_tc_kernel(const __grid_constant__ PrefixMaps maps, const PrefixAttnParams p)
{
    using C = PtCfg<D, MODE>;
    constexpr bool ROWS2 = C::ROWS2, DIRECT = MODE == PT_DIRECT;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_s = smem_u32(smem_raw);
    const uint32_t pad = ((raw_s + 1023u) & ~1023u) - raw_s;
    uint8_t *smem = smem_raw + pad;
    const uint32_t sbase = raw_s + pad;
    uint64_t *kfull = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);  // [SLOTS] K block landed
    uint64_t *kconv = kfull + C::SLOTS;    // [MARKS] K block converted
    uint64_t *vfull = kconv + C::MARKS;    // [MPAIRS] V of a pair landed
    uint64_t *kempty = vfull + C::MPAIRS;  // [PAIRS] K of a pair released: its S are complete (MMA commit)
    uint64_t *vempty = kempty + C::PAIRS;  // [PAIRS] V released: its P V are complete
    uint64_t *q_full = vempty + C::PAIRS;  // [2] query tile prepared
    uint64_t *s_full = q_full + 2;         // [2] S of a pair complete
    uint64_t *p_full = s_full + 2;         // [2] P written
    uint64_t *o_done = p_full + 2;         // [2] O += P V of a pair complete, but the last
    uint64_t *o_final = o_done + 2;        // [2] of the stream's last pair
    uint64_t *turn = o_final + 2;          // [2][4] a softmax warp of the stream is done with a pair
    int8_t *kexp = reinterpret_cast<int8_t *>(smem + C::KEXP_OFF);
    int8_t *qexp = reinterpret_cast<int8_t *>(smem + C::QSC_OFF);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + C::HOLD_OFF);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = blockIdx.x, g = blockIdx.y;
    // rows row_base .. of a KV head, up to row_end: of the whole batch, or (DIRECT) of one sequence
    const long long R = static_cast<long long>(p.B) * p.T_out * G;
    const int seq_tiles = DIRECT ? gridDim.z / p.B : 1, b_own = DIRECT ? blockIdx.z / seq_tiles : 0;
    const long long row_base =
        DIRECT ? static_cast<long long>(b_own) * p.T_out * G + static_cast<long long>(blockIdx.z % seq_tiles) * 256
               : static_cast<long long>(blockIdx.z) * 128 * C::TILES;
    const long long row_end = DIRECT ? static_cast<long long>(b_own + 1) * p.T_out * G : R;
    __shared__ volatile int s_abort;  // a wait has given up: the producer stops
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int s = 0; s < C::SLOTS; ++s)
            mbar_init(&kfull[s], 1);
        for (int s = 0; s < C::MPAIRS; ++s)
            mbar_init(&vfull[s], 1);
        for (int s = 0; s < C::MARKS; ++s) {
            mbar_init(&kconv[s], C::CONV_THREADS / 32);
            reinterpret_cast<uint64_t *>(smem + C::KFLAG_OFF)[s] = 0;
        }
        for (int s = 0; s < C::PAIRS; ++s) {
            mbar_init(&kempty[s], C::TILES);  // a commit of each stream that reads the pair
            mbar_init(&vempty[s], C::TILES);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&q_full[t], 8);
            mbar_init(&s_full[t], 1);
            mbar_init(&p_full[t], 4);
            mbar_init(&o_done[t], 1);
            mbar_init(&o_final[t], 1);
        }
        for (int i = 0; i < 8; ++i)
            mbar_init(&turn[i], 1);
        fence_barrier_init();
    }
    if (warp == 1)
        tmem_alloc(tmem_holder, 512);
    tc_fence_before();
    // the queries' and the scale-offset's lines on their way to L2 (no value is read yet)
    if (threadIdx.x >= 128 && threadIdx.x < 256) {
        for (int i = threadIdx.x - 128; i < G * D / 32; i += 128) {
            prefetch_l2(p.alpha_c + g * G * D + 32 * i);
            prefetch_l2(p.beta_c + g * G * D + 32 * i);
        }
    } else if (threadIdx.x >= 256 && !DIRECT) {
        for (int i = threadIdx.x - 256; i < 128 * C::TILES; i += 256) {
            const long long ri = row_base + i;
            if (ri < R) {
                const uint32_t bi = static_cast<uint32_t>(ri) / G, b = bi / static_cast<uint32_t>(p.T_out);
                const orthros_bf16 *q = p.qc + b * p.qc_bstride +
                                        (static_cast<long long>(bi - b * p.T_out) * p.Hq + g * G + static_cast<uint32_t>(ri) % G) * D;
                prefetch_l2(q);
                if (D == 128)
                    prefetch_l2(q + 64);
            }
        }
    }
    // what the kernels before wrote first, then a dependent grid may start beside this one
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (p.clear != nullptr && blockIdx.x + blockIdx.y + blockIdx.z == 0)
        for (int i = threadIdx.x; i < p.n_clear; i += blockDim.x)
            p.clear[i] = 0;
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_holder;
    const int js = DIRECT ? 0 : split * p.chunk, je = DIRECT ? p.P : min(js + p.chunk, p.P);
    const int nkb = (je - js + C::KB - 1) / C::KB;  // at least 1: the plan has no empty split
    const int pre_blocks = (nkb + 1) / 2 * 2;        // whole pairs
    // DIRECT: the sequence's own keys up to the largest position among the rows follow
    int kmax = -1;
    if constexpr (DIRECT) {
        __shared__ int kmax_s;
        if (threadIdx.x == 0)
            kmax_s = -1;
        __syncthreads();
        if (threadIdx.x < 256 && row_base + threadIdx.x < row_end) {
            const int pos = p.pos[static_cast<uint32_t>(row_base + threadIdx.x) / G];
            if (pos >= 0 && pos < p.T_kv)
                atomicMax(&kmax_s, pos);
            else if ((row_base + threadIdx.x) % G == 0)
                record_error(p.dev_err, ORTHROS_DEVERR_POSITION);
        }
        __syncthreads();
        kmax = kmax_s;
    }
    const int npair = pre_blocks / 2 + (DIRECT ? (kmax + 2 * C::KB) / (2 * C::KB) : 0);
    auto pairs_of = [&](int t) { return ROWS2 ? npair : (npair - t + 1) / 2; };  // of stream t
    auto pair_at = [&](int t, int u) { return ROWS2 ? u : 2 * u + t; };           // its u-th

    if (warp == 0 || warp == 3) {
        // ------------------------------------------------------------------ producers of K, of V
        if (lane == 0) {
            const bool kv = warp == 3;
            tma_prefetch_desc(kv ? &maps.v : &maps.k);
            for (int pp = 0; pp < npair; ++pp) {
                const int ps = pp % C::PAIRS;
                if ((pp >= C::PAIRS &&
                     !mbar_wait(kv ? &vempty[ps] : &kempty[ps], static_cast<uint32_t>((pp / C::PAIRS - 1) & 1))) ||
                    s_abort) {
                    record_error(p.dev_err, ORTHROS_DEVERR_TIMEOUT);
                    s_abort = 1;
                    break;
                }
                constexpr int BYTES = C::SLABS * C::KB * 128;
                if (kv)
                    mbar_arrive_expect_tx(&vfull[pp % C::MPAIRS], 2 * BYTES);
                for (int h = 0; h < 2; ++h) {
                    const int j = 2 * pp + h;
                    uint64_t *bar = kv ? &vfull[pp % C::MPAIRS] : &kfull[2 * ps + h];
                    uint8_t *dst = smem + (kv ? C::V_OFF : C::K_OFF) + ps * C::PAIR_BYTES + h * C::KB * 128;
                    const bool own = DIRECT && j >= pre_blocks;
                    const CUtensorMap *map = own ? (kv ? &maps.vo : &maps.ko) : (kv ? &maps.v : &maps.k);
                    const int j0 = own ? (j - pre_blocks) * C::KB : js + j * C::KB;
                    if (!kv)
                        mbar_arrive_expect_tx(bar, BYTES);
#pragma unroll
                    for (int sl = 0; sl < C::SLABS; ++sl)
                        tma_load_4d(dst + sl * C::PAIR_SLAB, map, bar, sl * 64, g, j0, own ? b_own : 0);
                }
            }
        }
    } else if (warp < 3) {
        // ------------------------------------------------------------------ MMA issuer of stream t
        if (lane == 0) {
            constexpr uint32_t IDESC_QK = umma_idesc(128, 128, false, false);
            constexpr uint32_t IDESC_PV = umma_idesc(128, D, true, true);
            const int t = warp - 1, nu = pairs_of(t);
            const uint32_t s_tm = tbase + C::TM_S + 128 * t, o_tm = tbase + C::TM_O + D * t;
            const uint64_t qdesc = umma_desc_sw128(sbase + C::Q_OFF + (ROWS2 ? t : 0) * C::Q_BYTES, 16, 1024);
            const uint64_t kdesc0 = umma_desc_sw128(sbase + C::K_OFF, 16, 1024);
            const uint64_t vdesc0 = umma_desc_sw128(sbase + C::V_OFF, C::PAIR_SLAB, 1024);
            auto issue_s = [&](int u) -> bool {
                const int pp = pair_at(t, u), ps = pp % C::PAIRS, j = 2 * pp + 1;
                // converted (every converter warp is done with the pair's first block before its second);
                // S overwrites the P that the stream's last P V reads
                if (!mbar_wait(&kconv[j % C::MARKS], static_cast<uint32_t>((j / C::MARKS) & 1)) ||
                    (u >= 1 && !mbar_wait(&o_done[t], static_cast<uint32_t>((u - 1) & 1))))
                    return false;
                tc_fence_after();
                const uint64_t kdesc = kdesc0 + static_cast<uint64_t>(ps * (C::PAIR_BYTES >> 4));
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = static_cast<uint32_t>((kk >> 2) * C::PAIR_SLAB + (kk & 3) * 32) >> 4;
                    static_assert(C::PAIR_SLAB == C::Q_SLAB, "one offset serves both operands");
                    umma_ss(s_tm, qdesc + off, kdesc + off, IDESC_QK, kk != 0);
                }
                umma_commit(&s_full[t]);
                if (pp + C::PAIRS < npair)     // the producer waits for it
                    umma_commit(&kempty[ps]);  // this stream's part of the pair's K
                return true;
            };
            auto issue_pv = [&](int u) -> bool {
                const int pp = pair_at(t, u), ps = pp % C::PAIRS;
                if (!mbar_wait(&vfull[pp % C::MPAIRS], static_cast<uint32_t>((pp / C::MPAIRS) & 1)) ||
                    !mbar_wait(&p_full[t], static_cast<uint32_t>(u & 1)))
                    return false;
                tc_fence_after();
                const uint64_t vdesc = vdesc0 + static_cast<uint64_t>(ps * (C::PAIR_BYTES >> 4));
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    umma_ts(o_tm, s_tm + 8 * kk, vdesc + static_cast<uint64_t>(kk * (2048 >> 4)), IDESC_PV,
                            (u > 0 || kk > 0) ? 1u : 0u);
                umma_commit(u == nu - 1 ? &o_final[t] : &o_done[t]);
                if (pp + C::PAIRS < npair)
                    umma_commit(&vempty[ps]);  // the same for its V
                return true;
            };
            bool ok = nu == 0 || (mbar_wait(&q_full[ROWS2 ? t : 0], 0) && issue_s(0));
            for (int u = 0; u < nu && ok; ++u)
                ok = issue_pv(u) && (u + 1 >= nu || issue_s(u + 1));
            // A stream whose tile has no row: nothing else waits for its last P V before shared and tensor
            // memory are given back.  All other commits have been waited for.
            if (ok && nu > 0)
                ok = mbar_wait(&o_final[t], 0);
            if (!ok) {
                s_abort = 1;
                record_error(p.dev_err, ORTHROS_DEVERR_TIMEOUT);
            }
        }
    } else if (warp >= 12) {
        // ------------------------------------------------------------------ K converters
        bool ok = true, bad = false;
        // K conversion: 8 consecutive lanes a key row, rows cid / 8 + STEP it of a block
        constexpr int STEP = C::CONV_THREADS / 8;
        const int cid = threadIdx.x - 384;
        const int cw = cid >> 5;
        constexpr int ITS = C::KB / STEP;
        static_assert(C::KB % STEP == 0, "a thread's rows are all in the block");
        for (int j = 0; j < 2 * npair && ok; ++j) {
            const int s = j % C::SLOTS;
            if (!(ok = mbar_wait(&kfull[s], static_cast<uint32_t>((j / C::SLOTS) & 1))))
                break;
            uint8_t *blk = smem + C::K_OFF + (s / 2) * C::PAIR_BYTES + (s % 2) * C::KB * 128;
            // DIRECT: own rows from this one on lie behind every copy's position: they have no weight, but may
            // hold anything, and become zeros before they are looked at
            const int beyond = DIRECT && j >= pre_blocks ? kmax + 1 - (j - pre_blocks) * C::KB : C::KB;
            if (DIRECT && beyond < C::KB)
                for (int r = cid >> 3; r < C::KB; r += STEP)
                    if (r >= beyond)
#pragma unroll
                        for (int sl = 0; sl < C::SLABS; ++sl)
                            *reinterpret_cast<uint4 *>(blk + sl * C::PAIR_SLAB + r * 128 + (cid & 7) * 16) = make_uint4(0, 0, 0, 0);
            uint4 u[ITS][C::SLABS];
            float most = 0.f, least = kSmallKey;  // of this lane's part of each row its largest |k|: the extremes
            float row_max[ITS];
#pragma unroll
            for (int it = 0; it < ITS; ++it) {
                row_max[it] = 0.f;
#pragma unroll
                for (int sl = 0; sl < C::SLABS; ++sl) {
                    u[it][sl] = *reinterpret_cast<const uint4 *>(blk + sl * C::PAIR_SLAB + ((cid >> 3) + STEP * it) * 128 +
                                                                 (cid & 7) * 16);
                    row_max[it] = fmaxf(row_max[it], bf16x8_absmax(u[it][sl]));
                }
                most = fmaxf(most, row_max[it]);
                least = fminf(least, row_max[it]);
            }
            bool wany = __any_sync(0xffffffffu, !(most < 65520.f) || least < kSmallKey);
            if (wany && !__any_sync(0xffffffffu, !(most < 65520.f))) {  // is a whole row (8 lanes) small, and not zero?
                wany = false;
#pragma unroll
                for (int it = 0; it < ITS; ++it) {
                    const uint32_t row = 0xffu << (lane & 24);
                    const uint32_t below = __ballot_sync(0xffffffffu, row_max[it] < kSmallKey) & row;
                    const uint32_t some = __ballot_sync(0xffffffffu, row_max[it] > 0.f) & row;
                    wany |= __any_sync(0xffffffffu, below == row && some != 0);
                }
            }
            if (!wany) {
#pragma unroll
                for (int it = 0; it < ITS; ++it)
#pragma unroll
                    for (int sl = 0; sl < C::SLABS; ++sl)
                        *reinterpret_cast<uint4 *>(blk + sl * C::PAIR_SLAB + ((cid >> 3) + STEP * it) * 128 + (cid & 7) * 16) =
                            k_to_fp16(u[it][sl]);
            } else {
                shift_key_rows<C::SLABS, true>(blk, C::PAIR_SLAB, 0, cid >> 3, STEP, ITS, cid & 7,
                                               kexp + (j % C::MARKS) * C::KB, bad);
            }
            if constexpr (DIRECT) {
                if (beyond < C::KB) {  // the same for V
                    if (!(ok = mbar_wait(&vfull[j / 2 % C::MPAIRS], static_cast<uint32_t>((j / 2 / C::MPAIRS) & 1))))
                        break;
                    for (int it = 0; it < ITS; ++it) {
                        const int r = (cid >> 3) + STEP * it;
                        if (r >= beyond)
#pragma unroll
                            for (int sl = 0; sl < C::SLABS; ++sl)
                                *reinterpret_cast<uint4 *>(blk + (C::V_OFF - C::K_OFF) + sl * C::PAIR_SLAB + r * 128 +
                                                           (cid & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
            }
            if (lane == 0)
                smem[C::KFLAG_OFF + (j % C::MARKS) * 8 + cw] = wany ? 1 : 0;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&kconv[j % C::MARKS]);
        }
        if (bad)
            record_error(p.dev_err, ORTHROS_DEVERR_RANGE);
        if (!ok) {
            s_abort = 1;
            if (lane == 0)
                record_error(p.dev_err, ORTHROS_DEVERR_TIMEOUT);
        }
    } else {
        // ------------------------------------------------------------------ softmax + partials
        // first the queries, from global memory to fp16 tiles, by all eight warps: a thread has 16 bytes of
        // every RPP-th row, all of one head, and its rows' loads are in flight together
        {
            const int tid = threadIdx.x - 128;  // 0 .. 255
            const int cr = tid % C::CPR, r0 = tid / C::CPR;
            constexpr int ROWS = 128 / C::RPP;
            static_assert(C::RPP % G == 0, "a thread's rows share a head");
            const int h = g * G + r0 % G;
            float al[8], be[8];
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const float4 y = __ldg(reinterpret_cast<const float4 *>(p.alpha_c + h * D + 8 * cr + e));
                const float4 z = __ldg(reinterpret_cast<const float4 *>(p.beta_c + h * D + 8 * cr + e));
                al[e] = y.x * p.qscale, al[e + 1] = y.y * p.qscale, al[e + 2] = y.z * p.qscale, al[e + 3] = y.w * p.qscale;
                be[e] = z.x * p.qscale, be[e + 1] = z.y * p.qscale, be[e + 2] = z.z * p.qscale, be[e + 3] = z.w * p.qscale;
            }
#pragma unroll
            for (int tl = 0; tl < C::TILES; ++tl) {
                uint8_t *qb = smem + C::Q_OFF + tl * C::Q_BYTES + (cr / 8) * C::Q_SLAB;
                // the raw rows go straight to their places in the tile, all of a thread's in flight, and are
                // turned into fp16 there (short code: the whole kernel is fetched anew at every launch)
                uint32_t have = 0;
#pragma unroll
                for (int x = 0; x < ROWS; ++x) {
                    const int r = r0 + x * C::RPP;
                    const long long ri = row_base + tl * 128 + r;
                    const PrefixRow row = prefix_row<G>(p, ri < row_end ? ri : R, g, D);
                    if (row.q != nullptr) {
                        cp_async16(qb + sw128_offset(r, cr % 8), row.q + 8 * cr);
                        have |= 1u << x;
                    }
                }
                cp_async_wait_all();
#pragma unroll 2
                for (int x = 0; x < ROWS; ++x) {
                    const int r = r0 + x * C::RPP;
                    uint4 *slot = reinterpret_cast<uint4 *>(qb + sw128_offset(r, cr % 8));
                    const uint4 raw = (have >> x) & 1u ? *slot : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
                    float f[8], amax = 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 y = ffma2(unpack_bf16x2(w[e]), make_float2(al[2 * e], al[2 * e + 1]),
                                               make_float2(be[2 * e], be[2 * e + 1]));
                        f[2 * e] = (have >> x) & 1u ? y.x : 0.f;
                        f[2 * e + 1] = (have >> x) & 1u ? y.y : 0.f;
                        amax = fmax3(amax, fabsf(f[2 * e]), fabsf(f[2 * e + 1]));
                    }
#pragma unroll
                    for (int off = 1; off < C::CPR; off <<= 1)
                        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
                    int sh = static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 14;
                    sh = amax == 0.f ? 0 : (sh < -126 ? -126 : sh);
                    const float sd = exp2i(-sh);
                    uint32_t o4[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const __half2 hv = __floats2half2_rn(f[2 * e] * sd, f[2 * e + 1] * sd);
                        o4[e] = *reinterpret_cast<const uint32_t *>(&hv);
                    }
                    *slot = make_uint4(o4[0], o4[1], o4[2], o4[3]);
                    if (cr == 0)
                        qexp[tl * 128 + r] = static_cast<int8_t>(sh);
                }
                fence_proxy_async_smem();  // the MMA reads q through the async proxy
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&q_full[tl]);
            }
        }
        const int t = (warp - 4) >> 2;  // stream
        const int tile = ROWS2 ? t : 0, rw = warp & 3, r = rw * 32 + lane;
        const long long row_i = row_base + tile * 128 + r;
        const bool work = row_base + tile * 128 + rw * 32 < row_end;  // the warp has a row
        const PrefixRow row = prefix_row<G>(p, row_i < row_end ? row_i : R, g, D);
        // the row's last own key; without a position none, and its results are not used
        const int pos = DIRECT && row.q != nullptr ? p.pos[static_cast<uint32_t>(row_i) / G] : -1;
        const uint32_t s_lane = tbase + (static_cast<uint32_t>(rw * 32) << 16) + C::TM_S + 128 * t;
        const uint32_t o_col = tbase + (static_cast<uint32_t>(rw * 32) << 16) + C::TM_O + D * t;
        const float NEG_INF = -__int_as_float(0x7f800000);
        const int nu = pairs_of(t);
        bool ok = mbar_wait(&q_full[tile], 0), range_bad = false;
        const float qf = exp2i(qexp[tile * 128 + r]);  // logit = S qf
        const float2 qf2 = make_float2(qf, qf);
        float m = NEG_INF, l = 0.f;
        for (int u = 0; u < nu && ok; ++u) {
            const int pp = pair_at(t, u);
            if (!(ok = mbar_wait(&s_full[t], static_cast<uint32_t>(u & 1)) &&
                       (t + u == 0 || mbar_wait(&turn[4 * (1 - t) + rw], static_cast<uint32_t>((t == 0 ? u - 1 : u) & 1)))))
                break;
            tc_fence_after();
            if (work) {
                float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
                for (int hh = 0; hh < 2 && ok; ++hh) {
                    const int j = 2 * pp + hh, ks = j % C::MARKS;
                    const uint32_t s_col = s_lane + 64 * hh;
                    // column c is a key iff c <= nvalid
                    const int nvalid = DIRECT && j >= pre_blocks ? pos - (j - pre_blocks) * C::KB : je - 1 - (js + j * C::KB);
                    uint32_t va[32], vb[32];
                    tmem_ld32(s_col, va);
                    tmem_ld32(s_col + 32, vb);
                    // the block's conversion completed before its S was issued: this test succeeds and
                    // orders the flag read after the converters' writes
                    const uint32_t kph = static_cast<uint32_t>((j / C::MARKS) & 1);
                    const bool seen = mbar_test_wait(&kconv[ks], kph);
                    const uint64_t kf = *reinterpret_cast<const volatile uint64_t *>(smem + C::KFLAG_OFF + ks * 8);
                    tmem_wait_ld();
                    if (!seen || kf != 0) {
                        if (!(ok = mbar_wait(&kconv[ks], kph)))
                            break;
                        const uint64_t kf2 = *reinterpret_cast<const volatile uint64_t *>(smem + C::KFLAG_OFF + ks * 8);
                        uint32_t kw = 0;
#pragma unroll
                        for (int cw = 0; cw < C::CONV_THREADS / 32; ++cw)
                            kw |= (((kf2 >> (8 * cw)) & 0xffu) ? 1u : 0u) << cw;
                        if (kw != 0) {  // logits of shifted key rows times 2^e (rare), in tensor memory
                            unshift_chunk32(s_col, kexp + ks * C::KB, 0, kw, C::CONV_THREADS / 8, 4, range_bad, nvalid);
                            unshift_chunk32(s_col + 32, kexp + ks * C::KB, 32, kw, C::CONV_THREADS / 8, 4, range_bad, nvalid - 32);
                            tmem_ld32(s_col, va);
                            tmem_ld32(s_col + 32, vb);
                            tmem_wait_ld();
                        }
                    }
                    if (nvalid < C::KB - 1) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            if (e > nvalid)
                                va[e] = __float_as_uint(NEG_INF);
                            if (32 + e > nvalid)
                                vb[e] = __float_as_uint(NEG_INF);
                        }
                    }
                    float m4[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        m4[(e >> 1) & 3] = fmax3(m4[(e >> 1) & 3], __uint_as_float(va[e]), __uint_as_float(va[e + 1]));
                        m4[(e >> 1) & 3] = fmax3(m4[(e >> 1) & 3], __uint_as_float(vb[e]), __uint_as_float(vb[e + 1]));
                    }
                    const float mb = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * qf;
                    const bool raise = mb > m + 8.f;
                    if (__any_sync(0xffffffffu, raise)) {
                        const float f = raise ? fast_exp2(m - mb) : 1.f;  // m = -inf before the first key: 0
                        if (u > 0) {
                            // O holds the stream's pairs before u: their P V completed before S of u was issued
                            if (!(ok = mbar_wait(&o_done[t], static_cast<uint32_t>((u - 1) & 1))))
                                break;
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D; c += 32) {
                                uint32_t w[32];
                                tmem_ld32(o_col + c, w);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    w[e] = __float_as_uint(__uint_as_float(w[e]) * f);
                                tmem_st32(o_col + c, w);
                            }
                        }
                        if (hh == 1) {  // P of the first half was taken against the old maximum
                            tmem_wait_st();
                            uint32_t w[32];
                            tmem_ld32(s_lane, w);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const float2 pq = unpack_bf16x2(w[e]);
                                w[e] = pack_bf16x2(pq.x * f, pq.y * f);
                            }
                            tmem_st32(s_lane, w);
                            l2[0].x *= f;
                            l2[0].y *= f;
                            l2[1].x *= f;
                            l2[1].y *= f;
                        }
                        if (raise) {
                            l *= f;
                            m = mb;
                        }
                    }
                    const float uo = m == NEG_INF ? 0.f : m;
                    const float2 nm = make_float2(-uo, -uo);
#pragma unroll
                    for (int hq = 0; hq < 2; ++hq) {
                        const uint32_t *v = hq ? vb : va;
                        uint32_t pw[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float2 d = ffma2(make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), qf2, nm);
                            const float2 y = make_float2(fast_exp2(d.x), fast_exp2(d.y));
                            l2[e & 1] = fadd2(l2[e & 1], y);
                            pw[e] = pack_bf16x2(y.x, y.y);
                        }
                        tmem_st16(s_lane + 32 * hh + 16 * hq, pw);
                    }
                }
                if (!ok)
                    break;
                l += (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&p_full[t]);
                mbar_arrive(&turn[4 * t + rw]);
            }
        }
        // ---- the stream's partial: a thread a row
        if (ok && work) {
            const bool store = row.slot >= 0, valid = row.q != nullptr && nu > 0;
            const long long part = ROWS2 ? split : 2 * split + t;
            const long long slot = part * R * p.Hkv + row.slot;
            if (!DIRECT && store)
                p.part_ml[slot] = valid ? make_float2(m, l) : make_float2(NEG_INF, 0.f);
            const float inv = l > 0.f ? 1.f / l : 0.f;
            const uint32_t i_own = DIRECT ? static_cast<uint32_t>(row_i - static_cast<long long>(b_own) * p.T_out * G) / G : 0;
            orthros_bf16 *orow =
                DIRECT ? p.oc + b_own * p.oc_bstride + (static_cast<long long>(i_own) * p.Hq + row.head) * D : nullptr;
            if (nu > 0 && !(ok = mbar_wait(&o_final[t], 0)))
                record_error(p.dev_err, ORTHROS_DEVERR_TIMEOUT);
            if (ok) {
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t v[32];
                    if (nu > 0) {
                        tmem_ld32(o_col + c, v);
                        tmem_wait_ld();
                    }
                    if (store) {
                        if constexpr (DIRECT) {
#pragma unroll
                            for (int e = 0; e < 32; e += 8) {
                                uint32_t w[4];
#pragma unroll
                                for (int x = 0; x < 4; ++x)
                                    w[x] = valid ? pack_bf16x2(__uint_as_float(v[e + 2 * x]) * inv,
                                                               __uint_as_float(v[e + 2 * x + 1]) * inv) : 0u;
                                *reinterpret_cast<uint4 *>(orow + c + e) = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; e += 8) {
                                const uint4 a = valid ? make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]) : make_uint4(0, 0, 0, 0);
                                const uint4 b = valid ? make_uint4(v[e + 4], v[e + 5], v[e + 6], v[e + 7]) : make_uint4(0, 0, 0, 0);
                                st_global_v8(p.part_o + slot * D + c + e, a, b);
                            }
                        }
                    }
                }
            }
        }
        if (range_bad)
            record_error(p.dev_err, ORTHROS_DEVERR_RANGE);
        if (!ok) {
            s_abort = 1;
            if (lane == 0)
                record_error(p.dev_err, ORTHROS_DEVERR_TIMEOUT);
        }
    }

    // ---------------------------------------------------------------------- teardown
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

template <int D, int G, int MODE>
static cudaError_t launch_ptc(const PrefixMaps &maps, const PrefixAttnParams &p, int splits, int tiles,
                              cudaStream_t stream)
{
    using C = PtCfg<D, MODE>;
    auto kern = prefix_tc_kernel<D, G, MODE>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(splits, p.Hkv, tiles);
    cfg.blockDim = dim3(512);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, maps, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

template <int D, int G>
static cudaError_t launch_ptc_mode(int mode, const PrefixMaps &maps, const PrefixAttnParams &p, int splits, int tiles,
                                   cudaStream_t stream)
{
    return mode == PT_KEYS2   ? launch_ptc<D, G, PT_KEYS2>(maps, p, splits, tiles, stream)
           : mode == PT_ROWS2 ? launch_ptc<D, G, PT_ROWS2>(maps, p, splits, tiles, stream)
                              : launch_ptc<D, G, PT_DIRECT>(maps, p, 1, tiles, stream);
}

cudaError_t launch_prefix_tc(int D, int mode, const PrefixMaps &maps, const PrefixAttnParams &p, int splits, int tiles,
                             cudaStream_t stream)
{
    const int G = p.Hq / p.Hkv;
#define ORTHROS_PTC_CASE(DD, GG) \
    if (D == DD && G == GG)      \
        return launch_ptc_mode<DD, GG>(mode, maps, p, splits, tiles, stream);
    ORTHROS_PTC_CASE(128, 1)
    ORTHROS_PTC_CASE(128, 2)
    ORTHROS_PTC_CASE(128, 4)
    ORTHROS_PTC_CASE(128, 8)
    ORTHROS_PTC_CASE(128, 16)
    ORTHROS_PTC_CASE(64, 1)
    ORTHROS_PTC_CASE(64, 2)
    ORTHROS_PTC_CASE(64, 4)
    ORTHROS_PTC_CASE(64, 8)
    ORTHROS_PTC_CASE(64, 16)
#undef ORTHROS_PTC_CASE
    return cudaErrorInvalidValue;
}

// Prefix and own rows in one pass (tiles of 256 rows of one sequence, one launch, no partials) or the
// prefix split over all SMs, the own rows by warp MMAs and a join?  The first takes 2.1 us for every
// 128 keys one CTA runs over (in as many waves as 152 SMs need) and 9 us around them; the second 20 us
// for its three launches, 2 ns a row to join, the prefix's tiles shared out evenly and the own rows at
// some 210 TFLOP/s.  Measured on a GB300 (split, direct, us): 3 x 37 copies over 617 + 1457 keys, G = 1:
// 26, 40; 2 x 24 over 53852 + 548, G = 2: 60, 926; 10 x 52 over 920 + 2, G = 4: 76, 33; 5 x 313 over 1766 + 1695,
// G = 2: 150, 81; 3 x 395 over 6 + 1, G = 4: 100, 30.  One copy a sequence has its own kernel.
int prefix_direct_tiles(int B, int T_out, int P, int T_kv, int Hq, int Hkv, int D)
{
    const long long rows = static_cast<long long>(T_out) * (Hq / Hkv), tiles = (rows + 255) / 256;
    if (T_out <= 1 || B * tiles > 65535)
        return 0;
    const double pairs = (P + 127) / 128 + (T_kv + 127) / 128;
    const double waves = static_cast<double>((B * tiles * Hkv + 151) / 152);
    const double direct = 9.0 + 2.1 * pairs * waves;
    const double all = static_cast<double>(B) * T_out * Hq;
    const double split = 20.0 + 0.002 * all +
                         2.1 * static_cast<double>((B * rows + 255) / 256) * Hkv * ((P + 127) / 128) / 152.0 +
                         all * T_kv * 4.0 * D / 210e6;
    return direct <= split ? static_cast<int>(tiles) : 0;
}

cudaError_t launch_prefix_direct(int D, const PrefixMaps &maps, const PrefixAttnParams &p, cudaStream_t stream)
{
    return launch_prefix_tc(D, PT_DIRECT, maps, p, 1, p.B * static_cast<int>((static_cast<long long>(p.T_out) * (p.Hq / p.Hkv) + 255) / 256),
                            stream);
}

}  // namespace orthros
