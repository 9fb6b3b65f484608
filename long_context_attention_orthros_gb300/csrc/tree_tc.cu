// tree_tc.cu -- both streams of a tree of drafted tokens over a KV cache on the 5th-generation tensor cores: the
// form of tree_step.cu for more query rows a KV head than its warp MMAs keep up with.
//
// One CTA an SM takes its share of the list of key blocks (tree.cuh) piece by piece, a piece being its blocks of
// one segment.  Within a piece two softmax streams run, so that one's MMAs run while the other's exponentials do:
//   ROWS2: tiles of 128 rows each; every pair of 64-key blocks serves both (more than 128 rows a KV head);
//   KEYS2: one tile of 128 rows; the streams take pairs of blocks in turn, each with its own maximum, sum and O,
//          which are joined at the piece's end, and the ring is one pair deeper.
// Per pair of blocks and stream
//   S = q K^T   fp16, fp32 accumulators in tensor memory.  A q row is scaled by a power of two to a largest value
//               in [2^14, 2^15) before it is rounded; K is converted from bf16 in shared memory, a key row whose
//               largest |k| reaches 65520, or lies below 2^-9, by an exact 2^-e first and its logits multiplied
//               back by 2^e;
//   softmax     a thread a row; blocks that every row sees whole take no mask, the others a 64-bit set a row (the
//               window, the sinks, the path); the running maximum is raised only when it grows by more than 8;
//   O += P V    bf16, fp32 accumulators in tensor memory.
// A piece that is its whole segment leaves as bf16, another as one partial (max, sum, o), which tree_join_kernel joins.
// Between pieces all roles meet, the barriers are set up anew and the next piece's queries are prepared: some 4 us.
//
// Roles (512 threads): warps 0, 3 TMA producers of K and of V; warps 1, 2 lane 0 issues the MMAs of stream 0, 1;
// warps 4-7, 8-11 queries, then softmax and results of stream 0, 1 (their softmaxes take turns, warp by warp);
// warps 12-15 K to fp16, and zeros over the K and V rows that no query of the segment sees.
// Tensor memory: S of stream t at 128 t; O at 256 + D t.  Every mbarrier wait is bounded; a timeout records
// ORTHROS_DEVERR_TIMEOUT and all roles go to the common exit.
#include <cuda_fp16.h>

#include "tc.cuh"
#include "tree_rows.cuh"

namespace orthros {

template <int D, bool ROWS2>
struct TtCfg {
    static constexpr int KB = TREE_KB;
    static constexpr int SLABS = D / 64;
    static constexpr int TILES = ROWS2 ? 2 : 1;
    static constexpr int TR = 128 * TILES;
    static constexpr int Q_SLAB = 128 * 128;
    static constexpr int Q_BYTES = SLABS * Q_SLAB;
    static constexpr int PAIR_SLAB = 128 * 128;           // 128 keys of one 64-wide slab
    static constexpr int PAIR_BYTES = SLABS * PAIR_SLAB;  // K, or V, of a pair
    static constexpr int PAIRS = ROWS2 ? 2 : 3;
    static constexpr int SLOTS = 2 * PAIRS;  // 64-key blocks of the ring
    static constexpr int K_OFF = 0;
    static constexpr int V_OFF = PAIRS * PAIR_BYTES;
    static constexpr int Q_OFF = 2 * PAIRS * PAIR_BYTES;
    // Marks of a block's conversion live two rounds of the ring: K is released when its S are complete,
    // before the softmax has read them, and the block two rounds later is converted after it has.
    static constexpr int MARKS = 2 * SLOTS;
    static constexpr int KEXP_OFF = Q_OFF + TILES * Q_BYTES;  // int8 [MARKS][KB]: key row shift
    static constexpr int KFLAG_OFF = KEXP_OFF + MARKS * KB;   // uint8 [MARKS][8]
    static constexpr int QSC_OFF = KFLAG_OFF + MARKS * 8;     // int8 [TILES][128]: query row shift
    static constexpr int BAR_OFF = QSC_OFF + TILES * 128;
    static constexpr int MPAIRS = 2 * PAIRS;  // an even number: a mark of a pair belongs to one stream for good
    static constexpr int NBARS = SLOTS + MARKS + MPAIRS + 2 * PAIRS + 18;
    static constexpr int HOLD_OFF = BAR_OFF + NBARS * 8;
    static constexpr int USED = HOLD_OFF + 16 + 1024;
    static constexpr int SMEM = USED > 120 * 1024 ? USED : 120 * 1024;  // one CTA an SM: it takes all of tensor memory
    static_assert(SMEM + 256 <= 232448, "shared memory budget");
    static constexpr uint32_t TM_S = 0, TM_O = 256;
    static constexpr int CPR = D / 8;      // 16-byte chunks of a query row
    static constexpr int RPP = 256 / CPR;  // rows one pass of the softmax warps' 256 threads covers
    static constexpr int CONV_THREADS = 128;
};

// the piece at hand, and where the CTA stands in the list; written by one thread between pieces
template <int TR>
struct TreePiece {
    TreeCursor<TR, TREE_TC_COST> cur;  // the piece's segment, at its first place
    int first, m;                      // its blocks: first .. first + m - 1; m = 0: none left
    int alone;                         // the whole segment
    long long slot;                    // of its partial
    long long it, it1, W, n;
};

template <int D, bool ROWS2>
__global__ void __launch_bounds__(512, 1) tree_tc_kernel(const __grid_constant__ TreeMaps maps, const TreeParams p)
{
    using C = TtCfg<D, ROWS2>;
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
    __shared__ volatile int s_abort;  // a wait has given up
    __shared__ TreePiece<C::TR> piece;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.Hq / p.Hkv;
    if (warp == 1)
        tmem_alloc(tmem_holder, 512);
    tc_fence_before();
    // what the kernels before wrote first, then a dependent grid may start beside this one
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 0) {
        const TreeShare<C::TR, TREE_TC_COST> sh = tree_share<C::TR, TREE_TC_COST>(p, blockIdx.x, gridDim.x);
        if (lane == 0) {
            piece.cur = sh.cur;
            piece.it = sh.it0;
            piece.it1 = sh.it1;
            piece.W = sh.W;
            piece.n = sh.n;
            piece.m = 0;
            s_abort = 0;
        }
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_holder;
    int paths_b = -1;
    TreePaths paths = {};

    bool barriers = false;  // they exist (one thread's)
    while (true) {
        __syncthreads();  // every role is done with the piece before
        if (threadIdx.x == 0) {
            // the next piece that has blocks (a share may begin or end with a segment's empty places)
            int m = 0;
            while (m == 0 && piece.it < piece.it1 && !s_abort) {
                if (piece.cur.r == piece.cur.places())
                    piece.cur.next_segment(p);
                const int at = piece.cur.r, all = piece.cur.places();
                const long long left = piece.it1 - piece.it;
                const int places = static_cast<int>(all - at < left ? all - at : left);
                const int first = max(at - TREE_TC_COST, 0);
                m = max(at + places - TREE_TC_COST - first, 0);
                const long long s0 = piece.it - at + TREE_TC_COST, s1 = piece.it - at + all;
                const long long c0 = ((s0 + 1) * piece.n - 1) / piece.W, c1 = (s1 * piece.n - 1) / piece.W;
                piece.first = first;
                piece.alone = c0 == c1;
                piece.slot = 2 * static_cast<long long>(blockIdx.x) + (blockIdx.x == c0 ? 1 : 0);
                piece.it += places;
                piece.cur.r = at + places;
            }
            piece.m = m;
            if (m > 0) {
                for (int s = 0; s < C::NBARS && barriers; ++s)
                    asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_u32(kfull + s)) : "memory");
                barriers = true;
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
        }
        __syncthreads();
        const int m = piece.m;
        if (m == 0)
            break;
        const int b = piece.cur.b, g = piece.cur.g, base = piece.cur.base, first = piece.first;
        const int npair = (m + 1) / 2;
        auto pairs_of = [&](int t) { return ROWS2 ? npair : (npair - t + 1) / 2; };  // of stream t
        auto pair_at = [&](int t, int u) { return ROWS2 ? u : 2 * u + t; };           // its u-th
        // first cached row of the piece's block x; -1: the tree's own rows; -2: the place that fills the last pair
        auto row_of = [&](int x) { return x < m ? piece.cur.first_row(first + x) : -2; };

        if (warp == 0 || warp == 3) {
            // -------------------------------------------------------------- producers of K, of V
            if (lane == 0) {
                const bool kv = warp == 3;
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
                        const int j0 = row_of(2 * pp + h);
                        uint64_t *bar = kv ? &vfull[pp % C::MPAIRS] : &kfull[2 * ps + h];
                        uint8_t *dst = smem + (kv ? C::V_OFF : C::K_OFF) + ps * C::PAIR_BYTES + h * C::KB * 128;
                        const CUtensorMap *map = j0 == -1 ? (kv ? &maps.vt : &maps.kt) : (kv ? &maps.v : &maps.k);
                        const int row = j0 >= 0 ? j0 : (j0 == -1 ? 0 : p.L_max);  // behind the cache: zeros
                        if (!kv)
                            mbar_arrive_expect_tx(bar, BYTES);
#pragma unroll
                        for (int sl = 0; sl < C::SLABS; ++sl)
                            tma_load_4d(dst + sl * C::PAIR_SLAB, map, bar, sl * 64, g, row, b);
                    }
                }
            }
        } else if (warp < 3) {
            // -------------------------------------------------------------- MMA issuer of stream t
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
                // no commit is in flight when the piece ends: all others have been waited for
                if (ok && nu > 0)
                    ok = mbar_wait(&o_final[t], 0);
                if (!ok) {
                    s_abort = 1;
                    record_error(p.dev_err, ORTHROS_DEVERR_TIMEOUT);
                }
            }
        } else if (warp >= 12) {
            // -------------------------------------------------------------- K converters
            bool ok = true, bad = false;
            // K conversion: 8 consecutive lanes a key row, rows cid / 8 + STEP it of a block
            constexpr int STEP = C::CONV_THREADS / 8;
            const int cid = threadIdx.x - 384;
            const int cw = cid >> 5;
            constexpr int ITS = C::KB / STEP;
            static_assert(C::KB % STEP == 0, "a thread's rows are all in the block");
            const int len = piece.cur.s.len, live = piece.cur.s.n;
            int span_lo, span_first;
            tree_span(p, piece.cur.s, base, span_lo, span_first);
            for (int j = 0; j < 2 * npair && ok; ++j) {
                const int s = j % C::SLOTS;
                if (!(ok = mbar_wait(&kfull[s], static_cast<uint32_t>((j / C::SLOTS) & 1))))
                    break;
                uint8_t *blk = smem + C::K_OFF + (s / 2) * C::PAIR_BYTES + (s % 2) * C::KB * 128;
                // rows that no query of the segment sees have no weight, but may hold anything: zeros, in V too
                const int j0 = row_of(j), end = j0 >= 0 ? len - j0 : (j0 == -1 ? live : C::KB);
                auto counts = [&](int r) { return r < end && (j0 < 0 || j0 + r >= span_lo || j0 + r < span_first); };
                const bool part = end < C::KB || (j0 >= 0 && j0 < span_lo);
                if (part)
                    for (int r = cid >> 3; r < C::KB; r += STEP)
                        if (!counts(r))
#pragma unroll
                            for (int sl = 0; sl < C::SLABS; ++sl)
                                *reinterpret_cast<uint4 *>(blk + sl * C::PAIR_SLAB + r * 128 + (cid & 7) * 16) =
                                    make_uint4(0, 0, 0, 0);
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
                            *reinterpret_cast<uint4 *>(blk + sl * C::PAIR_SLAB + ((cid >> 3) + STEP * it) * 128 +
                                                       (cid & 7) * 16) = k_to_fp16(u[it][sl]);
                } else {
                    shift_key_rows<C::SLABS, true>(blk, C::PAIR_SLAB, 0, cid >> 3, STEP, ITS, cid & 7,
                                                   kexp + (j % C::MARKS) * C::KB, bad);
                }
                if (part) {
                    if (!(ok = mbar_wait(&vfull[j / 2 % C::MPAIRS], static_cast<uint32_t>((j / 2 / C::MPAIRS) & 1))))
                        break;
                    for (int r = cid >> 3; r < C::KB; r += STEP)
                        if (!counts(r))
#pragma unroll
                            for (int sl = 0; sl < C::SLABS; ++sl)
                                *reinterpret_cast<uint4 *>(blk + (C::V_OFF - C::K_OFF) + sl * C::PAIR_SLAB + r * 128 +
                                                           (cid & 7) * 16) = make_uint4(0, 0, 0, 0);
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
            // -------------------------------------------------------------- queries, softmax, results
            const TreeSeq seq = piece.cur.s;
            const int tile_row = piece.cur.tile * C::TR;
            if (b != paths_b) {
                paths = tree_paths(p.parent + static_cast<long long>(b) * p.N, seq.n);
                paths_b = b;
            }
            // first the queries, from global memory to fp16 tiles, by all eight warps: a thread has 16 bytes of
            // every RPP-th row, all of one head, and its rows' loads are in flight together
            {
                const orthros_bf16 *src = base ? p.q_new : p.qc_new;
                const float *alpha = base ? p.alpha : p.alpha_c, *beta = base ? p.beta : p.beta_c;
                const int tid = threadIdx.x - 128;  // 0 .. 255
                const int cr = tid % C::CPR, r0 = tid / C::CPR;
                constexpr int ROWS = 128 / C::RPP;
                static_assert(C::RPP % 16 == 0, "a thread's rows share a head");
                const int h = g * G + r0 % G;
                float al[8], be[8];
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    const float4 y = __ldg(reinterpret_cast<const float4 *>(alpha + h * D + 8 * cr + e));
                    const float4 z = __ldg(reinterpret_cast<const float4 *>(beta + h * D + 8 * cr + e));
                    al[e] = y.x * p.qscale, al[e + 1] = y.y * p.qscale, al[e + 2] = y.z * p.qscale, al[e + 3] = y.w * p.qscale;
                    be[e] = z.x * p.qscale, be[e + 1] = z.y * p.qscale, be[e + 2] = z.z * p.qscale, be[e + 3] = z.w * p.qscale;
                }
#pragma unroll 1
                for (int tl = 0; tl < C::TILES; ++tl) {
                    uint8_t *qb = smem + C::Q_OFF + tl * C::Q_BYTES + (cr / 8) * C::Q_SLAB;
                    uint32_t have = 0;
#pragma unroll
                    for (int x = 0; x < ROWS; ++x) {
                        const int r = r0 + x * C::RPP, node = (tile_row + tl * 128 + r) / G;
                        if (node < seq.n) {
                            cp_async16(qb + sw128_offset(r, cr % 8),
                                       src + ((static_cast<long long>(b) * p.N + node) * p.Hq + h) * D + 8 * cr);
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
            const int row_i = tile_row + tile * 128 + r, node = row_i / G;
            const bool work = (tile_row + tile * 128 + rw * 32) / G < seq.n;  // the warp has a row
            const TreeRow row = tree_row(p, seq, paths, base, node);
            const uint32_t s_lane = tbase + (static_cast<uint32_t>(rw * 32) << 16) + C::TM_S + 128 * t;
            const uint32_t o_col = tbase + (static_cast<uint32_t>(rw * 32) << 16) + C::TM_O + D * t;
            const float NEG_INF = -__int_as_float(0x7f800000);
            const int nu = pairs_of(t);
            bool ok = mbar_wait(&q_full[tile], 0), range_bad = false;
            const float qf = exp2i(qexp[tile * 128 + r]);  // logit = S qf
            const float2 qf2 = make_float2(qf, qf);
            float mx = NEG_INF, l = 0.f;
            for (int u = 0; u < nu && ok; ++u) {
                const int pp = pair_at(t, u);
                if (!(ok = mbar_wait(&s_full[t], static_cast<uint32_t>(u & 1)) &&
                           (t + u == 0 ||
                            mbar_wait(&turn[4 * (1 - t) + rw], static_cast<uint32_t>((t == 0 ? u - 1 : u) & 1)))))
                    break;
                tc_fence_after();
                if (work) {
                    float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
                    for (int hh = 0; hh < 2 && ok; ++hh) {
                        const int j = 2 * pp + hh, ks = j % C::MARKS;
                        const uint32_t s_col = s_lane + 64 * hh;
                        // the columns that the row sees
                        const int j0 = row_of(j);
                        unsigned long long see = 0;
                        if (j0 == -1) {
                            see = row.mask;
                        } else if (j0 >= 0) {
                            auto below = [](int n) { return n >= 64 ? ~0ull : (n <= 0 ? 0ull : (1ull << n) - 1); };
                            // lo - j0 does not overflow: both lie in [0, 2^31)
                            see = below(seq.len - j0) & (~below(row.lo - j0) | below(row.first - j0));
                        }
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
                                bool any = false;
                                unshift_chunk32(s_col, kexp + ks * C::KB, 0, kw, C::CONV_THREADS / 8, 4, any);
                                unshift_chunk32(s_col + 32, kexp + ks * C::KB, 32, kw, C::CONV_THREADS / 8, 4, any);
                                tmem_ld32(s_col, va);
                                tmem_ld32(s_col + 32, vb);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e) {  // is it a logit that counts?
                                    range_bad |= any && isinf(__uint_as_float(va[e])) && ((see >> e) & 1);
                                    range_bad |= any && isinf(__uint_as_float(vb[e])) && ((see >> (32 + e)) & 1);
                                }
                            }
                        }
                        if (__any_sync(0xffffffffu, see != ~0ull)) {
                            const uint32_t sa = static_cast<uint32_t>(see), sb = static_cast<uint32_t>(see >> 32);
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                if (!(sa & (1u << e)))
                                    va[e] = __float_as_uint(NEG_INF);
                                if (!(sb & (1u << e)))
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
                        const bool raise = mb > mx + 8.f;
                        if (__any_sync(0xffffffffu, raise)) {
                            const float f = raise ? fast_exp2(mx - mb) : 1.f;  // mx = -inf before the first key: 0
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
                                mx = mb;
                            }
                        }
                        const float uo = mx == NEG_INF ? 0.f : mx;
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
            // ---- results: ROWS2 a thread a row; KEYS2 both streams' threads half of a row's columns each, the
            // maximum and sum of the other stream through the columns of its S, which its last P V has read
            if (nu > 0 && !(ok = ok && mbar_wait(&o_final[t], 0)))
                record_error(p.dev_err, ORTHROS_DEVERR_TIMEOUT);
            tc_fence_after();
            if (!ROWS2) {
                const uint32_t w[8] = {__float_as_uint(mx), __float_as_uint(l), 0, 0, 0, 0, 0, 0};
                tmem_st8(s_lane, w);
                tmem_wait_st();
                tc_fence_before();
                named_barrier(1 + rw, 64);  // the two warps of these rows
                tc_fence_after();
            }
            if (ok && work) {
                const bool store = node < seq.n, none = seq.full || ((paths.bad >> (node & 63)) & 1);
                float f0 = 1.f, f1 = 0.f, M = mx, L = l;
                if (!ROWS2) {
                    uint32_t w[16];
                    tmem_ld16(s_lane + (t ? -128 : 128), w);
                    tmem_wait_ld();
                    const float om = __uint_as_float(w[0]), ol = __uint_as_float(w[1]);
                    M = fmaxf(mx, om);
                    const float own = l == 0.f ? 0.f : fast_exp2(mx - M), other = ol == 0.f ? 0.f : fast_exp2(om - M);  // a NaN goes on
                    L = own * l + other * ol;
                    f0 = t ? other : own;
                    f1 = t ? own : other;
                }
                const bool two = !ROWS2 && pairs_of(1) > 0;
                if (ok) {
                    tc_fence_after();
                    const bool alone = piece.alone;
                    const float inv = L > 0.f ? 1.f / L : L;  // a NaN stays one
                    const long long prow = piece.slot * C::TR + tile * 128 + r;
                    orthros_bf16 *orow = (base ? p.o : p.oc) +
                                         ((static_cast<long long>(b) * p.N + node) * p.Hq + g * G + row_i % G) * D;
                    if (!alone && store && (ROWS2 || t == 0))
                        p.part_ml[prow] = none ? make_float2(NEG_INF, 0.f) : make_float2(M, L);
                    const uint32_t o0 = tbase + (static_cast<uint32_t>(rw * 32) << 16) + C::TM_O + (ROWS2 ? D * t : 0);
                    const int c_lo = ROWS2 ? 0 : t * (D / 2), c_hi = ROWS2 ? D : c_lo + D / 2;
#pragma unroll 1
                    for (int c = c_lo; c < c_hi; c += 32) {
                        uint32_t v[32];
                        tmem_ld32(o0 + c, v);
                        if (two) {
                            uint32_t w[32];
                            tmem_ld32(o0 + D + c, w);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                v[e] = __float_as_uint(fmaf(f0, __uint_as_float(v[e]), f1 * __uint_as_float(w[e])));
                        } else {
                            tmem_wait_ld();
                            if (!ROWS2)
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    v[e] = __float_as_uint(f0 * __uint_as_float(v[e]));
                        }
                        if (!store)
                            continue;
                        if (none)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                v[e] = 0u;
                        if (alone) {
#pragma unroll
                            for (int e = 0; e < 32; e += 8) {
                                uint32_t w[4];
#pragma unroll
                                for (int x = 0; x < 4; ++x)
                                    w[x] = pack_bf16x2(__uint_as_float(v[e + 2 * x]) * inv, __uint_as_float(v[e + 2 * x + 1]) * inv);
                                *reinterpret_cast<uint4 *>(orow + c + e) = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
                                st_global_v8(p.part_o + prow * D + c + e, make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]),
                                             make_uint4(v[e + 4], v[e + 5], v[e + 6], v[e + 7]));
                        }
                    }
                }
            }
            if (!base && g == 0 && piece.cur.tile == 0 && threadIdx.x == 128) {
                const int raw = __ldcg(p.cache_len + b);
                if (raw < 0 || raw > p.L_max)
                    record_error(p.dev_err, ORTHROS_DEVERR_CACHE_FULL);
                else if (seq.full || paths.bad != 0)
                    record_error(p.dev_err, ORTHROS_DEVERR_POSITION);
            }
            if (range_bad)
                record_error(p.dev_err, ORTHROS_DEVERR_RANGE);
            if (!ok) {
                s_abort = 1;
                if (lane == 0)
                    record_error(p.dev_err, ORTHROS_DEVERR_TIMEOUT);
            }
            tc_fence_before();  // the next piece's MMAs write over S and O
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

template <int D, bool ROWS2>
static cudaError_t launch_tt(const TreeMaps &maps, const TreeParams &p, int ctas, cudaStream_t stream)
{
    using C = TtCfg<D, ROWS2>;
    auto kern = tree_tc_kernel<D, ROWS2>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(512);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, maps, p);
}

cudaError_t launch_tree_tc(int D, int tr, const TreeMaps &maps, const TreeParams &p, int ctas, cudaStream_t stream)
{
    if (D == 128)
        return tr == 128 ? launch_tt<128, false>(maps, p, ctas, stream) : launch_tt<128, true>(maps, p, ctas, stream);
    return tr == 128 ? launch_tt<64, false>(maps, p, ctas, stream) : launch_tt<64, true>(maps, p, ctas, stream);
}

}  // namespace orthros
