// rows_tc.cuh -- attention of tiles of query rows over runs of 64-key blocks on the 5th-generation tensor cores, each row
// with a set of keys of its own in the blocks that it does not see whole: drafted trees over a cache (tree_tc.cu), the
// base stream with sinks and wide windows (swa_wide.cu).  What a piece of work is, where its rows, keys and results
// lie and what a row sees is the job's (a struct of static functions).
//
// One CTA an SM takes its share of the work piece by piece.  Within a piece two softmax streams run, so that one's
// MMAs run while the other's exponentials do:
//   ROWS2: tiles of 128 rows each; every pair of 64-key blocks serves both;
//   KEYS2: one tile of 128 rows; the streams take pairs of blocks in turn, each with its own maximum, sum and O,
//          which are joined at the piece's end, and the ring is one pair deeper.
// Per pair of blocks and stream
//   S = q K^T   fp16, fp32 accumulators in tensor memory.  A q row is scaled by a power of two to a largest value
//               in [2^14, 2^15) before it is rounded; K is converted from bf16 in shared memory, a key row whose
//               largest |k| reaches 65520, or lies below 2^-9, by an exact 2^-e first and its logits multiplied
//               back by 2^e;
//   softmax     a thread a row; blocks that every row sees whole take no mask, the others a 64-bit set a row; the
//               running maximum is raised only when it grows by more than 8 (log2 units);
//   O += P V    bf16, fp32 accumulators in tensor memory.
// Between pieces all roles meet and the next piece's queries are prepared; what the next piece is, and its barriers
// (two sets, in turns), the V producer has settled by then.
//
// Roles (512 threads): warps 0, 3 TMA producers of K and of V; warps 1, 2 lane 0 issues the MMAs of stream 0, 1;
// warps 4-7, 8-11 queries, then softmax and results of stream 0, 1 (their softmaxes take turns, warp by warp);
// warps 12-15 K to fp16, and zeros over the K and V rows that no query of the piece sees (they may hold anything).
// Tensor memory: S of stream t at 128 t; O at 256 + D t.  Every mbarrier wait is bounded; a timeout records
// ORTHROS_DEVERR_TIMEOUT and all roles go to the common exit.
//
// A job J<D, TR> has
//   Params, Maps, Where, Piece { m: blocks (0: none left); plain0, plain1: every row sees these whole; ... }
//   share(p, seed, where)         the CTA's share; whole warp
//   next(p, from, to, where)      the piece behind `from`; one thread
//   place(piece, g, b)            KV head and sequence
//   row_of(p, piece, x)           first key row of block x; negative: rows of the second pair of maps (-1)
//   map(maps, v, j0)              tensor map of a block's K or V
//   span(p, piece, j0, end, lo, first)  the block's rows r < end with j0 + r >= lo or j0 + r < first count for some row
//   query(p, piece, r), vectors(p, piece, alpha, beta)   row r's query (NULL: none; head r % G), the scale-offset
//   See, see(p, piece, r), mask(p, piece, see, j0)       what row r sees of the block at j0; whole warp for see
//   out(p, piece, see, r)         where its result goes
#pragma once

#define ORTHROS_RARE __forceinline__  // this kernel's warps change their register count

#include <cuda_fp16.h>

#include "serve.cuh"
#include "tc.cuh"

namespace orthros {

template <int D, bool ROWS2>
struct RtCfg {
    static constexpr int KB = 64;
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
    // barriers: K block landed [SLOTS], converted [MARKS]; V of a pair landed [MPAIRS]; K, V of a pair released [PAIRS]
    // (its S, its P V complete: MMA commits); of each stream: query tile prepared, S of a pair complete, P written,
    // O += P V of a pair complete but the last, of the last, a softmax warp done with a pair [4]
    static constexpr int B_KCONV = SLOTS, B_VFULL = B_KCONV + MARKS, B_KEMPTY = B_VFULL + MPAIRS, B_VEMPTY = B_KEMPTY + PAIRS;
    static constexpr int B_QFULL = B_VEMPTY + PAIRS, B_SFULL = B_QFULL + 2, B_PFULL = B_SFULL + 2, B_ODONE = B_PFULL + 2;
    static constexpr int B_OFINAL = B_ODONE + 2, B_TURN = B_OFINAL + 2, NBARS = B_TURN + 8;
    static constexpr int HOLD_OFF = BAR_OFF + 2 * NBARS * 8;  // two sets
    static constexpr int USED = HOLD_OFF + 16 + 1024;
    static constexpr int SMEM = USED > 120 * 1024 ? USED : 120 * 1024;  // one CTA an SM: it takes all of tensor memory
    static_assert(SMEM + 256 <= 232448, "shared memory budget");
    static constexpr uint32_t TM_S = 0, TM_O = 256;
    static constexpr int CPR = D / 8;      // 16-byte chunks of a query row
    static constexpr int RPP = 256 / CPR;  // rows one pass of the softmax warps' 256 threads covers
    static constexpr int CONV_THREADS = 128;
};

// a set of 64 with the n lowest
__device__ __forceinline__ unsigned long long bits_below(int n) { return n >= 64 ? ~0ull : (n <= 0 ? 0ull : (1ull << n) - 1); }

// where a row's result goes: as bf16 at `row`, or as a partial (max, sum, unnormalised o) at ml and part
struct RowOut {
    orthros_bf16 *row;  // NULL with part NULL: nowhere
    float *part;
    float2 *ml;
    float *lse;  // optional, beside row: natural log of the row's sum
    bool none;   // the row sees nothing by rule: zeros
};

template <int D, bool ROWS2, template <int, int> class JOB>
__global__ void __launch_bounds__(512, 1)
    rows_tc_kernel(const __grid_constant__ typename JOB<D, RtCfg<D, ROWS2>::TR>::Maps maps,
                   const typename JOB<D, RtCfg<D, ROWS2>::TR>::Params p)
{
    using C = RtCfg<D, ROWS2>;
    using J = JOB<D, C::TR>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_s = smem_u32(smem_raw);
    const uint32_t pad = ((raw_s + 1023u) & ~1023u) - raw_s;
    uint8_t *smem = smem_raw + pad;
    const uint32_t sbase = raw_s + pad;
    int8_t *kexp = reinterpret_cast<int8_t *>(smem + C::KEXP_OFF);
    int8_t *qexp = reinterpret_cast<int8_t *>(smem + C::QSC_OFF);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + C::HOLD_OFF);
    __shared__ volatile int s_abort;  // a wait has given up
    __shared__ typename J::Piece pieces[2];
    __shared__ typename J::Where where;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.Hq / p.Hkv;
    if (warp == 1)
        tmem_alloc(tmem_holder, 512);
    tc_fence_before();
    // what the kernels before wrote first, then a dependent grid may start beside this one
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // one thread: the piece behind `from`, and the barriers of set x, which no role uses
    auto prepare = [&](const typename J::Piece &from, int x, bool exist) {
        if (s_abort)
            pieces[x].m = 0;
        else
            J::next(p, from, pieces[x], where);
        if (pieces[x].m == 0)
            return;
        uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF) + x * C::NBARS;
        for (int i = 0; i < C::NBARS && exist; ++i)
            asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_u32(bar + i)) : "memory");
        for (int i = 0; i < C::SLOTS; ++i)
            mbar_init(bar++, 1);  // kfull
        for (int i = 0; i < C::MARKS; ++i)
            mbar_init(bar++, C::CONV_THREADS / 32);  // kconv
        for (int i = 0; i < C::MPAIRS; ++i)
            mbar_init(bar++, 1);  // vfull
        for (int i = 0; i < 2 * C::PAIRS; ++i)
            mbar_init(bar++, C::TILES);  // kempty, vempty: a commit of each stream that reads the pair
        for (int i = 0; i < 18; ++i)
            mbar_init(bar++, i < 2 ? 8 : (i == 4 || i == 5 ? 4 : 1));  // q_full, s_full, p_full, o_done, o_final, turn
        fence_barrier_init();
    };
    if (warp == 3) {
        J::share(p, pieces[1], where);
        __syncwarp();
        if (lane == 0) {
            s_abort = 0;
            for (int i = 0; i < C::MARKS; ++i)
                reinterpret_cast<uint64_t *>(smem + C::KFLAG_OFF)[i] = 0;
            prepare(pieces[1], 0, false);
        }
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_holder;

    // a role's work on each piece: role(piece, its number of pairs of blocks, KV head, sequence, barriers, number)
    auto each = [&](auto role) {
        for (int number = 0;; ++number) {
            const typename J::Piece &piece = pieces[number & 1];
            if (piece.m == 0)
                break;
            int b, g;
            J::place(piece, g, b);
            role(piece, (piece.m + 1) / 2, g, b, reinterpret_cast<uint64_t *>(smem + C::BAR_OFF) + (number & 1) * C::NBARS, number);
            __syncthreads();  // every role is done with the piece
            if (s_abort)
                break;
        }
    };
    // pairs of stream t, and its u-th
    auto pairs_of = [](int npair, int t) { return ROWS2 ? npair : (npair - t + 1) / 2; };
    auto pair_at = [](int t, int u) { return ROWS2 ? u : 2 * u + t; };
    // first key row of the piece's block x; -1: of the second maps; -2: the place that fills the last pair
    auto row_of = [&](const typename J::Piece &piece, int x) { return x < piece.m ? J::row_of(p, piece, x) : -2; };

    // The softmax warps need more registers than a quarter of the SM's, the others fewer: 56 + 2 * 176 + 104 is what
    // the block was launched with (4 * 128, a thread of each warpgroup).
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        each([&](const typename J::Piece &piece, int npair, int g, int b, uint64_t *bars, int number) {
            uint64_t *kfull = bars, *kconv = bars + C::B_KCONV, *vfull = bars + C::B_VFULL, *kempty = bars + C::B_KEMPTY;
            uint64_t *vempty = bars + C::B_VEMPTY, *q_full = bars + C::B_QFULL, *s_full = bars + C::B_SFULL;
            uint64_t *p_full = bars + C::B_PFULL, *o_done = bars + C::B_ODONE, *o_final = bars + C::B_OFINAL;
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
                        const int j0 = row_of(piece, 2 * pp + h);
                        uint64_t *bar = kv ? &vfull[pp % C::MPAIRS] : &kfull[2 * ps + h];
                        uint8_t *dst = smem + (kv ? C::V_OFF : C::K_OFF) + ps * C::PAIR_BYTES + h * C::KB * 128;
                        const CUtensorMap *map = J::map(maps, kv, j0);
                        const int row = j0 >= 0 ? j0 : (j0 == -1 ? 0 : J::keys(p));  // behind the keys: zeros
                        if (!kv)
                            mbar_arrive_expect_tx(bar, BYTES);
#pragma unroll
                        for (int sl = 0; sl < C::SLABS; ++sl)
                            tma_load_4d(dst + sl * C::PAIR_SLAB, map, bar, sl * 64, g, row, b);
                    }
                }
                if (kv)
                    prepare(piece, (number + 1) & 1, number > 0);
            }
        } else {
            // -------------------------------------------------------------- MMA issuer of stream t
            if (lane == 0) {
                constexpr uint32_t IDESC_QK = umma_idesc(128, 128, false, false);
                constexpr uint32_t IDESC_PV = umma_idesc(128, D, true, true);
                const int t = warp - 1, nu = pairs_of(npair, t);
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
        }
        });
    } else if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        each([&](const typename J::Piece &piece, int npair, int, int, uint64_t *bars, int) {
            // -------------------------------------------------------------- K converters
            uint64_t *kfull = bars, *kconv = bars + C::B_KCONV, *vfull = bars + C::B_VFULL;
            bool ok = true, bad = false;
            // K conversion: 8 consecutive lanes a key row, rows cid / 8 + STEP it of a block
            constexpr int STEP = C::CONV_THREADS / 8;
            const int cid = threadIdx.x - 384;
            const int cw = cid >> 5;
            constexpr int ITS = C::KB / STEP;
            static_assert(C::KB % STEP == 0, "a thread's rows are all in the block");
            const int plain0 = piece.plain0;
            const unsigned plains = piece.plain1 - plain0;
            for (int j = 0; j < 2 * npair && ok; ++j) {
                const int s = j % C::SLOTS;
                if (!(ok = mbar_wait(&kfull[s], static_cast<uint32_t>((j / C::SLOTS) & 1))))
                    break;
                uint8_t *blk = smem + C::K_OFF + (s / 2) * C::PAIR_BYTES + (s % 2) * C::KB * 128;
                // rows that no query of the segment sees have no weight, but may hold anything: zeros, in V too
                int j0 = 0, end = C::KB, span_lo = 0, span_first = 0;
                if (static_cast<unsigned>(j - plain0) >= plains && (j0 = row_of(piece, j)) != -2)
                    J::span(p, piece, j0, end, span_lo, span_first);
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
        });
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        each([&](const typename J::Piece &piece, int npair, int g, int, uint64_t *bars, int) {
            // -------------------------------------------------------------- queries, softmax, results
            uint64_t *kconv = bars + C::B_KCONV, *q_full = bars + C::B_QFULL, *s_full = bars + C::B_SFULL;
            uint64_t *p_full = bars + C::B_PFULL, *o_done = bars + C::B_ODONE, *o_final = bars + C::B_OFINAL;
            uint64_t *turn = bars + C::B_TURN;
            // first the queries, from global memory to fp16 tiles, by all eight warps: a thread has 16 bytes of
            // every RPP-th row, all of one head, and its rows' loads are in flight together
            {
                const float *alpha, *beta;
                J::vectors(p, piece, alpha, beta);
                const int tid = threadIdx.x - 128;  // 0 .. 255
                const int cr = tid % C::CPR, r0 = tid / C::CPR;
                constexpr int ROWS = 128 / C::RPP;
                static_assert(C::RPP % 16 == 0, "a thread's rows share a head");
                const int h = g * G + r0 % G;
                uint32_t have[C::TILES];
#pragma unroll
                for (int tl = 0; tl < C::TILES; ++tl) {
                    have[tl] = 0;
#pragma unroll
                    for (int x = 0; x < ROWS; ++x) {
                        const int r = r0 + x * C::RPP;
                        const orthros_bf16 *src = J::query(p, piece, tl * 128 + r);
                        if (src != nullptr) {
                            cp_async16(smem + C::Q_OFF + tl * C::Q_BYTES + (cr / 8) * C::Q_SLAB + sw128_offset(r, cr % 8),
                                       src + 8 * cr);
                            have[tl] |= 1u << x;
                        }
                    }
                }
                float al[8], be[8];
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    const float4 y = __ldg(reinterpret_cast<const float4 *>(alpha + h * D + 8 * cr + e));
                    const float4 z = __ldg(reinterpret_cast<const float4 *>(beta + h * D + 8 * cr + e));
                    al[e] = y.x * p.qscale, al[e + 1] = y.y * p.qscale, al[e + 2] = y.z * p.qscale, al[e + 3] = y.w * p.qscale;
                    be[e] = z.x * p.qscale, be[e + 1] = z.y * p.qscale, be[e + 2] = z.z * p.qscale, be[e + 3] = z.w * p.qscale;
                }
                cp_async_wait_all();
#pragma unroll
                for (int tl = 0; tl < C::TILES; ++tl) {
                    uint8_t *qb = smem + C::Q_OFF + tl * C::Q_BYTES + (cr / 8) * C::Q_SLAB;
#pragma unroll 2
                    for (int x = 0; x < ROWS; ++x) {
                        const int r = r0 + x * C::RPP;
                        uint4 *slot = reinterpret_cast<uint4 *>(qb + sw128_offset(r, cr % 8));
                        const uint4 raw = (have[tl] >> x) & 1u ? *slot : make_uint4(0, 0, 0, 0);
                        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
                        float f[8], amax = 0.f;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 y = ffma2(unpack_bf16x2(w[e]), make_float2(al[2 * e], al[2 * e + 1]),
                                                   make_float2(be[2 * e], be[2 * e + 1]));
                            f[2 * e] = (have[tl] >> x) & 1u ? y.x : 0.f;
                            f[2 * e + 1] = (have[tl] >> x) & 1u ? y.y : 0.f;
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
            const bool work = J::query(p, piece, tile * 128 + rw * 32) != nullptr;  // the warp has a row
            const typename J::See see = J::see(p, piece, tile * 128 + r);
            const int plain0 = piece.plain0;
            const unsigned plains = piece.plain1 - plain0;
            const uint32_t s_lane = tbase + (static_cast<uint32_t>(rw * 32) << 16) + C::TM_S + 128 * t;
            const uint32_t o_col = tbase + (static_cast<uint32_t>(rw * 32) << 16) + C::TM_O + D * t;
            const float NEG_INF = -__int_as_float(0x7f800000);
            const int nu = pairs_of(npair, t);
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
                        uint32_t va[32], vb[32];
                        tmem_ld32(s_col, va);
                        tmem_ld32(s_col + 32, vb);
                        // the block's conversion completed before its S was issued: this test succeeds and
                        // orders the flag read after the converters' writes
                        const uint32_t kph = static_cast<uint32_t>((j / C::MARKS) & 1);
                        const bool seen = mbar_test_wait(&kconv[ks], kph);
                        const uint64_t kf = *reinterpret_cast<const volatile uint64_t *>(smem + C::KFLAG_OFF + ks * 8);
                        tmem_wait_ld();
                        const bool part = static_cast<unsigned>(j - plain0) >= plains;
                        uint32_t sa = ~0u, sb = ~0u;  // the columns that the row sees
                        if (part) {
                            const int j0 = row_of(piece, j);
                            const unsigned long long set = j0 == -2 ? 0 : J::mask(p, piece, see, j0);
                            sa = static_cast<uint32_t>(set);
                            sb = static_cast<uint32_t>(set >> 32);
                        }
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
                                    range_bad |= any && isinf(__uint_as_float(va[e])) && ((sa >> e) & 1);
                                    range_bad |= any && isinf(__uint_as_float(vb[e])) && ((sb >> e) & 1);
                                }
                            }
                        }
                        if (part) {
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
                const RowOut to = J::out(p, piece, see, tile * 128 + r);
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
                const bool two = !ROWS2 && pairs_of(npair, 1) > 0;
                if (ok) {
                    tc_fence_after();
                    const float inv = L > 0.f ? 1.f / L : L;  // a NaN stays one
                    if (to.part != nullptr && (ROWS2 || t == 0))
                        *to.ml = to.none ? make_float2(NEG_INF, 0.f) : make_float2(M, L);
                    if (to.lse != nullptr && (ROWS2 || t == 0))
                        *to.lse = (M + __log2f(L)) * kLn2F;
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
                        if (to.none)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                v[e] = 0u;
                        if (to.row != nullptr) {
#pragma unroll
                            for (int e = 0; e < 32; e += 8) {
                                uint32_t w[4];
#pragma unroll
                                for (int x = 0; x < 4; ++x)
                                    w[x] = pack_bf16x2(__uint_as_float(v[e + 2 * x]) * inv, __uint_as_float(v[e + 2 * x + 1]) * inv);
                                *reinterpret_cast<uint4 *>(to.row + c + e) = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        } else if (to.part != nullptr) {
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
                                st_global_v8(to.part + c + e, make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]),
                                             make_uint4(v[e + 4], v[e + 5], v[e + 6], v[e + 7]));
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
            tc_fence_before();  // the next piece's MMAs write over S and O
        });
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

template <int D, bool ROWS2, template <int, int> class JOB>
static cudaError_t launch_rows_tc(const typename JOB<D, RtCfg<D, ROWS2>::TR>::Maps &maps,
                                  const typename JOB<D, RtCfg<D, ROWS2>::TR>::Params &p, int ctas, cudaStream_t stream)
{
    using C = RtCfg<D, ROWS2>;
    auto kern = rows_tc_kernel<D, ROWS2, JOB>;
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

}  // namespace orthros
