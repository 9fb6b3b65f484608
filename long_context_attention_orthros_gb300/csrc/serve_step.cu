// serve_step.cu -- one decode step over an 8-bit KV cache, or over a prompt prefix that the
// whole batch shares and each sequence's own bf16 cache.  Per sequence with p = cache_len[b]:
//   append k_new / v_new at own row p (as codes in the 8-bit form),
//   o  = Eq. (4) for the new base token over its last `window` rows,
//   oc = Eq. (5) for its output copy over every row (prefix, own rows, the new one),
//   cache_len[b] = p + 1.
//
// Bound by the cache's bytes (2 (d + 1) a row and head as codes, 4 d in bf16) where there are many, by the
// start, the segments' borders and the join where there are few.  Measured (32/8 heads, d = 128): codes,
// 2 x 131072 rows 90 us (6.0 TB/s: 90% of a plain copy's rate), 8 ragged caches of up to 16384 rows 40 us
// (57%), 1 x 300 rows (8/2 heads, d = 64) 9.1 us.
//
// The work of a step is a list of segments, two for each (b, KV head): the copy's own rows
// 0 .. p, and the base token's window (which in the prefix form may begin in the prefix).  Each
// is a run of 64-key blocks; laid end to end they form one list of W blocks, and CTA c of n takes
// blocks floor(c W / n) .. floor((c + 1) W / n) - 1, whatever sequence they belong to: a ragged
// batch loads every SM alike.  A CTA's blocks arrive by TMA through a ring that runs on across
// segment borders (one producer warp); a segment counts a few places more than its blocks, for
// what its start and end cost.  Four warps take 16 keys of a block each (or 32 of
// every other block), with the query
// rows of a KV head on the MMA's N side, and their results meet in shared memory.  A segment that
// one CTA holds whole is written out at once; otherwise each CTA writes one partial (max, sum,
// o), goes on, and when it has run out of blocks counts itself in: the last to finish a segment
// joins its partials (a counter, no spin).  Partials are bounded by the grid (two a CTA: one
// segment can run in from the CTA before, one can run out).
//
// The block that holds row p is patched in shared memory by the warp that owns the rows: the
// new row goes in, rows behind it (whatever the cache holds there) become zeros.  The last CTA
// of the grid to finish advances cache_len.
//
// In the prefix form the copy's attention over the prefix itself runs in a kernel of its own
// before this one, for all rows of the batch at once (prefix_attn.cu); this kernel is launched as
// its programmatic dependent and waits for it only where it joins a copy's partials.  The same
// kernel without window and append serves one copy a sequence behind a prefix (a prompt's end).
#include <type_traits>

#include "serve.cuh"
#include "warp_b16.cuh"
#include "warp_q8.cuh"

namespace orthros {

constexpr int SERVE_CTAS = 304;  // two on each of 152 SMs (G = 16, d = 128 behind a prefix: one, two rounds)

// a segment whose partials have to be joined, kept until the CTA has run out of blocks
struct Join {
    int bh, base, c0, parts;  // own parts: CTAs c0 .. c0 + parts - 1
    int last;                 // this CTA was the last of them to finish
    int pad;
};
constexpr int MAX_JOINS = 32;

// what the kernel does beside the two 8-bit forms (ORTHROS_KV_E4M3, ORTHROS_KV_INT8)
constexpr int SV_PREFIX = -1;  // a decode step behind a shared prefix
constexpr int SV_COPIES = -2;  // one copy a sequence behind a shared prefix: no window, no append

template <int D, int G, int CODE>
struct SvCfg {
    static constexpr bool Q8 = CODE >= 0, STEP = CODE != SV_COPIES;
    static constexpr int SEGS = STEP ? 2 : 1;  // segments of a (b, KV head)
    static constexpr int KB = 64;
    static constexpr int KV_BYTES = KB * D * (Q8 ? 1 : 2);
    static constexpr int SLAB = KB * 128;  // bf16: one 64-wide slab
    // A step of 16 keys is a chain of some 300 dependent instructions.  A warp takes 32 keys at once,
    // two independent chains, and the warps take blocks by pairs (G = 16 has no registers for it).
    static constexpr int KT = G <= 8 ? 2 : 1;
    static constexpr int CWARPS = 4;
    static constexpr int GROUP = 4 / KT;  // warps that share a block
    static constexpr int SCR_ROWS = CWARPS * G;
    static constexpr int SCR_BYTES = SCR_ROWS * (D + 3) * 4;  // the warps' o, max, sum, scale of o
    static constexpr int LIMIT = 113 * 1024 - 2048;            // two CTAs share an SM (see STAGES)
    // a segment's queries, its alpha and beta and the new K and V row come through a buffer of their
    // own, free again once the segment has begun
    static constexpr int HB = 1;
    static constexpr int HDR_NEW = G * D * (2 + 4 + 4);
    static constexpr int HDR_BYTES = HDR_NEW + 2 * D * 2;
    static constexpr int FIT = (LIMIT - SCR_BYTES - HB * HDR_BYTES) / (2 * KV_BYTES + 2 * KB);
    // A slot of the ring always holds blocks of the same warps (a multiple of KT stages): warps that
    // skipped one of a slot's phases could take the phase before it for the one they wait for.
    // At most four stages: with more bytes in flight the SMs that are nearer to memory get ahead of
    // the others, and equal shares end as late as the last one.  A step over 2 x 131072 rows (D = 128,
    // e4m3): 6 stages 100 us, 4 stages 89 us, the median CTA at 78 us in both.
    // bf16 at G = 16, D = 128 has room for one stage beside the warps' results; it takes two (122 KB), and one CTA an SM.
    static constexpr int MOST = 4;
    static constexpr int STAGES = FIT < 2 ? 2 : (FIT > MOST ? MOST : FIT / KT * KT);
    static_assert(STAGES % KT == 0, "a slot belongs to one group of warps");
    static constexpr int EXP_OFF = STAGES * 2 * KV_BYTES;
    static constexpr int HDR_OFF = EXP_OFF + STAGES * 2 * KB;
    static constexpr int SCR_OFF = HDR_OFF + HB * HDR_BYTES;
    static constexpr int BAR_OFF = SCR_OFF + SCR_BYTES;
    static constexpr int JOIN_OFF = BAR_OFF + (2 * STAGES + 2 * HB) * 8;
    static constexpr int FLAG_OFF = JOIN_OFF + MAX_JOINS * static_cast<int>(sizeof(Join));
    static constexpr int SMEM = FLAG_OFF + 16 + 1024;
    static_assert(SMEM <= 232448, "shared memory budget");
    static_assert(HDR_OFF % 16 == 0 && SCR_OFF % 16 == 0 && BAR_OFF % 8 == 0 && JOIN_OFF % 8 == 0, "alignment");
    static constexpr int CTHREADS = CWARPS * 32;
    static constexpr int THREADS = CTHREADS + 32;
};

// What a segment costs beside its blocks (its queries' loads, the warps' and the CTAs' joins), in
// blocks: every segment begins with so many empty places in the list, so that a CTA with many
// short segments gets fewer blocks.
constexpr int SEG_COST = 4;

// what a sequence's length makes of it
struct SeqPlan {
    int p;         // the last own row: the new token's, or the copy's position
    int full;      // no such row: zero outputs, no append
    int nc, nb;    // blocks of the copy's segment and of the base token's
    int npb;       // window blocks in the prefix; they come first
    int pb0, ob0;  // their first block, and the first own block of the window
    int lo_p, lo;  // first prefix row and first own row of the window
};

template <class C>
__device__ __forceinline__ SeqPlan seq_plan(const ServeParams &p, int len)
{
    SeqPlan s;
    s.p = len;
    s.full = s.p < 0 || s.p >= p.L_max;
    s.npb = s.pb0 = s.ob0 = s.lo_p = s.lo = 0;
    s.nc = 1;
    s.nb = C::SEGS - 1;
    if (!s.full) {
        s.nc = s.p / 64 + 1;
        if constexpr (C::STEP) {
            const int lo = s.p - p.window + 1;  // window >= 1, p >= 0: no overflow
            s.lo = lo > 0 ? lo : 0;
            if (p.P > 0 && lo < 0) {
                s.lo_p = p.P + lo > 0 ? p.P + lo : 0;
                s.pb0 = s.lo_p / 64;
                s.npb = (p.P - 1) / 64 + 1 - s.pb0;
            }
            s.ob0 = s.lo / 64;
            s.nb = s.nc - s.ob0 + s.npb;
        }
    }
    return s;
}

// a position in the list: place r of segment (b, g, base), which holds block r - SEG_COST
struct Cursor {
    int b, g, base, r;
    SeqPlan s;
    __device__ __forceinline__ int blocks() const { return base ? s.nb : s.nc; }
    __device__ __forceinline__ int places() const { return SEG_COST + blocks(); }
    template <class C>
    __device__ __forceinline__ void next_segment(const ServeParams &p)
    {
        r = 0;
        if (C::SEGS == 2 && !base) {
            base = 1;
            return;
        }
        base = 0;
        if (++g == p.Hkv) {
            g = 0;
            if (++b < p.B)
                s = seq_plan<C>(p, __ldcg(p.cache_len + b));
        }
    }
    // block r of the segment: whether it lies in the prefix, and which 64 rows it holds there
    template <class C>
    __device__ __forceinline__ int block(int i, bool &pre) const
    {
        pre = C::STEP && base && i < s.npb;
        return pre ? s.pb0 + i : (base ? s.ob0 + i - s.npb : i);
    }
};

template <class C>
__device__ __forceinline__ long long seq_places(const ServeParams &p, int len)
{
    const SeqPlan s = seq_plan<C>(p, len);
    return static_cast<long long>(s.nc + s.nb + C::SEGS * SEG_COST) * p.Hkv;
}

// Called by a whole warp: CTA c of at most n takes places it0 .. it1 - 1 of the list's W, and its
// cursor stands at it0.  Up to 32 sequences the lengths are read once.
struct Share {
    long long W, n, it0, it1;
    Cursor cur;
};

template <class C>
__device__ __forceinline__ Share plan_share(const ServeParams &p, long long c, long long n)
{
    const int lane = threadIdx.x & 31;
    Share sh;
    int len = lane < p.B ? __ldcg(p.cache_len + lane) : 0;
    long long w = lane < p.B ? seq_places<C>(p, len) : 0, W = w;
    for (int b = lane + 32; b < p.B; b += 32)
        W += seq_places<C>(p, __ldcg(p.cache_len + b));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        W += __shfl_xor_sync(0xffffffffu, W, off);
    sh.W = W;
    sh.n = n < W ? n : W;
    sh.it0 = c < sh.n ? c * W / sh.n : W;
    sh.it1 = c < sh.n ? (c + 1) * W / sh.n : W;
    sh.cur = Cursor{};
    if (sh.it0 >= sh.it1)
        return sh;
    long long it = sh.it0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        if (b0 > 0) {
            len = b0 + lane < p.B ? __ldcg(p.cache_len + b0 + lane) : 0;
            w = b0 + lane < p.B ? seq_places<C>(p, len) : 0;
        }
        long long inc = w;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off)
                inc += y;
        }
        const uint32_t here = __ballot_sync(0xffffffffu, inc > it);
        if (here != 0) {
            const int f = __ffs(here) - 1;
            it -= __shfl_sync(0xffffffffu, inc - w, f);
            sh.cur.b = b0 + f;
            sh.cur.s = seq_plan<C>(p, __shfl_sync(0xffffffffu, len, f));
            break;
        }
        it -= __shfl_sync(0xffffffffu, inc, 31);
    }
    const int per = sh.cur.s.nc + sh.cur.s.nb + C::SEGS * SEG_COST;
    sh.cur.g = static_cast<int>(it / per);
    sh.cur.r = static_cast<int>(it % per);
    sh.cur.base = C::SEGS == 2 && sh.cur.r >= sh.cur.s.nc + SEG_COST;
    sh.cur.r -= sh.cur.base ? sh.cur.s.nc + SEG_COST : 0;
    return sh;
}

struct ServeMaps {
    CUtensorMap k, v, kp, vp;  // own cache; the prefix (prefix form)
};

template <int D, int G, int CODE>
__global__ void __launch_bounds__(SvCfg<D, G, CODE>::THREADS, 2)
    serve_step_kernel(const __grid_constant__ ServeMaps maps, const ServeParams p)
{
    using C = SvCfg<D, G, CODE>;
    constexpr bool Q8 = C::Q8, STEP = C::STEP;
    constexpr int NT = (G + 7) / 8;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_s = smem_u32(smem_raw);
    const uint32_t pad = ((raw_s + 1023u) & ~1023u) - raw_s;
    uint8_t *smem = smem_raw + pad;
    const uint32_t sbase = raw_s + pad;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);
    uint64_t *empty = full + C::STAGES;
    uint64_t *hfull = empty + C::STAGES, *hempty = hfull + C::HB;
    Join *joins = reinterpret_cast<Join *>(smem + C::JOIN_OFF);
    int *s_flag = reinterpret_cast<int *>(smem + C::FLAG_OFF);
    volatile int *s_abort = s_flag + 1;  // a wait has given up: the producer stops
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float NEG_INF = -__int_as_float(0x7f800000);

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], C::GROUP);
        }
        for (int s = 0; s < C::HB; ++s) {
            mbar_init(&hfull[s], 1);
            mbar_init(&hempty[s], C::CWARPS);
        }
        *s_abort = 0;
        fence_barrier_init();
    }
    // Programmatic dependent launch.  8-bit form: everything the step before wrote is waited for
    // here.  Prefix form: the prefix kernel waited for it before it let this grid start; its own
    // partials are waited for where they are read.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if constexpr (Q8)
        asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long c = blockIdx.x;
    const Share sh = plan_share<C>(p, c, gridDim.x);
    const long long W = sh.W, n = sh.n, it0 = sh.it0, it1 = sh.it1;
    Cursor cur = sh.cur;
    __syncthreads();  // barriers are set up, and every warp has read cache_len

    if (warp == C::CWARPS) {
        // ------------------------------------------------------------------ producer
        if (lane != 0)
            return;
        long long i = 0;
        int segs = 0;
        bool header = true;
        for (long long it = it0; it < it1; ++it) {
            if (cur.r < SEG_COST) {
                ++cur.r;
                continue;
            }
            if (header) {  // the segment's queries
                const int hb = segs % C::HB;
                if ((segs >= C::HB && !mbar_wait(&hempty[hb], static_cast<uint32_t>((segs / C::HB - 1) & 1))) ||
                    *s_abort) {
                    record_error(p.dev_err, ORTHROS_DEVERR_TIMEOUT);
                    drain_in_flight();
                    return;
                }
                uint8_t *h = smem + C::HDR_OFF + hb * C::HDR_BYTES;
                const long long go = static_cast<long long>(cur.g) * G * D;
                mbar_arrive_expect_tx(&hfull[hb], STEP ? C::HDR_BYTES : C::HDR_NEW);
                bulk_load(h, (cur.base ? p.q_new : p.qc_new) + cur.b * p.q_bstride + go, G * D * 2, &hfull[hb]);
                bulk_load(h + G * D * 2, (cur.base ? p.alpha : p.alpha_c) + go, G * D * 4, &hfull[hb]);
                bulk_load(h + G * D * 6, (cur.base ? p.beta : p.beta_c) + go, G * D * 4, &hfull[hb]);
                if constexpr (STEP) {
                    const long long no = (static_cast<long long>(cur.b) * p.Hkv + cur.g) * D;
                    bulk_load(h + C::HDR_NEW, p.k_new + no, D * 2, &hfull[hb]);
                    bulk_load(h + C::HDR_NEW + D * 2, p.v_new + no, D * 2, &hfull[hb]);
                }
                header = false;
                ++segs;
            }
            const int s = static_cast<int>(i % C::STAGES);
            if ((i >= C::STAGES && !mbar_wait(&empty[s], static_cast<uint32_t>(((i / C::STAGES) - 1) & 1))) || *s_abort) {
                record_error(p.dev_err, ORTHROS_DEVERR_TIMEOUT);
                drain_in_flight();
                return;
            }
            bool pre;
            const int blk = cur.block<C>(cur.r - SEG_COST, pre);
            const int j0 = blk * C::KB;
            uint8_t *dst = smem + s * 2 * C::KV_BYTES;
            if constexpr (Q8) {
                const int ne = min(C::KB, p.L_max - j0);  // a multiple of 16, as L_max is
                mbar_arrive_expect_tx(&full[s], 2 * C::KV_BYTES + 2 * ne);
                tma_load_4d(dst, &maps.k, &full[s], 0, cur.g, j0, cur.b);
                tma_load_4d(dst + C::KV_BYTES, &maps.v, &full[s], 0, cur.g, j0, cur.b);
                const long long eo = (static_cast<long long>(cur.b) * p.Hkv + cur.g) * p.L_max + j0;
                uint8_t *es = smem + C::EXP_OFF + s * 2 * C::KB;
                bulk_load(es, p.k_exp + eo, ne, &full[s]);
                bulk_load(es + C::KB, p.v_exp + eo, ne, &full[s]);
            } else {
                mbar_arrive_expect_tx(&full[s], 2 * C::KV_BYTES);
                const CUtensorMap *mk = pre ? &maps.kp : &maps.k, *mv = pre ? &maps.vp : &maps.v;
                const int bb = pre ? 0 : cur.b;
#pragma unroll
                for (int sl = 0; sl < D / 64; ++sl) {
                    tma_load_4d(dst + sl * C::SLAB, mk, &full[s], sl * 64, cur.g, j0, bb);
                    tma_load_4d(dst + C::KV_BYTES + sl * C::SLAB, mv, &full[s], sl * 64, cur.g, j0, bb);
                }
            }
            ++i;
            if (++cur.r == cur.places() && it + 1 < it1) {
                cur.next_segment<C>(p);
                header = true;
            }
        }
        return;
    }

    // ---------------------------------------------------------------------- consumers
    const int t = threadIdx.x;
    float *os = reinterpret_cast<float *>(smem + C::SCR_OFF);  // [CWARPS][G][D]
    float *ms = os + C::CWARPS * G * D, *ls = ms + C::CWARPS * G;
    float *vs = ls + C::CWARPS * G;  // codes: the scale of the warps' o
    bool ok = true, bad = false;
    long long i = 0;
    int segs = 0, njoin = 0;
    // Joins the segments on the list: each counts this CTA in (after its partials: the barrier orders
    // them before the fence), and those that it was the last to finish are joined, half a warp a row.
    // At the end of the CTA's work only, so that no wait for memory stands between two segments.
    auto join_all = [&](bool final) {
        // the prefix kernel's partials and, for SV_COPIES, the counters that it cleared; and the step
        // has ended only when that kernel has
        if constexpr (!Q8)
            asm volatile("griddepcontrol.wait;" ::: "memory");
        named_barrier(1, C::CTHREADS);
        if (t < njoin) {
            Join &j = joins[t];
            int *cnt = p.cnt_seg + j.c0;  // at most one segment runs out of a CTA
            __threadfence();
            j.last = j.parts == 1 || atomicAdd(cnt, 1) == j.parts - 1;
            __threadfence();
            if (j.parts > 1 && j.last)
                *cnt = 0;
        }
        if (STEP && final && t == C::CTHREADS - 1)  // every warp of this CTA has read cache_len for the last time
            s_flag[0] = atomicAdd(p.cnt_all, 1) == static_cast<int>(gridDim.x) - 1;
        named_barrier(1, C::CTHREADS);
        const long long BH = static_cast<long long>(p.B) * p.Hkv;
        // half a warp a row (or two halves, each every other part): E columns a lane, 16 parts' weights in
        // its lanes, 8 parts' loads in flight
        constexpr int E = D / 16;
        const int half = lane >> 4, hl = lane & 15, total = njoin * G, two = p.join_two;
        for (int x0 = warp << (1 - two); x0 < total; x0 += C::CWARPS << (1 - two)) {
            const int x = two ? x0 : x0 + half;
            const bool on = x < total;
            const Join j = joins[on ? x / G : 0];
            const int row = x % G;
            const bool base = j.base;
            // parts: the CTAs' own, then (a copy behind a prefix) the prefix splits'
            const int nown = j.parts;
            const int nall = on && j.last ? nown + (!Q8 && !base ? p.n_part : 0) : 0;
            const int nq = two ? (nall + 1 - half) / 2 : nall;  // this half's; its q-th is the row's part_of(q)
            auto part_of = [&](int q) { return two ? 2 * q + half : q; };
            const int nmax = max(nq, __shfl_xor_sync(0xffffffffu, nq, 16));
            if (nmax == 0)
                continue;
            auto slot_of = [&](int q) -> long long {
                return q < nown ? (j.parts == 1 ? 2LL * gridDim.x + j.bh
                                                : 2LL * (j.c0 + q) + (q == 0 ? 1 : 0)) * G + row
                                : ((q - nown) * BH + j.bh) * G + row;
            };
            auto ml_of = [&](int q) -> float2 {
                if (q >= nq)
                    return make_float2(NEG_INF, 0.f);
                q = part_of(q);
                return __ldcg((q < nown ? p.part_ml : p.pre_ml) + slot_of(q));
            };
            float y[8][E];
            auto load = [&](int q0) {  // past the end the last part again: its weight there is zero
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int q = part_of(min(q0 + k, nq - 1));
#pragma unroll
                    for (int e = 0; e < E; e += 4) {
                        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (nq > 0)
                            v = __ldcg(reinterpret_cast<const float4 *>((q < nown ? p.part_o : p.pre_o) + slot_of(q) * D +
                                                                        hl * E + e));
                        y[k][e] = v.x;
                        y[k][e + 1] = v.y;
                        y[k][e + 2] = v.z;
                        y[k][e + 3] = v.w;
                    }
                }
            };
            float2 ml = ml_of(hl);
            load(0);
            float M = ml.x, L = 0.f, w = 0.f;
            for (int q = hl + 16; q < nq; q += 16)
                M = fmaxf(M, ml_of(q).x);
#pragma unroll
            for (int off = 8; off > 0; off >>= 1)
                M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
            if (two)
                M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
            float a[E];
#pragma unroll
            for (int e = 0; e < E; ++e)
                a[e] = 0.f;
            for (int q0 = 0; q0 < nmax; q0 += 8) {
                if (q0 % 16 == 0) {
                    if (q0 > 0)
                        ml = ml_of(q0 + hl);
                    w = ml.y == 0.f ? 0.f : fast_exp2(ml.x - M);  // a NaN reaches the output
                    L += w * ml.y;
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float wk = __shfl_sync(0xffffffffu, w, 16 * half + q0 % 16 + k);
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        a[e] = fmaf(wk, y[k][e], a[e]);
                }
                if (q0 + 8 < nmax)
                    load(q0 + 8);
            }
#pragma unroll
            for (int off = 8; off > 0; off >>= 1)
                L += __shfl_xor_sync(0xffffffffu, L, off);
            if (two) {
                L += __shfl_xor_sync(0xffffffffu, L, 16);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    a[e] += __shfl_xor_sync(0xffffffffu, a[e], 16);
            }
            const float inv = L > 0.f ? 1.f / L : 0.f;
            orthros_bf16 *orow = (base ? p.o : p.oc) + (j.bh / p.Hkv) * p.o_bstride +
                                 ((j.bh % p.Hkv) * G + row) * D + hl * E;
            if (nq > 0 && !(two && half)) {
#pragma unroll
                for (int e = 0; e < E; e += 4)
                    *reinterpret_cast<uint2 *>(orow + e) = make_uint2(pack_bf16x2(a[e] * inv, a[e + 1] * inv),
                                                                      pack_bf16x2(a[e + 2] * inv, a[e + 3] * inv));
            }
        }
        njoin = 0;
        named_barrier(1, C::CTHREADS);  // the list may be filled again
    };
    for (long long it = it0; it < it1;) {
        const int b = cur.b, g = cur.g, seg_places = cur.places();
        const SeqPlan sp = cur.s;
        const int places = static_cast<int>(seg_places - cur.r < it1 - it ? seg_places - cur.r : it1 - it);
        const int first = max(cur.r - SEG_COST, 0), m = cur.r + places - SEG_COST - first;  // blocks first .. first + m - 1
        if (m <= 0) {  // the CTA's last places are a segment's empty ones
            it += places;
            continue;
        }
        typename std::conditional<Q8, WarpQ8<D, NT, Q8 ? CODE : 0>, WarpB16<D, NT>>::type st;
        {
            const int hb = segs % C::HB;
            if (ok && !mbar_wait(&hfull[hb], static_cast<uint32_t>((segs / C::HB) & 1)))
                ok = false, *s_abort = 1;
            const orthros_bf16 *q = reinterpret_cast<const orthros_bf16 *>(smem + C::HDR_OFF + hb * C::HDR_BYTES);
            const float *al = reinterpret_cast<const float *>(q + G * D), *be = al + G * D;
            st.load_q(q, al, be, G, p.qscale);
        }
        // the new rows as this lane takes them: lanes 0 .. 15 of K's, 16 .. 31 of V's, D / 16 values each
        const int kv = lane >> 4;
        uint32_t fresh_w[D / 32];
        if constexpr (STEP) {
            const uint32_t *src = reinterpret_cast<const uint32_t *>(smem + C::HDR_OFF + (segs % C::HB) * C::HDR_BYTES +
                                                                     C::HDR_NEW) + lane * (D / 32);
#pragma unroll
            for (int e = 0; e < D / 32; ++e)
                fresh_w[e] = src[e];
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&hempty[segs % C::HB]);
        ++segs;
        st.reset();
        for (int x = 0; x < m; ++x, ++i) {
            if (C::KT == 2 && (i & 1) != (warp >> 1))
                continue;  // the other pair's block
            const int s = static_cast<int>(i % C::STAGES);
            bool pre;
            const int blk = cur.block<C>(first + x, pre);
            // the block's rows that count: lo .. hi
            const int lo = (cur.base ? (pre ? sp.lo_p : sp.lo) : 0) - blk * C::KB, hi = (pre ? p.P - 1 : sp.p) - blk * C::KB;
            if (ok && !mbar_wait(&full[s], static_cast<uint32_t>((i / C::STAGES) & 1)))
                ok = false, *s_abort = 1;
            constexpr int WK = 16 * C::KT;  // this warp's keys: rows r0 .. r0 + WK - 1 of the block
            const int r0 = (warp % C::GROUP) * WK;
            if (ok && !sp.full && r0 <= hi && r0 + WK - 1 >= lo) {
                uint8_t *kb = smem + s * 2 * C::KV_BYTES, *vb = kb + C::KV_BYTES;
                int8_t *ke = reinterpret_cast<int8_t *>(smem + C::EXP_OFF + s * 2 * C::KB), *ve = ke + C::KB;
                bool patched = false;
                // V rows that do not count become zeros: their weight is zero, but they may hold anything
                // (before the window, and behind the last row, which no token has reached)
                auto zero_rows = [&](int from, int to) {
                    constexpr int CH = D * (Q8 ? 1 : 2) / 16;  // 16-byte chunks of a row
                    from = max(from, r0);
                    to = min(to, r0 + WK);
#pragma unroll 1
                    for (int e = lane; e < (to - from) * CH; e += 32) {
                        const int rr = from + e / CH, c16 = e % CH;
                        uint8_t *dst;
                        if constexpr (Q8) {
                            dst = vb + q8_offset<D>(rr, c16);
                            if (c16 == 0)
                                ve[rr] = -127;
                        } else {
                            dst = vb + (c16 / 8) * C::SLAB + sw128_offset(rr, c16 % 8);
                        }
                        *reinterpret_cast<uint4 *>(dst) = make_uint4(0, 0, 0, 0);
                    }
                    patched = true;
                };
                if (hi < r0 + WK - 1)
                    zero_rows(hi + 1, r0 + WK);
                if (lo > r0)
                    zero_rows(r0, lo);
                if (STEP && !pre && hi < r0 + WK) {  // the new row goes where it belongs
                    const long long row = (static_cast<long long>(b) * p.L_max + sp.p) * p.Hkv + g;
                    const bool append = !cur.base;
                    if constexpr (Q8) {
                        constexpr int E = D / 16;
                        float f[E], amax = 0.f;
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            const float2 two = unpack_bf16x2(fresh_w[e / 2]);
                            f[e] = (e & 1) ? two.y : two.x;
                            if (fabsf(f[e]) < __int_as_float(0x7f800000))
                                amax = fmaxf(amax, fabsf(f[e]));
                            else
                                bad = true;
                        }
#pragma unroll
                        for (int off = 8; off > 0; off >>= 1)
                            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
                        const int ex = q8_exponent<Q8 ? CODE : 0>(amax);
                        const float sd = q8_pow2(-ex);
                        uint32_t w[E / 4];
#pragma unroll
                        for (int e = 0; e < E; e += 4)
                            w[e / 4] = q8_codes2<Q8 ? CODE : 0>(f[e] * sd, f[e + 1] * sd) |
                                       q8_codes2<Q8 ? CODE : 0>(f[e + 2] * sd, f[e + 3] * sd) << 16;
                        const int d = E * (lane & 15);
                        uint8_t *to = (kv ? vb : kb) + q8_offset<D>(hi, d / 16) + d % 16;
                        uint8_t *cache = static_cast<uint8_t *>(kv ? p.v_cache : p.k_cache) + row * D + d;
#pragma unroll
                        for (int e = 0; e < E / 4; ++e) {
                            reinterpret_cast<uint32_t *>(to)[e] = w[e];
                            if (append)
                                reinterpret_cast<uint32_t *>(cache)[e] = w[e];
                        }
                        if ((lane & 15) == 0) {
                            (kv ? ve : ke)[hi] = static_cast<int8_t>(ex);
                            if (append)
                                (kv ? p.v_exp : p.k_exp)[(static_cast<long long>(b) * p.Hkv + g) * p.L_max + sp.p] =
                                    static_cast<int8_t>(ex);
                        }
                    } else {
                        const int d = (D / 16) * (lane & 15);
                        uint8_t *to = (kv ? vb : kb) + (d / 64) * C::SLAB + sw128_offset(hi, d % 64 / 8) + d % 8 * 2;
                        orthros_bf16 *cache = static_cast<orthros_bf16 *>(kv ? p.v_cache : p.k_cache) + row * D + d;
#pragma unroll
                        for (int e = 0; e < D / 32; ++e) {
                            reinterpret_cast<uint32_t *>(to)[e] = fresh_w[e];
                            if (append)
                                reinterpret_cast<uint32_t *>(cache)[e] = fresh_w[e];
                        }
                    }
                    patched = true;
                }
                if (patched)
                    __syncwarp();
                const bool whole = lo <= r0 && r0 + WK - 1 <= hi;
                if constexpr (Q8) {
                    st.template step<C::KT>(kb, vb, ke, ve, r0, whole, lo, hi);
                } else {
                    const uint32_t ks = sbase + s * 2 * C::KV_BYTES;
                    st.template step<C::KT>(ks, ks + C::KV_BYTES, C::SLAB, r0, whole, lo, hi);
                }
                if (patched)
                    fence_proxy_async_smem();  // before TMA writes over what was patched
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&empty[s]);
        }
        st.finish_sums();

        // ---- the four warps' results meet in shared memory
        named_barrier(1, C::CTHREADS);  // the segment before has been read
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r2 = 0; r2 < 2; ++r2) {
                const int row = 8 * nt + 2 * (lane & 3) + r2, gq = lane >> 2;
                if (row >= G)
                    continue;
                if (gq == 0) {
                    ms[warp * G + row] = st.m[nt][r2];
                    ls[warp * G + row] = st.l[nt][r2];
                    if constexpr (Q8)
                        vs[warp * G + row] = st.mv[nt][r2];
                }
                float *po = os + (warp * G + row) * D;
#pragma unroll
                for (int mt = 0; mt < D / 16; ++mt)
                    if constexpr (Q8) {
                        *reinterpret_cast<float2 *>(po + (D / 8) * gq + 2 * mt) =
                            make_float2(st.o[nt][mt][r2], st.o[nt][mt][2 + r2]);
                    } else {
                        po[16 * mt + gq] = st.o[nt][mt][r2];
                        po[16 * mt + gq + 8] = st.o[nt][mt][2 + r2];
                    }
            }
        named_barrier(1, C::CTHREADS);
        // segment bounds in the list, and who else has a share
        const long long s0 = it - cur.r + SEG_COST, s1 = it - cur.r + seg_places;
        const long long c0 = ((s0 + 1) * n - 1) / W, c1 = (s1 * n - 1) / W;  // owners of its first and last block
        const bool joins_prefix = !Q8 && !cur.base && !sp.full;
        const bool alone = c0 == c1 && !joins_prefix;
        // one slot for a segment that began before this CTA, one for one that runs out of it, and one
        // for each copy that only the prefix has to be joined with
        const long long slot = c0 == c1 ? 2LL * gridDim.x + static_cast<long long>(b) * p.Hkv + g : 2 * c + (c == c0 ? 1 : 0);
        for (int e = t; e < G * (D / 4); e += C::CTHREADS) {
            const int row = e / (D / 4), d4 = 4 * (e % (D / 4));
            float M = NEG_INF, L = 0.f;
#pragma unroll
            for (int w = 0; w < C::CWARPS; ++w)
                M = fmaxf(M, ms[w * G + row]);
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < C::CWARPS; ++w) {
                const float lw = ls[w * G + row];
                if (lw == 0.f)  // no key (a NaN has a sum of NaN, and goes on)
                    continue;
                float f = fast_exp2(ms[w * G + row] - M);
                L += f * lw;
                if constexpr (Q8) {  // o stands for o 2^(mv - 6); in two factors, as 2^(mv - 6 - M) can pass fp32's range
                    f = fast_exp2(0.5f * (vs[w * G + row] - 6.f - M));
                    const float4 y = *reinterpret_cast<const float4 *>(os + (w * G + row) * D + d4);
                    a.x += f * (f * y.x);
                    a.y += f * (f * y.y);
                    a.z += f * (f * y.z);
                    a.w += f * (f * y.w);
                } else {
                    const float4 y = *reinterpret_cast<const float4 *>(os + (w * G + row) * D + d4);
                    a.x += f * y.x;
                    a.y += f * y.y;
                    a.z += f * y.z;
                    a.w += f * y.w;
                }
            }
            if (alone) {
                const float inv = L > 0.f ? 1.f / L : 0.f;
                orthros_bf16 *out = (cur.base ? p.o : p.oc) + b * p.o_bstride + (g * G + row) * D + d4;
                *reinterpret_cast<uint2 *>(out) =
                    make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
            } else {
                *reinterpret_cast<float4 *>(p.part_o + (slot * G + row) * D + d4) = a;
                if (d4 == 0)
                    p.part_ml[slot * G + row] = make_float2(M, L);
            }
        }
        if (sp.full && !cur.base && g == 0 && t == 0)
            record_error(p.dev_err, STEP ? ORTHROS_DEVERR_CACHE_FULL : ORTHROS_DEVERR_POSITION);
        if (!alone && !p.join_after) {
            if (t == 0)
                joins[njoin] = {b * p.Hkv + g, cur.base, static_cast<int>(c0), static_cast<int>(c1 - c0) + 1, 0, 0};
            if (++njoin == MAX_JOINS)
                join_all(false);
        }
        it += places;
        cur.r += places;
        if (cur.r == seg_places && it < it1)
            cur.next_segment<C>(p);
    }
    if (bad)
        record_error(p.dev_err, ORTHROS_DEVERR_RANGE);
    if (!ok) {
        if (lane == 0)
            record_error(p.dev_err, ORTHROS_DEVERR_TIMEOUT);
        drain_in_flight();
    }
    if (p.join_after) {  // serve_join_kernel joins the partials and advances the lengths
        if constexpr (!Q8)
            asm volatile("griddepcontrol.wait;" ::: "memory");  // it waits for this grid, and the prefix kernel's too
        return;
    }
    join_all(true);
    // the last CTA of the grid advances the lengths: every one has read them by now
    if (STEP && s_flag[0]) {
        for (int b = t; b < p.B; b += C::CTHREADS) {
            const int len = __ldcg(p.cache_len + b);
            if (len >= 0 && len < p.L_max)
                p.cache_len[b] = len + 1;
        }
        if (t == 0)
            *p.cnt_all = 0;
    }
}

// Many parts of few segments (a long cache or prefix of one KV head over all SMs): one CTA a row, its
// eight half-warps take every eighth part each.  The CTAs that held a segment are found by the same
// arithmetic as in the step.  The last CTA advances the lengths.
template <int D, int G, int CODE>
__global__ void __launch_bounds__(128) serve_join_kernel(const ServeParams p, int ctas)
{
    using C = SvCfg<D, G, CODE>;
    constexpr int E = D / 16;
    __shared__ float red_s[4], o_s[8][D];
    __shared__ int last_s;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, hw = t >> 4, hl = t & 15;
    const int row = blockIdx.x % G, base = blockIdx.x / G % C::SEGS, bh = blockIdx.x / (G * C::SEGS);
    const int b = bh / p.Hkv, g = bh % p.Hkv;
    const float NEG_INF = -__int_as_float(0x7f800000);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    long long W = 0, before = 0;  // places of the list, and those before sequence b
    for (int i = lane; i < p.B; i += 32) {
        const long long w = seq_places<C>(p, __ldcg(p.cache_len + i));
        W += w;
        before += i < b ? w : 0;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        W += __shfl_xor_sync(0xffffffffu, W, off);
        before += __shfl_xor_sync(0xffffffffu, before, off);
    }
    const SeqPlan sp = seq_plan<C>(p, __ldcg(p.cache_len + b));
    const long long n = ctas < W ? ctas : W;
    const long long s0 = before + static_cast<long long>(sp.nc + sp.nb + C::SEGS * SEG_COST) * g + SEG_COST +
                         (base ? sp.nc + SEG_COST : 0);
    const long long s1 = s0 + (base ? sp.nb : sp.nc);
    const long long c0 = ((s0 + 1) * n - 1) / W, c1 = (s1 * n - 1) / W;
    // what one CTA held whole is written already, but for a copy that the prefix has to be joined with
    const bool joins_prefix = !C::Q8 && !base && !sp.full;
    if (c0 != c1 || joins_prefix) {
        const int nown = static_cast<int>(c1 - c0) + 1, nq = nown + (joins_prefix ? p.n_part : 0);
        const long long BH = static_cast<long long>(p.B) * p.Hkv;
        auto slot_of = [&](int q) -> long long {
            return q < nown ? (c0 == c1 ? 2LL * ctas + bh : 2LL * (c0 + q) + (q == 0 ? 1 : 0)) * G + row
                            : ((q - nown) * BH + bh) * G + row;
        };
        auto ml_of = [&](int q) -> float2 { return __ldcg((q < nown ? p.part_ml : p.pre_ml) + slot_of(q)); };
        float M = NEG_INF;
        for (int q = t; q < nq; q += 128)
            M = fmaxf(M, ml_of(q).x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        if (lane == 0)
            red_s[warp] = M;
        __syncthreads();
        M = fmaxf(fmaxf(red_s[0], red_s[1]), fmaxf(red_s[2], red_s[3]));
        float L = 0.f, a[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            a[e] = 0.f;
        for (int q0 = hw; q0 < nq; q0 += 64) {
            float2 ml[8];
            float4 y[8][E / 4];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int q = q0 + 8 * k;
                ml[k] = make_float2(NEG_INF, 0.f);
                if (q < nq) {
                    ml[k] = ml_of(q);
                    const float *src = (q < nown ? p.part_o : p.pre_o) + slot_of(q) * D + hl * E;
#pragma unroll
                    for (int e = 0; e < E / 4; ++e)
                        y[k][e] = __ldcg(reinterpret_cast<const float4 *>(src) + e);
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (ml[k].y == 0.f)
                    continue;
                const float w = fast_exp2(ml[k].x - M);
                L += w * ml[k].y;
#pragma unroll
                for (int e = 0; e < E / 4; ++e) {
                    a[4 * e] = fmaf(w, y[k][e].x, a[4 * e]);
                    a[4 * e + 1] = fmaf(w, y[k][e].y, a[4 * e + 1]);
                    a[4 * e + 2] = fmaf(w, y[k][e].z, a[4 * e + 2]);
                    a[4 * e + 3] = fmaf(w, y[k][e].w, a[4 * e + 3]);
                }
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e)
            o_s[hw][hl * E + e] = a[e];
        __syncthreads();  // red_s has been read, o_s is complete
        L += __shfl_xor_sync(0xffffffffu, L, 16);  // all lanes of a half-warp hold its sum
        if (lane == 0)
            red_s[warp] = L;
        __syncthreads();
        L = (red_s[0] + red_s[1]) + (red_s[2] + red_s[3]);
        const float inv = L > 0.f ? 1.f / L : 0.f;
        if (t < D) {
            float x = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x += o_s[i][t];
            (base ? p.o : p.oc)[b * p.o_bstride + (g * G + row) * D + t] = __bfloat16_as_ushort(__float2bfloat16_rn(x * inv));
        }
    }
    if constexpr (C::STEP) {
        __syncthreads();  // every warp has read cache_len
        if (t == 0)
            last_s = atomicAdd(p.cnt_all, 1) == static_cast<int>(gridDim.x) - 1;
        __syncthreads();
        if (last_s) {
            for (int i = t; i < p.B; i += 128) {
                const int len = __ldcg(p.cache_len + i);
                if (len >= 0 && len < p.L_max)
                    p.cache_len[i] = len + 1;
            }
            if (t == 0)
                *p.cnt_all = 0;
        }
    }
}

// ------------------------------------------------------------------ host side

struct ServeLayout {
    int ctas;
    size_t part_o, part_ml, pre_o, pre_ml, total;
};

// the grid: never more CTAs than the longest caches could give places
static ServeLayout serve_layout(int B, int P, int L_max, int Hq, int Hkv, int D)
{
    const size_t G = Hq / Hkv, BH = static_cast<size_t>(B) * Hkv;
    const size_t most = 2 * BH * ((static_cast<size_t>(L_max) + 63) / 64 + (static_cast<size_t>(P) + 63) / 64 + SEG_COST);
    ServeLayout l;
    l.ctas = static_cast<int>(most < SERVE_CTAS ? most : SERVE_CTAS);
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t slots = (2 * static_cast<size_t>(l.ctas) + (P > 0 ? BH : 0)) * G;
    l.part_o = up((SERVE_CTAS + 1) * sizeof(int));  // the counters come first, for any sizes
    l.part_ml = l.part_o + up(slots * D * sizeof(float));
    l.pre_o = l.part_ml + up(slots * sizeof(float2));
    const size_t pre = P > 0 ? static_cast<size_t>(prefix_attn_parts(B, P, Hq, Hkv)) * BH * G : 0;
    l.pre_ml = l.pre_o + up(pre * D * sizeof(float));
    l.total = l.pre_ml + up(pre * sizeof(float2));
    return l;
}

size_t serve_workspace_bytes(int B, int P, int L_max, int Hq, int Hkv, int D)
{
    return serve_layout(B, P, L_max, Hq, Hkv, D).total;
}

// A join inside the step costs the CTA that does it 8.5 ns a part and row at d = 128 (one SM reads all of
// them, 60 GB/s); a kernel of its own costs 3 us, whatever their number.  With one KV head of 16 query
// heads and 4 sequences (76 parts a copy) the step took 57 us with the join inside.
static bool join_after(const ServeParams &p, long long parts, int D) { return parts * (p.Hq / p.Hkv) * D >= 45000; }

template <int D, int G, int CODE>
static cudaError_t launch_serve_tc(const ServeMaps &maps, ServeParams p, int ctas, cudaStream_t stream)
{
    using C = SvCfg<D, G, CODE>;
    auto kern = serve_step_kernel<D, G, CODE>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess)
        return e;
    const long long parts = ctas / (static_cast<long long>(p.B) * p.Hkv) + p.n_part;  // about, of a long segment
    p.join_after = join_after(p, parts, D);
    // Two half-warps a row where rows are few and their partials many.  Steps with one and with two, us on one
    // GB300: 4 sequences behind 16384 rows (2 heads, d = 64) 19.6, 15.2; 4 behind 131072 (8 heads, d = 128) 99.4, 97.0;
    // codes, 2 x 131072 rows 91.2, 89.9; but 64 behind 16384 (7 rows a CTA) 64.2, 65.4.
    p.join_two = parts > 8 && static_cast<long long>(p.B) * p.Hq <= 4LL * ctas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, maps, p);
    if (e == cudaSuccess && p.join_after) {
        cfg.gridDim = dim3(static_cast<unsigned>(p.B) * p.Hkv * C::SEGS * G);
        cfg.blockDim = dim3(128);
        cfg.dynamicSmemBytes = 0;
        e = cudaLaunchKernelEx(&cfg, serve_join_kernel<D, G, CODE>, p, ctas);
    }
    return e == cudaSuccess ? cudaGetLastError() : e;
}

template <int D, int G>
static cudaError_t launch_serve_t(int code, const ServeMaps &maps, const ServeParams &p, int ctas, cudaStream_t stream)
{
    if (code == ORTHROS_KV_E4M3)
        return launch_serve_tc<D, G, ORTHROS_KV_E4M3>(maps, p, ctas, stream);
    if (code == ORTHROS_KV_INT8)
        return launch_serve_tc<D, G, ORTHROS_KV_INT8>(maps, p, ctas, stream);
    if (code == SV_PREFIX)
        return launch_serve_tc<D, G, SV_PREFIX>(maps, p, ctas, stream);
    return launch_serve_tc<D, G, SV_COPIES>(maps, p, ctas, stream);
}

static cudaError_t launch_any(int D, int code, const CUtensorMap *m, ServeParams p, void *workspace, cudaStream_t stream)
{
    const bool step = code != SV_COPIES;
    const ServeLayout l = serve_layout(p.B, p.P, p.L_max, p.Hq, p.Hkv, D);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.cnt_seg = reinterpret_cast<int *>(ws);
    p.cnt_all = p.cnt_seg + SERVE_CTAS;
    p.part_o = reinterpret_cast<float *>(ws + l.part_o);
    p.part_ml = reinterpret_cast<float2 *>(ws + l.part_ml);
    p.pre_o = reinterpret_cast<float *>(ws + l.pre_o);
    p.pre_ml = reinterpret_cast<float2 *>(ws + l.pre_ml);
    if (p.P > 0) {
        PrefixAttnParams a{};
        a.qc = p.qc_new;
        a.alpha_c = p.alpha_c;
        a.beta_c = p.beta_c;
        a.part_o = p.pre_o;
        a.part_ml = p.pre_ml;
        a.dev_err = p.dev_err;
        a.qc_bstride = p.q_bstride;
        a.B = p.B;
        a.T_out = 1;
        a.P = p.P;
        a.Hq = p.Hq;
        a.Hkv = p.Hkv;
        a.qscale = p.qscale;
        if (!step) {  // its workspace comes as it is: the prefix kernel clears the counters
            a.clear = p.cnt_seg;
            a.n_clear = SERVE_CTAS;
        }
        const cudaError_t e = launch_prefix_attn(D, m[2], m[3], a, stream);
        if (e != cudaSuccess)
            return e;
        p.n_part = prefix_attn_parts(p.B, p.P, p.Hq, p.Hkv);
    }
    const ServeMaps maps = {m[0], m[1], m[2], m[3]};
    const int G = p.Hq / p.Hkv;
#define ORTHROS_SERVE_CASE(DD, GG) \
    if (D == DD && G == GG)        \
        return launch_serve_t<DD, GG>(code, maps, p, l.ctas, stream);
    ORTHROS_SERVE_CASE(128, 1)
    ORTHROS_SERVE_CASE(128, 2)
    ORTHROS_SERVE_CASE(128, 4)
    ORTHROS_SERVE_CASE(128, 8)
    ORTHROS_SERVE_CASE(128, 16)
    ORTHROS_SERVE_CASE(64, 1)
    ORTHROS_SERVE_CASE(64, 2)
    ORTHROS_SERVE_CASE(64, 4)
    ORTHROS_SERVE_CASE(64, 8)
    ORTHROS_SERVE_CASE(64, 16)
#undef ORTHROS_SERVE_CASE
    return cudaErrorInvalidValue;
}

cudaError_t launch_serve(int D, int code, const CUtensorMap *maps, ServeParams p, void *workspace, cudaStream_t stream)
{
    p.q_bstride = p.o_bstride = static_cast<long long>(p.Hq) * D;
    return launch_any(D, code, maps, p, workspace, stream);
}

cudaError_t launch_serve_copies(int D, const CUtensorMap *maps, const XattnParams &x, int P, void *workspace,
                                cudaStream_t stream)
{
    ServeParams p{};
    p.qc_new = x.qc;
    p.cache_len = const_cast<int32_t *>(x.pos);  // read only in this form
    p.alpha_c = x.alpha_c;
    p.beta_c = x.beta_c;
    p.oc = x.oc;
    p.q_bstride = x.qc_bstride;
    p.o_bstride = x.oc_bstride;
    p.dev_err = x.dev_err;
    p.B = x.B;
    p.Hq = x.Hq;
    p.Hkv = x.Hkv;
    p.L_max = x.T_kv;
    p.window = 1;
    p.P = P;
    p.qscale = x.qscale;
    return launch_any(D, SV_COPIES, maps, p, workspace, stream);
}

}  // namespace orthros
