// serve_step.cu -- one decode step over an 8-bit KV cache, or over a prompt prefix that the
// whole batch shares and each sequence's own bf16 cache.  Per sequence with p = cache_len[b]:
//   append k_new / v_new at own row p (as codes in the 8-bit form),
//   o  = Eq. (4) for the new base token over its last `window` rows,
//   oc = Eq. (5) for its output copy over every row (prefix, own rows, the new one),
//   cache_len[b] = p + 1.
//
// The work of a step is a list of segments, two for each (b, KV head): the copy's own rows
// 0 .. p, and the base token's window (which in the prefix form may begin in the prefix).  Each
// is a run of 64-key blocks; laid end to end they form one list of W blocks, and CTA c of n takes
// blocks floor(c W / n) .. floor((c + 1) W / n) - 1, whatever sequence they belong to: a ragged
// batch loads every SM alike.  A CTA's blocks arrive by TMA through a ring that runs on across
// segment borders (one producer warp), four warps take 16 keys of a block each, with the G query
// rows of a KV head on the MMA's N side, and their results meet in shared memory.  A segment that
// one CTA holds whole is written out at once; otherwise each CTA writes one partial (max, sum,
// o) and the last to arrive joins them (a counter, no spin).  Partials are bounded by the grid
// (two a CTA: one segment can run in from the CTA before, one can run out), not by the batch.
//
// The block that holds row p is patched in shared memory by the warp that owns the rows: the
// new row goes in, rows behind it (whatever the cache holds there) become zeros.  The last CTA
// of the grid to finish advances cache_len.
//
// In the prefix form the copy's attention over the prefix itself runs in a kernel of its own
// before this one, for all rows of the batch at once (prefix_attn.cu); this kernel is launched as
// its programmatic dependent and waits for it only where it joins a copy's partials.
#include <type_traits>

#include "kernels.cuh"
#include "warp_q8.cuh"
#include "xattn.cuh"

namespace orthros {

constexpr int SERVE_CTAS = 304;  // two on each of 152 SMs

template <int D, int G, int CODE>
struct SvCfg {
    static constexpr bool Q8 = CODE >= 0;
    static constexpr int KB = 64;
    static constexpr int KV_BYTES = KB * D * (Q8 ? 1 : 2);
    static constexpr int SLAB = KB * 128;  // bf16: one 64-wide slab
    static constexpr int SCR_ROWS = 4 * G;
    static constexpr int SCR_BYTES = SCR_ROWS * (D + 3) * 4;  // four warps' o, max, sum, exponent
    static constexpr int LIMIT = 112 * 1024 - 2048;            // two CTAs share an SM
    static constexpr int FIT = (LIMIT - SCR_BYTES) / (2 * KV_BYTES + 2 * KB);
    static constexpr int STAGES = FIT < 2 ? 2 : (FIT > 8 ? 8 : FIT);
    static constexpr int EXP_OFF = STAGES * 2 * KV_BYTES;
    static constexpr int SCR_OFF = EXP_OFF + STAGES * 2 * KB;
    static constexpr int BAR_OFF = SCR_OFF + SCR_BYTES;
    static constexpr int FLAG_OFF = BAR_OFF + 2 * STAGES * 8;
    static constexpr int SMEM = FLAG_OFF + 16 + 1024;
    static constexpr int CWARPS = 4;
    static constexpr int CTHREADS = CWARPS * 32;
    static constexpr int THREADS = CTHREADS + 32;
};

// what a sequence's cache_len makes of it
struct SeqPlan {
    int p;         // the new token's own row
    int full;      // nothing fits: zero outputs, no append
    int nc, nb;    // blocks of the copy's and of the base token's segment
    int npb;       // base blocks in the prefix (they come first)
    int pb0, ob0;  // their first block, and the first own block
    int lo_p, lo;  // first prefix row and first own row of the window
};

__device__ __forceinline__ SeqPlan seq_plan(const ServeParams &p, int b)
{
    SeqPlan s;
    s.p = __ldcg(p.cache_len + b);
    s.full = s.p < 0 || s.p >= p.L_max;
    s.npb = s.pb0 = s.ob0 = s.lo_p = s.lo = 0;
    s.nc = s.nb = 1;
    if (!s.full) {
        const int lo = s.p - p.window + 1;  // window >= 1, p >= 0: no overflow
        s.lo = lo > 0 ? lo : 0;
        s.ob0 = s.lo / 64;
        s.nc = s.p / 64 + 1;
        s.nb = s.nc - s.ob0;
        if (p.P > 0 && lo < 0) {
            s.lo_p = p.P + lo > 0 ? p.P + lo : 0;
            s.pb0 = s.lo_p / 64;
            s.npb = (p.P - 1) / 64 + 1 - s.pb0;
            s.nb += s.npb;
        }
    }
    return s;
}

// a position in the list of blocks: block r of segment (b, g, base)
struct Cursor {
    int b, g, base, r;
    SeqPlan s;
    __device__ __forceinline__ int blocks() const { return base ? s.nb : s.nc; }
    __device__ __forceinline__ void next_segment(const ServeParams &p)
    {
        r = 0;
        if (!base) {
            base = 1;
            return;
        }
        base = 0;
        if (++g == p.Hkv) {
            g = 0;
            if (++b < p.B)
                s = seq_plan(p, b);
        }
    }
};

// Called by a whole warp: W, and the cursor of block `it0(W)`.
__device__ __forceinline__ long long plan_total(const ServeParams &p)
{
    const int lane = threadIdx.x & 31;
    long long w = 0;
    for (int b = lane; b < p.B; b += 32) {
        const SeqPlan s = seq_plan(p, b);
        w += static_cast<long long>(s.nc + s.nb) * p.Hkv;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        w += __shfl_xor_sync(0xffffffffu, w, off);
    return w;
}

__device__ __forceinline__ Cursor plan_locate(const ServeParams &p, long long it)
{
    const int lane = threadIdx.x & 31;
    Cursor c;
    c.b = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        long long w = 0;
        if (b0 + lane < p.B) {
            const SeqPlan s = seq_plan(p, b0 + lane);
            w = static_cast<long long>(s.nc + s.nb) * p.Hkv;
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
            c.b = b0 + f;
            break;
        }
        it -= __shfl_sync(0xffffffffu, inc, 31);
    }
    c.s = seq_plan(p, c.b);
    const int per = c.s.nc + c.s.nb;
    c.g = static_cast<int>(it / per);
    c.r = static_cast<int>(it % per);
    c.base = c.r >= c.s.nc;
    c.r -= c.base ? c.s.nc : 0;
    return c;
}

struct ServeMaps {
    CUtensorMap k, v, kp, vp;  // own cache; the prefix (prefix form)
};

template <int D, int G, int CODE>
__global__ void __launch_bounds__(SvCfg<D, G, CODE>::THREADS, 2)
    serve_step_kernel(const __grid_constant__ ServeMaps maps, const ServeParams p)
{
    using C = SvCfg<D, G, CODE>;
    constexpr bool Q8 = C::Q8;
    constexpr int NT = (G + 7) / 8;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_s = smem_u32(smem_raw);
    const uint32_t pad = ((raw_s + 1023u) & ~1023u) - raw_s;
    uint8_t *smem = smem_raw + pad;
    const uint32_t sbase = raw_s + pad;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);
    uint64_t *empty = full + C::STAGES;
    int *s_flag = reinterpret_cast<int *>(smem + C::FLAG_OFF);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float NEG_INF = -__int_as_float(0x7f800000);

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], C::CWARPS);
        }
        fence_barrier_init();
    }
    // Programmatic dependent launch.  8-bit form: everything the step before wrote is waited for
    // here.  Prefix form: the prefix kernel waited for it before it let this grid start; its own
    // partials are waited for where they are read.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if constexpr (Q8)
        asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long W = plan_total(p);
    const long long n = gridDim.x < W ? gridDim.x : W;  // CTAs with work (every one then has a block)
    const long long c = blockIdx.x;
    const long long it0 = c < n ? c * W / n : W, it1 = c < n ? (c + 1) * W / n : W;
    Cursor cur{};
    if (it0 < it1)
        cur = plan_locate(p, it0);
    __syncthreads();  // barriers are set up, and every warp has read cache_len

    if (warp == C::CWARPS) {
        // ------------------------------------------------------------------ producer
        if (lane != 0)
            return;
        long long i = 0;
        for (long long it = it0; it < it1; ++it, ++i) {
            const int s = static_cast<int>(i % C::STAGES);
            if (i >= C::STAGES && !mbar_wait(&empty[s], static_cast<uint32_t>(((i / C::STAGES) - 1) & 1))) {
                record_error(p.dev_err, ORTHROS_DEVERR_TIMEOUT);
                return;
            }
            const bool pre = cur.base && cur.r < cur.s.npb;
            const int blk = cur.base ? (pre ? cur.s.pb0 + cur.r : cur.s.ob0 + cur.r - cur.s.npb) : cur.r;
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
            if (++cur.r == cur.blocks() && it + 1 < it1)
                cur.next_segment(p);
        }
        return;
    }

    // ---------------------------------------------------------------------- consumers
    const int t = threadIdx.x;
    float *os = reinterpret_cast<float *>(smem + C::SCR_OFF);  // [CWARPS][G][D]
    float *ms = os + C::CWARPS * G * D, *ls = ms + C::CWARPS * G;
    int *es = reinterpret_cast<int *>(ls + C::CWARPS * G);
    bool ok = true, joined_prefix = false, bad = false;
    long long i = 0;
    for (long long it = it0; it < it1;) {
        const int b = cur.b, g = cur.g, seg_blocks = cur.blocks();
        const SeqPlan sp = cur.s;
        const int m = static_cast<int>(seg_blocks - cur.r < it1 - it ? seg_blocks - cur.r : it1 - it);
        const orthros_bf16 *q = (cur.base ? p.q_new : p.qc_new) + (static_cast<long long>(b) * p.Hq + g * G) * D;
        const float *al = (cur.base ? p.alpha : p.alpha_c) + g * G * D, *be = (cur.base ? p.beta : p.beta_c) + g * G * D;
        typename std::conditional<Q8, WarpQ8<D, NT, Q8 ? CODE : 0>, WarpKeys16<D, NT, false>>::type st;
        if constexpr (Q8) {
            st.load_q(q, al, be, G, p.qscale);
        } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int kt = 0; kt < D / 16; ++kt)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const int row = 8 * nt + (lane >> 2);
                        uint32_t hi = 0, lo = 0;
                        if (row < G)
                            load_q_pair(q + row * D, al + row * D, be + row * D, kt * 16 + 2 * (lane & 3) + 8 * hf,
                                        p.qscale, hi, lo);
                        st.qb[nt][kt][hf] = hi;
                        st.ql[nt][kt][hf] = lo;
                    }
        }
        st.reset();
        for (int x = 0; x < m; ++x, ++i) {
            const int s = static_cast<int>(i % C::STAGES);
            const int r = cur.r + x;
            const bool pre = cur.base && r < sp.npb;
            const int blk = cur.base ? (pre ? sp.pb0 + r : sp.ob0 + r - sp.npb) : r;
            // the block's rows that count: lo .. hi
            const int lo = (cur.base ? (pre ? sp.lo_p : sp.lo) : 0) - blk * C::KB;
            const int hi = (pre ? p.P - 1 : sp.p) - blk * C::KB;
            if (ok && !mbar_wait(&full[s], static_cast<uint32_t>((i / C::STAGES) & 1)))
                ok = false;
            const int r0 = warp * 16;
            if (ok && !sp.full && r0 <= hi && r0 + 15 >= lo) {
                uint8_t *kb = smem + s * 2 * C::KV_BYTES, *vb = kb + C::KV_BYTES;
                int8_t *ke = reinterpret_cast<int8_t *>(smem + C::EXP_OFF + s * 2 * C::KB), *ve = ke + C::KB;
                const bool whole = lo <= r0 && r0 + 15 < (pre ? hi + 1 : hi);  // row p itself is patched in
                if (!whole) {
                    // V rows that do not count become zeros (their weight is zero, but they may hold
                    // anything), and the new row is put where it belongs
                    for (int rr = r0; rr < r0 + 16; ++rr) {
                        const bool fresh = !pre && rr == hi;
                        if (rr >= lo && rr <= hi && !fresh)
                            continue;
                        if constexpr (Q8) {
                            if (!fresh) {
                                if (lane < D / 16)
                                    *reinterpret_cast<uint4 *>(vb + q8_offset<D>(rr, lane)) = make_uint4(0, 0, 0, 0);
                                if (lane == 0)
                                    ve[rr] = -127;
                                continue;
                            }
#pragma unroll
                            for (int kv = 0; kv < 2; ++kv) {
                                // lane l holds values E l .. E l + E - 1
                                constexpr int E = D / 32;
                                const orthros_bf16 *src =
                                    (kv ? p.v_new : p.k_new) + (static_cast<long long>(b) * p.Hkv + g) * D + E * lane;
                                float f[E], amax = 0.f;
#pragma unroll
                                for (int e = 0; e < E; ++e) {
                                    f[e] = __uint_as_float(static_cast<uint32_t>(src[e]) << 16);
                                    if (fabsf(f[e]) < __int_as_float(0x7f800000))
                                        amax = fmaxf(amax, fabsf(f[e]));
                                    else
                                        bad = true;
                                }
#pragma unroll
                                for (int off = 16; off > 0; off >>= 1)
                                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
                                const int ex = q8_exponent<Q8 ? CODE : 0>(amax);
                                const float sd = q8_pow2(-ex);
                                uint32_t w[E / 2];
#pragma unroll
                                for (int e = 0; e < E; e += 2)
                                    w[e / 2] = q8_codes2<Q8 ? CODE : 0>(f[e] * sd, f[e + 1] * sd);
                                uint8_t *to = (kv ? vb : kb) + q8_offset<D>(rr, E * lane / 16) + E * lane % 16;
                                uint8_t *cache = static_cast<uint8_t *>(kv ? p.v_cache : p.k_cache) +
                                                 ((static_cast<long long>(b) * p.L_max + sp.p) * p.Hkv + g) * D + E * lane;
#pragma unroll
                                for (int e = 0; e < E / 2; ++e) {
                                    reinterpret_cast<uint16_t *>(to)[e] = static_cast<uint16_t>(w[e]);
                                    if (!cur.base)
                                        reinterpret_cast<uint16_t *>(cache)[e] = static_cast<uint16_t>(w[e]);
                                }
                                if (lane == 0) {
                                    (kv ? ve : ke)[rr] = static_cast<int8_t>(ex);
                                    if (!cur.base)
                                        (kv ? p.v_exp : p.k_exp)[(static_cast<long long>(b) * p.Hkv + g) * p.L_max +
                                                                 sp.p] = static_cast<int8_t>(ex);
                                }
                            }
                        } else {
                            const int sl = lane / 8, c8 = lane % 8;  // 16-byte chunk of the row
                            if (lane < D / 8) {
                                const long long off = (static_cast<long long>(b) * p.Hkv + g) * D + lane * 8;
                                uint4 kn = make_uint4(0, 0, 0, 0), vn = kn;
                                if (fresh) {
                                    kn = *reinterpret_cast<const uint4 *>(p.k_new + off);
                                    vn = *reinterpret_cast<const uint4 *>(p.v_new + off);
                                    *reinterpret_cast<uint4 *>(kb + sl * C::SLAB + sw128_offset(rr, c8)) = kn;
                                    if (!cur.base) {
                                        const long long row =
                                            ((static_cast<long long>(b) * p.L_max + sp.p) * p.Hkv + g) * D + lane * 8;
                                        *reinterpret_cast<uint4 *>(static_cast<orthros_bf16 *>(p.k_cache) + row) = kn;
                                        *reinterpret_cast<uint4 *>(static_cast<orthros_bf16 *>(p.v_cache) + row) = vn;
                                    }
                                }
                                *reinterpret_cast<uint4 *>(vb + sl * C::SLAB + sw128_offset(rr, c8)) = vn;
                            }
                        }
                    }
                    __syncwarp();
                }
                if constexpr (Q8) {
                    st.step(kb, vb, ke, ve, r0, whole, lo, hi);
                } else {
                    const uint32_t ks = sbase + s * 2 * C::KV_BYTES;
                    int lim[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        lim[nt][0] = lim[nt][1] = hi;
                    st.step(ks, C::SLAB, ks + C::KV_BYTES, C::SLAB, r0, r0, lim, whole, lo);
                }
                if (!whole)
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
                        es[warp * G + row] = st.E;
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
        const long long s0 = it - cur.r, s1 = s0 + seg_blocks;
        const long long c0 = ((s0 + 1) * n - 1) / W, c1 = (s1 * n - 1) / W;  // owners of its first and last block
        const bool joins_prefix = !Q8 && !cur.base && !sp.full;
        const bool alone = c0 == c1 && !joins_prefix;
        const long long slot = 2 * c + (c == c0 ? 1 : 0);  // a segment that began before this CTA: slot 0
        orthros_bf16 *out = (cur.base ? p.o : p.oc) + (static_cast<long long>(b) * p.Hq + g * G) * D;
        for (int e = t; e < G * (D / 4); e += C::CTHREADS) {
            const int row = e / (D / 4), d4 = 4 * (e % (D / 4));
            float M = NEG_INF, L = 0.f;
#pragma unroll
            for (int w = 0; w < C::CWARPS; ++w)
                M = fmaxf(M, ms[w * G + row]);
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < C::CWARPS; ++w) {
                const float mw = ms[w * G + row];
                if (mw == NEG_INF)
                    continue;
                float f = fast_exp2(mw - M);
                L += f * ls[w * G + row];
                if constexpr (Q8)
                    f *= q8_pow2(max(es[w * G + row] - 6, -126));
                const float4 y = *reinterpret_cast<const float4 *>(os + (w * G + row) * D + d4);
                a.x += f * y.x;
                a.y += f * y.y;
                a.z += f * y.z;
                a.w += f * y.w;
            }
            if (alone) {
                const float inv = L > 0.f ? 1.f / L : 0.f;
                *reinterpret_cast<uint2 *>(out + row * D + d4) =
                    make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
            } else {
                *reinterpret_cast<float4 *>(p.part_o + (slot * G + row) * D + d4) = a;
                if (d4 == 0)
                    p.part_ml[slot * G + row] = make_float2(M, L);
            }
        }
        if (sp.full && !cur.base && g == 0 && t == 0)
            record_error(p.dev_err, ORTHROS_DEVERR_CACHE_FULL);
        if (!alone) {
            int *cnt = p.cnt_bh + (static_cast<long long>(b) * p.Hkv + g) * 2 + cur.base;
            __threadfence();
            named_barrier(1, C::CTHREADS);
            if (t == 0)
                s_flag[0] = c0 == c1 || atomicAdd(cnt, 1) == static_cast<int>(c1 - c0);
            named_barrier(1, C::CTHREADS);
            if (s_flag[0]) {
                __threadfence();
                if (t == 0)
                    *cnt = 0;
                if (joins_prefix && !joined_prefix) {
                    asm volatile("griddepcontrol.wait;" ::: "memory");
                    joined_prefix = true;
                }
                // part q: own partials c0 .. c1, then the prefix splits
                const int nown = static_cast<int>(c1 - c0) + 1, nq = nown + (joins_prefix ? p.n_part : 0);
                const long long BH = static_cast<long long>(p.B) * p.Hkv;
                for (int row = warp; row < G; row += C::CWARPS) {
                    auto index = [&](int qi) -> long long {
                        return qi < nown ? (2 * (c0 + qi) + (qi == 0 ? 1 : 0)) * G + row : 0;
                    };
                    auto prefix_index = [&](int qi) -> long long {
                        return (static_cast<long long>(qi - nown) * BH + static_cast<long long>(b) * p.Hkv + g) * G + row;
                    };
                    auto ml_of = [&](int qi) -> float2 {
                        return qi < nown ? __ldcg(p.part_ml + index(qi)) : __ldcg(p.pre_ml + prefix_index(qi));
                    };
                    float M = NEG_INF, L = 0.f;
                    for (int qi = lane; qi < nq; qi += 32)
                        M = fmaxf(M, ml_of(qi).x);
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1)
                        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
                    constexpr int E = D / 32;
                    float a[E];
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        a[e] = 0.f;
                    for (int q0 = 0; q0 < nq; q0 += 32) {
                        float w = 0.f;
                        if (q0 + lane < nq) {
                            const float2 ml = ml_of(q0 + lane);
                            w = ml.x == NEG_INF ? 0.f : fast_exp2(ml.x - M);
                            L += w * ml.y;
                        }
                        const int nn = min(32, nq - q0);
#pragma unroll 8
                        for (int k = 0; k < nn; ++k) {
                            const float wk = __shfl_sync(0xffffffffu, w, k);
                            const int qi = q0 + k;
                            const float *src =
                                (qi < nown ? p.part_o + index(qi) * D : p.pre_o + prefix_index(qi) * D) + lane * E;
                            if constexpr (E == 4) {
                                const float4 y = __ldcg(reinterpret_cast<const float4 *>(src));
                                a[0] = fmaf(wk, y.x, a[0]);
                                a[1] = fmaf(wk, y.y, a[1]);
                                a[2] = fmaf(wk, y.z, a[2]);
                                a[3] = fmaf(wk, y.w, a[3]);
                            } else {
                                const float2 y = __ldcg(reinterpret_cast<const float2 *>(src));
                                a[0] = fmaf(wk, y.x, a[0]);
                                a[1] = fmaf(wk, y.y, a[1]);
                            }
                        }
                    }
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1)
                        L += __shfl_xor_sync(0xffffffffu, L, off);
                    const float inv = L > 0.f ? 1.f / L : 0.f;
#pragma unroll
                    for (int e = 0; e < E; e += 2)
                        *reinterpret_cast<uint32_t *>(out + row * D + lane * E + e) =
                            pack_bf16x2(a[e] * inv, a[e + 1] * inv);
                }
            }
        }
        it += m;
        cur.r += m;
        if (cur.r == seg_blocks && it < it1)
            cur.next_segment(p);
    }
    if constexpr (!Q8) {
        // the step has ended only when the prefix kernel has, whether or not a partial was joined
        if (!joined_prefix)
            asm volatile("griddepcontrol.wait;" ::: "memory");
    }
    if (bad)
        record_error(p.dev_err, ORTHROS_DEVERR_RANGE);
    if (!ok && lane == 0)
        record_error(p.dev_err, ORTHROS_DEVERR_TIMEOUT);

    // ---- the last CTA of the grid advances the lengths (every one has read them by now)
    named_barrier(1, C::CTHREADS);
    if (t == 0) {
        __threadfence();
        s_flag[0] = atomicAdd(p.cnt_all, 1) == static_cast<int>(gridDim.x) - 1;
    }
    named_barrier(1, C::CTHREADS);
    if (s_flag[0]) {
        for (int b = t; b < p.B; b += C::CTHREADS) {
            const int len = __ldcg(p.cache_len + b);
            if (len >= 0 && len < p.L_max)
                p.cache_len[b] = len + 1;
        }
        if (t == 0)
            *p.cnt_all = 0;
    }
}

// ------------------------------------------------------------------ host side

struct ServeLayout {
    int ctas;
    size_t part_ml, cnt, pre_o, pre_ml, total;
};

// the grid: never more CTAs than the longest caches could give blocks
static ServeLayout serve_layout(int B, int P, int L_max, int Hq, int Hkv, int D)
{
    const size_t G = Hq / Hkv, BH = static_cast<size_t>(B) * Hkv;
    const size_t most = 2 * BH * ((static_cast<size_t>(L_max) + 63) / 64 + (static_cast<size_t>(P) + 63) / 64 + 1);
    ServeLayout l;
    l.ctas = static_cast<int>(most < SERVE_CTAS ? most : SERVE_CTAS);
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t slots = 2 * static_cast<size_t>(l.ctas) * G;
    l.part_ml = up(slots * D * sizeof(float));
    l.cnt = l.part_ml + up(slots * sizeof(float2));
    l.pre_o = l.cnt + up((2 * BH + 1) * sizeof(int));
    const size_t pre = P > 0 ? static_cast<size_t>(prefix_attn_parts(B, P, Hq, Hkv)) * BH * G : 0;
    l.pre_ml = l.pre_o + up(pre * D * sizeof(float));
    l.total = l.pre_ml + up(pre * sizeof(float2));
    return l;
}

size_t serve_workspace_bytes(int B, int P, int L_max, int Hq, int Hkv, int D)
{
    return serve_layout(B, P, L_max, Hq, Hkv, D).total;
}

template <int D, int G, int CODE>
static cudaError_t launch_serve_tc(const ServeMaps &maps, const ServeParams &p, int ctas, cudaStream_t stream)
{
    using C = SvCfg<D, G, CODE>;
    auto kern = serve_step_kernel<D, G, CODE>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess)
        return e;
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
    return e == cudaSuccess ? cudaGetLastError() : e;
}

template <int D, int G>
static cudaError_t launch_serve_t(int code, const ServeMaps &maps, const ServeParams &p, int ctas, cudaStream_t stream)
{
    if (code == ORTHROS_KV_E4M3)
        return launch_serve_tc<D, G, ORTHROS_KV_E4M3>(maps, p, ctas, stream);
    if (code == ORTHROS_KV_INT8)
        return launch_serve_tc<D, G, ORTHROS_KV_INT8>(maps, p, ctas, stream);
    return launch_serve_tc<D, G, -1>(maps, p, ctas, stream);
}

cudaError_t launch_serve(int D, int code, const CUtensorMap *m, ServeParams p, void *workspace, cudaStream_t stream)
{
    const ServeLayout l = serve_layout(p.B, p.P, p.L_max, p.Hq, p.Hkv, D);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.part_o = reinterpret_cast<float *>(ws);
    p.part_ml = reinterpret_cast<float2 *>(ws + l.part_ml);
    p.cnt_bh = reinterpret_cast<int *>(ws + l.cnt);
    p.cnt_all = p.cnt_bh + 2 * static_cast<size_t>(p.B) * p.Hkv;
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
        a.qc_bstride = static_cast<long long>(p.Hq) * D;
        a.B = p.B;
        a.T_out = 1;
        a.P = p.P;
        a.Hq = p.Hq;
        a.Hkv = p.Hkv;
        a.qscale = p.qscale;
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

}  // namespace orthros
