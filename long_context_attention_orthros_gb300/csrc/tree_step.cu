// tree_step.cu -- both streams of a tree of drafted tokens over a KV cache, on warp MMAs: the form for up to 8
// query rows a KV head (a node's single token, a short chain), and the join of partial results.
//
// Bound by the cache's bytes (4 d a row and KV head).  The list of key blocks (tree.cuh) is shared alike by all
// CTAs, two an SM; a CTA's blocks arrive by TMA through a ring that runs on across segment borders (one
// producer warp); four warps take 32 keys of every other block each, the rows on the MMA's N side, and their
// results meet in shared memory.  A segment that one CTA holds whole is
// written at once, the others as one partial (max, sum, o) a CTA, which tree_join_kernel joins.
//
// The block that holds the last cached row is patched in shared memory: V rows that no query of the segment
// sees (behind the last row, before the window, behind the sinks, behind the last node) become zeros, as they
// may hold anything and have a weight of zero.
#include "tree_rows.cuh"
#include "warp_b16.cuh"

namespace orthros {

constexpr int TREE_CTAS = 304;  // two on each of 152 SMs
constexpr int TREE_COST = 4;

template <int D>
struct TsCfg {
    static constexpr int TR = 8;
    static constexpr int KB = TREE_KB;
    static constexpr int SLAB = KB * 128;
    static constexpr int KV_BYTES = KB * D * 2;
    static constexpr int KT = 2;  // a warp's step: two chunks of 16 keys
    static constexpr int CWARPS = 4;
    static constexpr int GROUP = 4 / KT;  // warps that share a block
    static constexpr int STAGES = D == 128 ? 2 : 4;  // a slot belongs to one group of warps: a multiple of KT
    static constexpr int SCR_OFF = STAGES * 2 * KV_BYTES;
    static constexpr int SCR_BYTES = CWARPS * TR * (D + 2) * 4;
    static constexpr int BAR_OFF = SCR_OFF + SCR_BYTES;
    static constexpr int SMEM = BAR_OFF + 2 * STAGES * 8 + 16 + 1024;
    static constexpr int CTHREADS = CWARPS * 32;
    static constexpr int THREADS = CTHREADS + 32;
    static_assert(STAGES % KT == 0, "a slot belongs to one group of warps");
    static_assert(2 * (SMEM + 1024) <= 233472, "two CTAs an SM");
};

template <int D>
__global__ void __launch_bounds__(TsCfg<D>::THREADS, 2)
    tree_step_kernel(const __grid_constant__ TreeMaps maps, const TreeParams p)
{
    using C = TsCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_s = smem_u32(smem_raw);
    const uint32_t pad = ((raw_s + 1023u) & ~1023u) - raw_s;
    uint8_t *smem = smem_raw + pad;
    const uint32_t sbase = raw_s + pad;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);
    uint64_t *empty = full + C::STAGES;
    __shared__ volatile int s_abort;  // a wait has given up: the producer stops
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float NEG_INF = -__int_as_float(0x7f800000);
    const int G = p.Hq / p.Hkv;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], C::GROUP);
        }
        s_abort = 0;
        fence_barrier_init();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long c = blockIdx.x;
    const TreeShare<C::TR, TREE_COST> sh = tree_share<C::TR, TREE_COST>(p, c, gridDim.x);
    const long long W = sh.W, n = sh.n, it0 = sh.it0, it1 = sh.it1;
    auto cur = sh.cur;
    __syncthreads();  // barriers are set up

    if (warp == C::CWARPS) {
        // ------------------------------------------------------------------ producer
        if (lane != 0)
            return;
        long long i = 0;
        for (long long it = it0; it < it1; ++it) {
            if (cur.r >= TREE_COST) {
                const int s = static_cast<int>(i % C::STAGES);
                if ((i >= C::STAGES && !mbar_wait(&empty[s], static_cast<uint32_t>(((i / C::STAGES) - 1) & 1))) ||
                    s_abort) {
                    record_error(p.dev_err, ORTHROS_DEVERR_TIMEOUT);
                    drain_in_flight();
                    return;
                }
                const int j0 = cur.first_row(cur.r - TREE_COST);
                uint8_t *dst = smem + s * 2 * C::KV_BYTES;
                mbar_arrive_expect_tx(&full[s], 2 * C::KV_BYTES);
                const CUtensorMap *mk = j0 < 0 ? &maps.kt : &maps.k, *mv = j0 < 0 ? &maps.vt : &maps.v;
#pragma unroll
                for (int sl = 0; sl < D / 64; ++sl) {
                    tma_load_4d(dst + sl * C::SLAB, mk, &full[s], sl * 64, cur.g, max(j0, 0), cur.b);
                    tma_load_4d(dst + C::KV_BYTES + sl * C::SLAB, mv, &full[s], sl * 64, cur.g, max(j0, 0), cur.b);
                }
                ++i;
            }
            if (++cur.r == cur.places() && it + 1 < it1)
                cur.next_segment(p);
        }
        return;
    }

    // ---------------------------------------------------------------------- consumers
    const int t = threadIdx.x;
    float *os = reinterpret_cast<float *>(smem + C::SCR_OFF);  // [CWARPS][TR][D]
    float *ms = os + C::CWARPS * C::TR * D, *ls = ms + C::CWARPS * C::TR;
    bool ok = true;
    long long i = 0;
    int paths_b = -1;
    TreePaths paths = {};
    for (long long it = it0; it < it1;) {
        const int b = cur.b, g = cur.g, base = cur.base, seg_places = cur.places();
        const TreeSeq s = cur.s;
        const int places = static_cast<int>(seg_places - cur.r < it1 - it ? seg_places - cur.r : it1 - it);
        const int first = max(cur.r - TREE_COST, 0), m = cur.r + places - TREE_COST - first;
        if (m <= 0) {  // the CTA's last places are a segment's empty ones
            it += places;
            continue;
        }
        if (b != paths_b) {
            paths = tree_paths(p.parent + static_cast<long long>(b) * p.N, s.n);
            paths_b = b;
        }
        // the lane's two rows: what they see
        TreeRow rows[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
            rows[e] = tree_row(p, s, paths, base, (cur.tile * C::TR + 2 * (lane & 3) + e) / G);
        WarpB16<D, 1> st;
        {
            const orthros_bf16 *q = base ? p.q_new : p.qc_new;
            const float *al = base ? p.alpha : p.alpha_c, *be = base ? p.beta : p.beta_c;
            const int row = cur.tile * C::TR + (lane >> 2), node = row / G, h = g * G + row % G;
            const bool live = node < s.n;
            const orthros_bf16 *x = q + ((static_cast<long long>(b) * p.N + (live ? node : 0)) * p.Hq + h) * D;
#pragma unroll
            for (int kt = 0; kt < D / 16; ++kt)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int d = kt * 16 + 2 * (lane & 3) + 8 * hf;
                    uint32_t hi = 0, lo = 0;
                    if (live) {
                        const float2 v = unpack_bf16x2(__ldg(reinterpret_cast<const uint32_t *>(x + d)));
                        const float2 a = __ldg(reinterpret_cast<const float2 *>(al + h * D + d));
                        const float2 z = __ldg(reinterpret_cast<const float2 *>(be + h * D + d));
                        split_q_pair(fmaf(v.x, a.x, z.x) * p.qscale, fmaf(v.y, a.y, z.y) * p.qscale, hi, lo);
                    }
                    st.qb[0][kt][hf] = hi;
                    st.ql[0][kt][hf] = lo;
                }
        }
        st.reset();
        int span_lo, span_first;
        tree_span(p, s, base, span_lo, span_first);
        for (int x = 0; x < m; ++x, ++i) {
            if (C::KT == 2 && (i & 1) != (warp >> 1))
                continue;  // the other pair's block
            const int slot = static_cast<int>(i % C::STAGES);
            const int j0 = cur.first_row(first + x);
            if (ok && !mbar_wait(&full[slot], static_cast<uint32_t>((i / C::STAGES) & 1)))
                ok = false, s_abort = 1;
            constexpr int WK = 16 * C::KT;  // this warp's keys: rows r0 .. r0 + WK - 1 of the block
            const int r0 = (warp % C::GROUP) * WK;
            const int end = j0 < 0 ? s.n : s.len - j0;  // rows of the block that exist
            if (ok && !s.full && r0 < end) {
                uint8_t *vb = smem + slot * 2 * C::KV_BYTES + C::KV_BYTES;
                auto counts = [&](int r) {
                    return r < end && (j0 < 0 || j0 + r >= span_lo || j0 + r < span_first);
                };
                const bool patch = r0 + WK > end || (j0 >= 0 && j0 + r0 < span_lo);
                if (patch) {
                    constexpr int CH = D / 8;  // 16-byte chunks of a row
#pragma unroll 1
                    for (int e = lane; e < WK * CH; e += 32) {
                        const int r = r0 + e / CH, c16 = e % CH;
                        if (!counts(r))
                            *reinterpret_cast<uint4 *>(vb + (c16 / 8) * C::SLAB + sw128_offset(r, c16 % 8)) =
                                make_uint4(0, 0, 0, 0);
                    }
                    __syncwarp();
                }
                const uint32_t ks = sbase + slot * 2 * C::KV_BYTES;
                if (j0 < 0) {
                    st.template step_where<C::KT>(ks, ks + C::KV_BYTES, C::SLAB, r0, false, [&](int y, int, int e) {
                        return ((rows[e].mask >> y) & 1) != 0;
                    });
                } else {
                    st.template step_where<C::KT>(ks, ks + C::KV_BYTES, C::SLAB, r0, !base && r0 + WK <= end,
                                                  [&](int y, int, int e) {
                        const int j = j0 + y;
                        return y < end && (j >= rows[e].lo || j < rows[e].first);
                    });
                }
                if (patch)
                    fence_proxy_async_smem();  // before TMA writes over what was patched
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&empty[slot]);
        }
        st.finish_sums();

        // ---- the four warps' results meet in shared memory
        named_barrier(1, C::CTHREADS);  // the segment before has been read
#pragma unroll
        for (int r2 = 0; r2 < 2; ++r2) {
            const int row = 2 * (lane & 3) + r2, gq = lane >> 2;
            if (gq == 0) {
                ms[warp * C::TR + row] = st.m[0][r2];
                ls[warp * C::TR + row] = st.l[0][r2];
            }
            float *po = os + (warp * C::TR + row) * D;
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
                po[16 * mt + gq] = st.o[0][mt][r2];
                po[16 * mt + gq + 8] = st.o[0][mt][2 + r2];
            }
        }
        named_barrier(1, C::CTHREADS);
        // segment bounds in the list, and who else has a share
        const long long s0 = it - cur.r + TREE_COST, s1 = it - cur.r + seg_places;
        const long long c0 = ((s0 + 1) * n - 1) / W, c1 = (s1 * n - 1) / W;  // owners of its first and last block
        const bool alone = c0 == c1;
        // one slot for a segment that began before this CTA, one for one that runs out of it
        const long long slot = 2 * c + (c == c0 ? 1 : 0);
        for (int e = t; e < C::TR * (D / 4); e += C::CTHREADS) {
            const int row = e / (D / 4), d4 = 4 * (e % (D / 4));
            const int node = (cur.tile * C::TR + row) / G;
            if (node >= s.n)
                continue;
            const bool none = s.full || ((paths.bad >> node) & 1);  // zeros
            float M = NEG_INF, L = 0.f;
#pragma unroll
            for (int w = 0; w < C::CWARPS; ++w)
                M = fmaxf(M, ms[w * C::TR + row]);
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < C::CWARPS; ++w) {
                const float lw = ls[w * C::TR + row];
                if (lw == 0.f || none)  // no key (a NaN has a sum of NaN, and goes on)
                    continue;
                const float f = fast_exp2(ms[w * C::TR + row] - M);
                L += f * lw;
                const float4 y = *reinterpret_cast<const float4 *>(os + (w * C::TR + row) * D + d4);
                a.x += f * y.x;
                a.y += f * y.y;
                a.z += f * y.z;
                a.w += f * y.w;
            }
            if (alone) {
                const float inv = L > 0.f ? 1.f / L : L;  // a NaN stays one
                const int h = g * G + (cur.tile * C::TR + row) % G;
                orthros_bf16 *out = (base ? p.o : p.oc) + ((static_cast<long long>(b) * p.N + node) * p.Hq + h) * D + d4;
                *reinterpret_cast<uint2 *>(out) =
                    make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
            } else {
                *reinterpret_cast<float4 *>(p.part_o + (slot * C::TR + row) * D + d4) = a;
                if (d4 == 0)
                    p.part_ml[slot * C::TR + row] = none ? make_float2(NEG_INF, 0.f) : make_float2(M, L);
            }
        }
        if (!base && g == 0 && cur.tile == 0 && t == 0) {
            const int len = __ldcg(p.cache_len + b);
            if (len < 0 || len > p.L_max)
                record_error(p.dev_err, ORTHROS_DEVERR_CACHE_FULL);
            else if (s.full || paths.bad != 0)
                record_error(p.dev_err, ORTHROS_DEVERR_POSITION);
        }
        it += places;
        cur.r += places;
        if (cur.r == seg_places && it < it1)
            cur.next_segment(p);
    }
    if (!ok) {
        if (lane == 0)
            record_error(p.dev_err, ORTHROS_DEVERR_TIMEOUT);
        drain_in_flight();
    }
}

// ------------------------------------------------------------------ the join

// One half-warp a query row: the partials of the CTAs that held a share of its segment, found by the same
// arithmetic as in the step; rows that one CTA held whole are written already.  Eight parts' loads in flight.
template <int D, int TR, int COST>
__global__ void __launch_bounds__(128) tree_join_kernel(const TreeParams p, int ctas)
{
    constexpr int E = D / 16;
    const int t = threadIdx.x, lane = t & 31, hl = t & 15;
    const int G = p.Hq / p.Hkv, most = (p.N * G + TR - 1) / TR;  // tiles of a full tree
    int x = blockIdx.x;
    const int piece = x % (TR / 8);
    x /= TR / 8;
    const int tile = x % most;
    x /= most;
    const int base = x % 2;
    x /= 2;
    const int g = x % p.Hkv, b = x / p.Hkv;
    const float NEG_INF = -__int_as_float(0x7f800000);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    long long W = 0, before = 0;  // places of the list, and those before sequence b
    TreeCursor<TR, COST> cur{};
    for (int i = lane; i < p.B; i += 32) {
        cur.s = tree_seq<TR>(p, i);
        const long long w = cur.seq_places(p.Hkv);
        W += w;
        before += i < b ? w : 0;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        W += __shfl_xor_sync(0xffffffffu, W, off);
        before += __shfl_xor_sync(0xffffffffu, before, off);
    }
    const TreeSeq s = tree_seq<TR>(p, b);
    if (tile >= s.tiles)
        return;
    const long long n = ctas < W ? ctas : W;
    const int pc = s.nc + COST, pb = s.nb + COST;
    const long long s0 = before + static_cast<long long>(pc + pb) * s.tiles * g +
                         (base ? static_cast<long long>(pc) * s.tiles + static_cast<long long>(pb) * tile
                               : static_cast<long long>(pc) * tile) + COST;
    const long long s1 = s0 + (base ? s.nb : s.nc);
    const long long c0 = ((s0 + 1) * n - 1) / W, c1 = (s1 * n - 1) / W;
    const int row = piece * 8 + (t >> 4), node = (tile * TR + row) / G;
    if (c0 == c1)
        return;
    const int nq = node < s.n ? static_cast<int>(c1 - c0) + 1 : 0;  // the whole warp stays for the shuffles
    auto slot_of = [&](int q) { return (2 * (c0 + q) + (q == 0 ? 1 : 0)) * TR + row; };
    float M = NEG_INF;
    for (int q = hl; q < nq; q += 16)
        M = fmaxf(M, __ldcg(p.part_ml + slot_of(q)).x);
#pragma unroll
    for (int off = 8; off > 0; off >>= 1)
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float L = 0.f, a[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        a[e] = 0.f;
    for (int q0 = 0; q0 < nq; q0 += 8) {
        float2 ml[8];
        float4 y[8][E / 4];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            ml[k] = make_float2(NEG_INF, 0.f);
            if (q0 + k < nq) {
                const long long sl = slot_of(q0 + k);
                ml[k] = __ldcg(p.part_ml + sl);
#pragma unroll
                for (int e = 0; e < E / 4; ++e)
                    y[k][e] = __ldcg(reinterpret_cast<const float4 *>(p.part_o + sl * D + hl * E) + e);
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (ml[k].y == 0.f)  // no key there; a NaN reaches the output
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
    if (nq > 0) {
        const float inv = L > 0.f ? 1.f / L : L;
        const int h = g * G + (tile * TR + row) % G;
        orthros_bf16 *out = (base ? p.o : p.oc) + ((static_cast<long long>(b) * p.N + node) * p.Hq + h) * D + hl * E;
#pragma unroll
        for (int e = 0; e < E; e += 4)
            *reinterpret_cast<uint2 *>(out + e) = make_uint2(pack_bf16x2(a[e] * inv, a[e + 1] * inv),
                                                             pack_bf16x2(a[e + 2] * inv, a[e + 3] * inv));
    }
}

// ------------------------------------------------------------------ host side

struct TreePlan {
    int tr, ctas;
    size_t part_ml, total;
};

// Warp MMAs keep up with memory for up to 8 query rows a KV head (2 x 131072 rows of 32/8 heads, d = 128: 167 us; two
// tiles of 8 would be 16 rows, which took 233 with a step of 16 keys, and 185 on tensor memory); more go to tensor
// memory, in tiles of 128 rows (64 rows a KV head over 2 x 131072: 183 us, in the form for 256 rows 263) or, where
// one does not hold them, two at a time.
static TreePlan tree_plan(int B, int N, int L_max, int Hq, int Hkv, int D)
{
    TreePlan pl;
    const long long R = static_cast<long long>(N) * (Hq / Hkv);
    pl.tr = R <= 8 ? 8 : (R <= 128 ? 128 : 256);
    // never more CTAs than the longest caches could give places
    const long long tiles = (R + pl.tr - 1) / pl.tr;
    const long long most = 2 * tiles * B * Hkv * (TREE_COST + 2 + (L_max + 63LL) / 64), ctas = pl.tr == 8 ? TREE_CTAS : TREE_TC_CTAS;
    pl.ctas = static_cast<int>(most < ctas ? most : ctas);
    const size_t slots = 2 * static_cast<size_t>(pl.ctas) * pl.tr;
    pl.part_ml = (slots * D * sizeof(float) + 255) / 256 * 256;
    pl.total = pl.part_ml + (slots * sizeof(float2) + 255) / 256 * 256;
    return pl;
}

size_t tree_workspace_bytes(int B, int N, int L_max, int Hq, int Hkv, int D)
{
    return tree_plan(B, N, L_max, Hq, Hkv, D).total;
}

template <int D>
static cudaError_t launch_tree_step(const TreeMaps &maps, const TreeParams &p, int ctas, cudaStream_t stream)
{
    using C = TsCfg<D>;
    auto kern = tree_step_kernel<D>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
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
    return cudaLaunchKernelEx(&cfg, kern, maps, p);
}

template <int D, int TR>
static cudaError_t launch_tree_t(const TreeMaps &maps, const TreeParams &p, int ctas, cudaStream_t stream)
{
    constexpr int COST = TR == 8 ? TREE_COST : TREE_TC_COST;
    cudaError_t e;
    if constexpr (TR == 8)
        e = launch_tree_step<D>(maps, p, ctas, stream);
    else
        e = launch_tree_tc(D, TR, maps, p, ctas, stream);
    if (e != cudaSuccess)
        return e;
    const int tiles = (p.N * (p.Hq / p.Hkv) + TR - 1) / TR;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.B) * p.Hkv * 2 * tiles * (TR / 8));
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, tree_join_kernel<D, TR, COST>, p, ctas);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_tree(int D, const TreeMaps &maps, TreeParams p, void *workspace, cudaStream_t stream)
{
    const TreePlan pl = tree_plan(p.B, p.N, p.L_max, p.Hq, p.Hkv, D);
    p.part_o = static_cast<float *>(workspace);
    p.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(workspace) + pl.part_ml);
#define ORTHROS_TREE_CASE(DD, RR) \
    if (D == DD && pl.tr == RR)   \
        return launch_tree_t<DD, RR>(maps, p, pl.ctas, stream);
    ORTHROS_TREE_CASE(128, 8)
    ORTHROS_TREE_CASE(128, 128)
    ORTHROS_TREE_CASE(128, 256)
    ORTHROS_TREE_CASE(64, 8)
    ORTHROS_TREE_CASE(64, 128)
    ORTHROS_TREE_CASE(64, 256)
#undef ORTHROS_TREE_CASE
    return cudaErrorInvalidValue;
}

// ------------------------------------------------------------------ what was accepted

// A cluster of eight CTAs a sequence: each finds the path (log2 N rounds of path doubling in one warp), copies
// every eighth row of it, and the first writes the new length when all have read the old one.  Bound by its
// latency: the length, the paths and one round of copies.
constexpr int ACCEPT_CTAS = 8;

__global__ void __cluster_dims__(ACCEPT_CTAS, 1, 1) __launch_bounds__(256) tree_accept_kernel(const TreeAcceptParams p)
{
    const int b = blockIdx.y, rank = blockIdx.x;
    const int node = __ldg(p.node + b), len = __ldcg(p.cache_len + b);
    const int n = p.nodes != nullptr ? __ldg(p.nodes + b) : p.N;
    const bool sized = n >= 0 && n <= p.N, inside = sized && node >= 0 && node < n;
    // every warp finds the path by itself
    const TreePaths t = tree_paths(p.parent + static_cast<long long>(b) * p.N, inside ? node + 1 : 0);
    unsigned long long path = inside ? t.of(node) : 0;
    int err = !sized || node < -1 || node >= n || (inside && ((t.bad >> node) & 1)) ? ORTHROS_DEVERR_POSITION : 0;
    if (err == 0 && (len < 0 || len > p.L_max || __popcll(path) > p.L_max - len))
        err = ORTHROS_DEVERR_CACHE_FULL;
    if (err != 0)
        path = 0;
    const int count = __popcll(path);
    // position k of the path is its k-th lowest bit
    auto at = [&](int k) {
        unsigned long long m = path;
        for (int i = 0; i < k; ++i)
            m &= m - 1;
        return __ffsll(static_cast<long long>(m)) - 1;
    };
    if (rank == 0) {
        for (int k = threadIdx.x; k < p.N; k += blockDim.x)
            p.path[static_cast<long long>(b) * p.N + k] = k < count ? at(k) : -1;
        if (threadIdx.x == 0 && err != 0)
            record_error(p.dev_err, err);
    }
    const int chunks = p.row / 8;  // 16 bytes each
    for (int k = rank; k < count; k += ACCEPT_CTAS) {
        const long long from = (static_cast<long long>(b) * p.N + at(k)) * p.row;
        const long long to = (static_cast<long long>(b) * p.L_max + len + k) * p.row;
        for (int x = threadIdx.x; x < 2 * chunks; x += blockDim.x) {
            const bool v = x >= chunks;
            const int e = 8 * (v ? x - chunks : x);
            const uint4 y = __ldg(reinterpret_cast<const uint4 *>((v ? p.v_new : p.k_new) + from + e));
            *reinterpret_cast<uint4 *>((v ? p.v_cache : p.k_cache) + to + e) = y;
        }
    }
    asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
    if (rank == 0 && threadIdx.x == 0 && count > 0)
        p.cache_len[b] = len + count;
}

cudaError_t launch_tree_accept(const TreeAcceptParams &p, cudaStream_t stream)
{
    tree_accept_kernel<<<dim3(ACCEPT_CTAS, p.B), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace orthros
