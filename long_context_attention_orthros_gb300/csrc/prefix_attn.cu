// prefix_attn.cu -- attention of every query row of a batch over one shared prompt prefix, computed
// once for all: rows (sequence b, copy i, head of the KV head's group) lie end to end, so each K/V
// byte of the prefix serves the whole batch.  Results are partials (max, sum, unnormalised o) per
// split of the prefix's keys, in the layout the combine kernel and the decode step join with
// the sequences' own rows:  slot (split, b, KV head, copy * G + head).
//
// This kernel serves up to 16 rows a KV head (beyond that its warp MMAs fall behind memory and
// prefix_tc.cu takes over): bound by the prefix's bytes.  4 sequences over 511 + 70 rows (8/2 heads,
// d = 64), this kernel and the step behind it: 9.6 us, two dependent launches' latency.
//
// Grid (split, KV head).  A CTA streams its keys through a TMA ring (64-key blocks, one producer
// warp); four warps run the online softmax of the 16 rows on warp MMAs, each on a quarter of the
// keys, and merge in shared memory.
#include "prefix_rows.cuh"
#include "serve.cuh"
#include "xattn.cuh"

namespace orthros {

template <int D>
struct PaCfg {
    static constexpr int KB = 64;
    static constexpr int SLAB = KB * 128;
    static constexpr int KV_BYTES = KB * D * 2;
    static constexpr int STAGE_BYTES = 2 * KV_BYTES;
    static constexpr int STAGES = 3;
    static constexpr int CWARPS = 4;
    static constexpr int THREADS = (CWARPS + 1) * 32;
    static constexpr int BAR_OFF = STAGES * STAGE_BYTES;
    static constexpr int SMEM = BAR_OFF + 2 * STAGES * 8 + 1024;
    static_assert(STAGES * STAGE_BYTES >= CWARPS * 16 * (D + 2) * 4, "the warps' merge reuses the ring");
};

template <int D, int G>
__global__ void __launch_bounds__(PaCfg<D>::THREADS)
    prefix_attn_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                       const PrefixAttnParams p)
{
    using C = PaCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_s = smem_u32(smem_raw);
    const uint32_t pad = ((raw_s + 1023u) & ~1023u) - raw_s;
    uint8_t *smem = smem_raw + pad;
    const uint32_t sbase = raw_s + pad;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);
    uint64_t *empty = full + C::STAGES;
    const int split = blockIdx.x, g = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ volatile int s_abort;  // a wait has given up: the producer stops
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], C::CWARPS);
        }
        fence_barrier_init();
    }
    // what the kernels before wrote first, then a dependent grid may start beside this one
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (p.clear != nullptr && blockIdx.x + blockIdx.y == 0)
        for (int i = threadIdx.x; i < p.n_clear; i += blockDim.x)
            p.clear[i] = 0;
    __syncthreads();
    const int js = split * p.chunk, je = min(js + p.chunk, p.P);
    const int nblk = je > js ? (je - js + C::KB - 1) / C::KB : 0;

    if (warp == C::CWARPS) {
        if (lane != 0)
            return;
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
        for (int i = 0; i < nblk; ++i) {
            const int s = i % C::STAGES;
            if ((i >= C::STAGES && !mbar_wait(&empty[s], static_cast<uint32_t>(((i / C::STAGES) - 1) & 1))) || s_abort) {
                record_error(p.dev_err, ORTHROS_DEVERR_TIMEOUT);
                drain_in_flight();
                return;
            }
            uint8_t *dst = smem + s * C::STAGE_BYTES;
            mbar_arrive_expect_tx(&full[s], C::STAGE_BYTES);
#pragma unroll
            for (int sl = 0; sl < D / 64; ++sl) {
                tma_load_4d(dst + sl * C::SLAB, &kmap, &full[s], sl * 64, g, js + i * C::KB, 0);
                tma_load_4d(dst + C::KV_BYTES + sl * C::SLAB, &vmap, &full[s], sl * 64, g, js + i * C::KB, 0);
            }
        }
        return;
    }

    const int gr = lane >> 2, qd = (lane & 3) * 2;
    const PrefixRow rows[2] = {prefix_row<G>(p, gr, g, D), prefix_row<G>(p, gr + 8, g, D)};
    WarpRows16<D> st;
#pragma unroll
    for (int kt = 0; kt < D / 16; ++kt)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const PrefixRow &row = rows[r & 1];
            uint32_t hi = 0, lo = 0;
            if (row.q != nullptr)
                load_q_pair(row.q, p.alpha_c + row.head * D, p.beta_c + row.head * D,
                            kt * 16 + qd + ((r & 2) ? 8 : 0), p.qscale, hi, lo);
            st.qa[kt][r] = hi;
            st.ql[kt][r] = lo;
        }
    st.reset();
    bool ok = true;
    for (int i = 0; i < nblk; ++i) {
        const int s = i % C::STAGES;
        if (ok && !mbar_wait(&full[s], static_cast<uint32_t>((i / C::STAGES) & 1)))
            ok = false, s_abort = 1;
        const uint32_t kbase = sbase + s * C::STAGE_BYTES;
        const int j0 = js + i * C::KB + warp * 16;
        if (ok && j0 < je)
            st.step(kbase, C::SLAB, kbase + C::KV_BYTES, C::SLAB, warp * 16, j0, je - 1, je - 1, j0 + 15 < je);
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&empty[s]);
    }
    if (!ok) {
        if (lane == 0)
            record_error(p.dev_err, ORTHROS_DEVERR_TIMEOUT);
        drain_in_flight();
    }
    st.finish_sums();

    // the four warps, scaled to their common max, summed through shared memory
    float *os = reinterpret_cast<float *>(smem);  // [CWARPS][16][D]; the ring is free once all are here
    float *ms = os + C::CWARPS * 16 * D, *ls = ms + C::CWARPS * 16;
    named_barrier(1, C::CWARPS * 32);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int r = warp * 16 + gr + 8 * half;
        if ((lane & 3) == 0) {
            ms[r] = half ? st.mB : st.mA;
            ls[r] = half ? st.lB : st.lA;
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<float2 *>(os + r * D + 8 * i + qd) = make_float2(st.o[i][2 * half], st.o[i][2 * half + 1]);
    }
    named_barrier(1, C::CWARPS * 32);
    const float NEG_INF = -__int_as_float(0x7f800000);
    const long long BHR = static_cast<long long>(p.B) * p.Hkv * p.T_out * G;
    for (int e = threadIdx.x; e < 16 * (D / 4); e += C::CWARPS * 32) {
        const int r = e / (D / 4), d4 = 4 * (e % (D / 4));
        const PrefixRow row = prefix_row<G>(p, r, g, D);
        if (row.slot < 0)
            continue;
        float M = NEG_INF, L = 0.f;
#pragma unroll
        for (int w = 0; w < C::CWARPS; ++w)
            M = fmaxf(M, ms[w * 16 + r]);
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < C::CWARPS; ++w) {
            const int x = w * 16 + r;
            if (ls[x] == 0.f)  // no key
                continue;
            const float f = fast_exp2(ms[x] - M);
            L += f * ls[x];
            const float4 y = *reinterpret_cast<const float4 *>(os + x * D + d4);
            a.x += f * y.x;
            a.y += f * y.y;
            a.z += f * y.z;
            a.w += f * y.w;
        }
        if (row.q == nullptr) {  // a copy without a position takes no key
            M = NEG_INF;
            L = 0.f;
        }
        const long long slot = split * BHR + row.slot;
        *reinterpret_cast<float4 *>(p.part_o + slot * D + d4) = a;
        if (d4 == 0)
            p.part_ml[slot] = make_float2(M, L);
    }
}

// ------------------------------------------------------------------ host side

struct PaPlan {
    int tc;     // 0: warp MMAs; 1: tensor memory, one tile of rows; 2: two tiles
    int tiles, splits, chunk, parts;
};

// warp MMAs: two CTAs on each of 152 SMs in one wave, at least 256 keys a split; tensor memory: one
// CTA an SM, at least 512 keys a split.  Up to 16 rows warp MMAs keep up with memory and start sooner.
// A decode step with them, with tensor memory, us (16 rows a KV head, G = 4): 511 prefix rows of 2 heads,
// d = 64: 9.7, 13.8; of 8 heads, d = 128: 16.1, 20.5; 16384 rows 30.1, 32.2; 131072 rows 97.3, 96.4.
// With 32 rows over 131072 the step took 151 us on warp MMAs, 101 on tensor memory.
static PaPlan pa_plan(long long copies, int P, int Hq, int Hkv)
{
    PaPlan pl;
    const long long R = copies * (Hq / Hkv);
    pl.tc = R <= 16 ? 0 : (R <= 128 ? 1 : 2);
    const int rows = pl.tc ? 128 * pl.tc : 16, ctas = pl.tc ? 152 : 304, keys = pl.tc ? 512 : 256;
    const long long tiles = (R + rows - 1) / rows;
    pl.tiles = static_cast<int>(tiles);
    long long splits = ctas / (tiles * Hkv);
    const long long most = (static_cast<long long>(P) + keys - 1) / keys;
    splits = splits > most ? most : splits;
    splits = splits < 1 ? 1 : splits;
    const int unit = pl.tc ? 128 : 64;
    const long long chunk = ((P + splits - 1) / splits + unit - 1) / unit * unit;
    pl.chunk = static_cast<int>(chunk);
    pl.splits = static_cast<int>((P + chunk - 1) / chunk);
    pl.parts = pl.splits * (pl.tc == 1 ? 2 : 1);
    return pl;
}

int prefix_attn_parts(long long copies, int P, int Hq, int Hkv) { return pa_plan(copies, P, Hq, Hkv).parts; }

template <int D, int G>
static cudaError_t launch_pa(const CUtensorMap &k, const CUtensorMap &v, const PrefixAttnParams &p, const PaPlan &pl,
                             cudaStream_t stream)
{
    auto kern = prefix_attn_kernel<D, G>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, PaCfg<D>::SMEM);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(pl.splits, p.Hkv);
    cfg.blockDim = dim3(PaCfg<D>::THREADS);
    cfg.dynamicSmemBytes = PaCfg<D>::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, k, v, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_prefix_attn(int D, const CUtensorMap &k, const CUtensorMap &v, PrefixAttnParams p,
                               cudaStream_t stream)
{
    const PaPlan pl = pa_plan(static_cast<long long>(p.B) * p.T_out, p.P, p.Hq, p.Hkv);
    if (static_cast<long long>(pl.tiles) * p.Hkv > 65535)
        return cudaErrorInvalidValue;
    p.chunk = pl.chunk;
    if (pl.tc)
        return launch_prefix_tc(D, pl.tc - 1, PrefixMaps{k, v, k, v}, p, pl.splits, pl.tiles, stream);
    const int G = p.Hq / p.Hkv;
#define ORTHROS_PA_CASE(DD, GG) \
    if (D == DD && G == GG)     \
        return launch_pa<DD, GG>(k, v, p, pl, stream);
    ORTHROS_PA_CASE(128, 1)
    ORTHROS_PA_CASE(128, 2)
    ORTHROS_PA_CASE(128, 4)
    ORTHROS_PA_CASE(128, 8)
    ORTHROS_PA_CASE(128, 16)
    ORTHROS_PA_CASE(64, 1)
    ORTHROS_PA_CASE(64, 2)
    ORTHROS_PA_CASE(64, 4)
    ORTHROS_PA_CASE(64, 8)
    ORTHROS_PA_CASE(64, 16)
#undef ORTHROS_PA_CASE
    return cudaErrorInvalidValue;
}

}  // namespace orthros
