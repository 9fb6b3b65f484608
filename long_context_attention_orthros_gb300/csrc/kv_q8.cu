// kv_q8.cu -- prompt rows written into the 8-bit KV cache, and read back as bf16.
//
// A group of d / 8 lanes takes one row of one KV head, eight values a lane: the row's largest
// |x| by shuffles, its exponent, the codes.  A block takes TR rows of one sequence and up to
// HG heads of K or of V, so that the exponents, which lie [head][row], leave as runs of TR
// bytes through shared memory.
#include "kv_q8.cuh"

namespace orthros {

constexpr int KQ_TR = 32;       // rows of a block
constexpr int KQ_HG = 64;       // KV heads of a block
constexpr int KQ_THREADS = 256;

// rows start .. start + rows - 1 of sequence b, or none (with an error bit) if they do not fit
__device__ __forceinline__ int kv_q8_rows(const KvQ8Params &p, int b, int &start, bool report)
{
    start = p.start ? p.start[b] : 0;
    const int rows = p.rows ? p.rows[b] : p.T;
    if (rows < 0 || rows > p.T || start < 0) {
        if (report)
            record_error(p.dev_err, ORTHROS_DEVERR_POSITION);
        return 0;
    }
    if (start > p.L_max - rows) {
        if (report)
            record_error(p.dev_err, ORTHROS_DEVERR_CACHE_FULL);
        return 0;
    }
    return rows;
}

template <int D, int CODE, bool WRITE>
__global__ void __launch_bounds__(KQ_THREADS) kv_q8_kernel(const KvQ8Params p)
{
    constexpr int LANES = D / 8;
    constexpr int GROUPS = KQ_THREADS / LANES;
    __shared__ int8_t exp_s[KQ_HG][KQ_TR];
    const int tiles = (p.T + KQ_TR - 1) / KQ_TR;
    const int b = blockIdx.x / tiles, t0 = (blockIdx.x % tiles) * KQ_TR;
    const int h0 = blockIdx.y * KQ_HG, nh = min(KQ_HG, p.Hkv - h0);
    const bool is_v = blockIdx.z != 0;
    orthros_bf16 *x = is_v ? p.v : p.k;
    uint8_t *c = is_v ? p.v8 : p.k8;
    int8_t *ex = is_v ? p.v_exp : p.k_exp;
    int start;
    const int rows = kv_q8_rows(p, b, start, t0 == 0 && h0 == 0 && threadIdx.x == 0);
    const int nr = min(KQ_TR, rows - t0);
    if (nr <= 0)
        return;
    x += b * p.kv_bstride;
    const long long row0 = static_cast<long long>(b) * p.L_max + start;  // cache row of the sequence's first
    int8_t *ehead = ex + (static_cast<long long>(b) * p.Hkv + h0) * p.L_max + start + t0;
    if constexpr (!WRITE) {
        for (int i = threadIdx.x; i < nh * nr; i += KQ_THREADS)
            exp_s[i / nr][i % nr] = ehead[static_cast<long long>(i / nr) * p.L_max + i % nr];
        __syncthreads();
    }
    const int gid = threadIdx.x / LANES, col = (threadIdx.x % LANES) * 8;
    bool bad = false;
    for (int it0 = 0; it0 < nr * nh; it0 += GROUPS) {
        const int it = it0 + gid;
        const bool on = it < nr * nh;
        const int r = on ? it / nh : 0, h = on ? it % nh : 0;
        orthros_bf16 *px = x + (static_cast<long long>(t0 + r) * p.Hkv + h0 + h) * D + col;
        uint8_t *pc = c + ((row0 + t0 + r) * p.Hkv + h0 + h) * D + col;
        if constexpr (WRITE) {
            const uint4 u = on ? *reinterpret_cast<const uint4 *>(px) : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
            float f[8], amax = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 g = unpack_bf16x2(w[e]);
                f[2 * e] = g.x;
                f[2 * e + 1] = g.y;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float a = fabsf(f[e]);
                if (a < __int_as_float(0x7f800000))
                    amax = fmaxf(amax, a);
                else
                    bad = true;
            }
#pragma unroll
            for (int off = 1; off < LANES; off <<= 1)
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
            const int e = q8_exponent<CODE>(amax);
            const float sd = q8_pow2(-e);
            const uint32_t lo = q8_codes2<CODE>(f[0] * sd, f[1] * sd) | (q8_codes2<CODE>(f[2] * sd, f[3] * sd) << 16);
            const uint32_t hi = q8_codes2<CODE>(f[4] * sd, f[5] * sd) | (q8_codes2<CODE>(f[6] * sd, f[7] * sd) << 16);
            if (on) {
                *reinterpret_cast<uint2 *>(pc) = make_uint2(lo, hi);
                if (col == 0)
                    exp_s[h][r] = static_cast<int8_t>(e);
            }
        } else if (on) {
            const uint2 u = *reinterpret_cast<const uint2 *>(pc);
            const float sd = q8_pow2(exp_s[h][r]);
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t two = (e < 2 ? u.x : u.y) >> (16 * (e & 1));
                o[e] = pack_bf16x2(q8_value<CODE>(two & 0xff) * sd, q8_value<CODE>((two >> 8) & 0xff) * sd);
            }
            *reinterpret_cast<uint4 *>(px) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
    if constexpr (WRITE) {
        if (bad)
            record_error(p.dev_err, ORTHROS_DEVERR_RANGE);
        __syncthreads();
        for (int i = threadIdx.x; i < nh * nr; i += KQ_THREADS)
            ehead[static_cast<long long>(i / nr) * p.L_max + i % nr] = exp_s[i / nr][i % nr];
    }
}

template <int D, int CODE, bool WRITE>
static cudaError_t launch_t(const KvQ8Params &p, cudaStream_t stream)
{
    const long long tiles = (static_cast<long long>(p.T) + KQ_TR - 1) / KQ_TR;
    const dim3 grid(static_cast<unsigned>(tiles * p.B), static_cast<unsigned>((p.Hkv + KQ_HG - 1) / KQ_HG), 2);
    kv_q8_kernel<D, CODE, WRITE><<<grid, KQ_THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

template <bool WRITE>
static cudaError_t launch_any(int D, int code, const KvQ8Params &p, cudaStream_t stream)
{
    if (code == ORTHROS_KV_E4M3)
        return D == 128 ? launch_t<128, ORTHROS_KV_E4M3, WRITE>(p, stream) : launch_t<64, ORTHROS_KV_E4M3, WRITE>(p, stream);
    return D == 128 ? launch_t<128, ORTHROS_KV_INT8, WRITE>(p, stream) : launch_t<64, ORTHROS_KV_INT8, WRITE>(p, stream);
}

cudaError_t launch_kv_quantize(int D, int code, const KvQ8Params &p, cudaStream_t stream)
{
    return launch_any<true>(D, code, p, stream);
}

cudaError_t launch_kv_dequantize(int D, int code, const KvQ8Params &p, cudaStream_t stream)
{
    return launch_any<false>(D, code, p, stream);
}

}  // namespace orthros
