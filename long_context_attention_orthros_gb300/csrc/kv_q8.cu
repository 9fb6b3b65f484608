// kv_q8.cu -- prompt rows written into the 8-bit KV cache, and read back as bf16.
//
// Both directions are bound by memory: 3 d + 1 bytes a row (2 d of bf16, d codes, an exponent).  A
// group of d / 8 lanes takes one row of one KV head, eight values (16 bytes of bf16, 8 of codes) a
// lane, two rows in flight a lane (more cost occupancy: 2 rows 303, 4 310, 8 329 us for 2 x 131072
// rows of 8 heads at d = 128).  Writing is close to the limit of the integer pipe, so the largest
// |x| of both rows go around the group in one word of two bf16 (a maximum of bf16 values is one),
// and the exponent is integer arithmetic on the bits.
// A block takes TR rows of one sequence and up to KQ_HG heads of K or of V, so that the exponents,
// which lie [head][row], pass as runs of TR bytes through shared memory.  TR is 32, or 8 where 32
// would leave SMs without a block (the launcher's rule): a few rows are bound by latency.
// Measured (e4m3, 8 heads, d = 128): 2 x 131072 rows written in 262 us (1.61 GB, 6.2 TB/s: 91% of a plain
// copy's rate), 2 x 16384 rows read back in 36 us (83%); 4 x 513 rows of 2 heads in 3.4 us, a launch's time.
#include "kv_q8.cuh"

namespace orthros {

constexpr int KQ_HG = 64;       // KV heads of a block
constexpr int KQ_THREADS = 256;
constexpr int KQ_U = 2;         // items a lane has in flight

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

// largest |x| of each half of eight packed bf16 values (NaN if one is), as bf16 pairs
__device__ __forceinline__ __nv_bfloat162 absmax8(const uint4 &u)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[0]));
#pragma unroll
    for (int e = 1; e < 4; ++e)
        m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[e])));
    return m;
}

// largest finite |x| of eight bf16 values, as bf16 bits
__device__ __noinline__ uint32_t finite_absmax8(uint4 u)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t a = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t x = (w[e / 2] >> (16 * (e & 1))) & 0x7fffu;
        a = x < 0x7f80u && x > a ? x : a;
    }
    return a;
}

template <int D, int CODE, int TR, bool WRITE>
__global__ void __launch_bounds__(KQ_THREADS) kv_q8_kernel(const KvQ8Params p)
{
    constexpr int LANES = D / 8;
    constexpr int GROUPS = KQ_THREADS / LANES;
    __shared__ int8_t exp_s[KQ_HG][TR];
    const int tiles = (p.T + TR - 1) / TR;
    const int b = blockIdx.x / tiles, t0 = (blockIdx.x % tiles) * TR;
    const int h0 = blockIdx.y * KQ_HG, nh = min(KQ_HG, p.Hkv - h0);
    const bool is_v = blockIdx.z != 0;
    int start;
    const int rows = kv_q8_rows(p, b, start, t0 == 0 && h0 == 0 && threadIdx.x == 0);
    const int nr = min(TR, rows - t0);
    if (nr <= 0)
        return;
    const long long row0 = static_cast<long long>(b) * p.L_max + start + t0;  // cache row of the block's first
    orthros_bf16 *x = (is_v ? p.v : p.k) + b * p.kv_bstride + (static_cast<long long>(t0) * p.Hkv + h0) * D;
    uint8_t *c = (is_v ? p.v8 : p.k8) + (row0 * p.Hkv + h0) * D;
    int8_t *ex = (is_v ? p.v_exp : p.k_exp) + (static_cast<long long>(b) * p.Hkv + h0) * p.L_max + start + t0;
    if constexpr (!WRITE) {
        for (int i = threadIdx.x; i < nh * nr; i += KQ_THREADS)
            exp_s[i / nr][i % nr] = ex[static_cast<long long>(i / nr) * p.L_max + i % nr];
        __syncthreads();
    }
    const int gid = threadIdx.x / LANES, col = (threadIdx.x % LANES) * 8;
    const int n = nr * nh;
    bool bad = false;
    // an item is one row of one head, heads first; the lane's next item is GROUPS further
    const int dr = GROUPS / nh, dh = GROUPS % nh;
    int r = gid / nh, h = gid % nh;
    for (int it0 = 0; it0 < n; it0 += GROUPS * KQ_U) {
        int off[KQ_U], ri[KQ_U], hi[KQ_U];  // the same offset in both buffers (rows are Hkv * D apart)
#pragma unroll
        for (int u = 0; u < KQ_U; ++u) {
            ri[u] = r;
            hi[u] = h;
            off[u] = (r * p.Hkv + h) * D + col;
            r += dr;
            h += dh;
            if (h >= nh) {
                h -= nh;
                ++r;
            }
        }
        if constexpr (WRITE) {
            static_assert(KQ_U == 2, "two rows' maxima go around the group in one word");
            uint4 in[KQ_U];
#pragma unroll
            for (int u = 0; u < KQ_U; ++u)
                in[u] = ri[u] < nr ? __ldcs(reinterpret_cast<const uint4 *>(x + off[u])) : make_uint4(0, 0, 0, 0);
            const __nv_bfloat162 m0 = absmax8(in[0]), m1 = absmax8(in[1]);
            __nv_bfloat162 m = __hmax2_nan(__lows2bfloat162(m0, m1), __highs2bfloat162(m0, m1));  // item 0 low, 1 high
            uint32_t mb = *reinterpret_cast<const uint32_t *>(&m);
            const bool odd = ((mb + 0x00800080u) & 0x80008000u) != 0;  // an infinity or a NaN
            if (odd) {
                bad = true;
                mb = finite_absmax8(in[0]) | finite_absmax8(in[1]) << 16;
            }
#pragma unroll
            for (int o = 1; o < LANES; o <<= 1) {
                const uint32_t other = __shfl_xor_sync(0xffffffffu, mb, o);
                m = __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&mb), *reinterpret_cast<const __nv_bfloat162 *>(&other));
                mb = *reinterpret_cast<const uint32_t *>(&m);
            }
            const float2 amax = unpack_bf16x2(mb);
#pragma unroll
            for (int u = 0; u < KQ_U; ++u) {
                const int e = q8_exponent<CODE>(u ? amax.y : amax.x);
                const float sd = q8_pow2(-e);
                const uint32_t w[4] = {in[u].x, in[u].y, in[u].z, in[u].w};
                uint32_t q[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 f = unpack_bf16x2(w[k]);
                    q[k] = q8_codes2_finite<CODE>(f.x * sd, f.y * sd);
                }
                if (odd) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 f = unpack_bf16x2(w[k]);
                        q[k] = q8_codes2<CODE>(f.x * sd, f.y * sd);
                    }
                }
                if (ri[u] < nr) {
                    *reinterpret_cast<uint2 *>(c + off[u]) =
                        make_uint2(__byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410));
                    if (col == 0)
                        exp_s[hi[u]][ri[u]] = static_cast<int8_t>(e);
                }
            }
        } else {
            uint2 in[KQ_U];
#pragma unroll
            for (int u = 0; u < KQ_U; ++u)
                in[u] = ri[u] < nr ? __ldcs(reinterpret_cast<const uint2 *>(c + off[u])) : make_uint2(0, 0);
#pragma unroll
            for (int u = 0; u < KQ_U; ++u) {
                if (ri[u] >= nr)
                    continue;
                const float sd = q8_pow2(exp_s[hi[u]][ri[u]]);
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t hv = q8_half2<CODE>(k < 2 ? in[u].x : in[u].y, k & 1);
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hv));
                    o[k] = pack_bf16x2(f.x * sd, f.y * sd);
                }
                *reinterpret_cast<uint4 *>(x + off[u]) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    }
    if constexpr (WRITE) {
        if (bad)
            record_error(p.dev_err, ORTHROS_DEVERR_RANGE);
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += KQ_THREADS)
            ex[static_cast<long long>(i / nr) * p.L_max + i % nr] = exp_s[i / nr][i % nr];
    }
}

template <int D, int CODE, bool WRITE>
static cudaError_t launch_t(const KvQ8Params &p, cudaStream_t stream)
{
    const unsigned heads = static_cast<unsigned>((p.Hkv + KQ_HG - 1) / KQ_HG);
    const long long tiles = (static_cast<long long>(p.T) + 31) / 32 * p.B;
    if (tiles * heads * 2 >= 304) {
        kv_q8_kernel<D, CODE, 32, WRITE><<<dim3(static_cast<unsigned>(tiles), heads, 2), KQ_THREADS, 0, stream>>>(p);
    } else {
        const unsigned small = static_cast<unsigned>((static_cast<long long>(p.T) + 7) / 8 * p.B);
        kv_q8_kernel<D, CODE, 8, WRITE><<<dim3(small, heads, 2), KQ_THREADS, 0, stream>>>(p);
    }
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
