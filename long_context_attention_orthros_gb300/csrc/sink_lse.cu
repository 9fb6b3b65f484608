// sink_lse.cu -- the log-sum-exp of rows that see at most 64 keys, for orthros_swa_sink_fwd: lse_t = ln sum_j exp(scale
// q_t . k_j), computed to its fp32.
//
// The forward kernels' logits take q as one fp16 (2^-12 off), which the sum over many keys evens out: at 128 keys the
// log-sum-exp is some 1e-5 of itself off, but 1.4e-4 where a row sees one or two (and 1e-4 where one of many has all the
// weight, which is left so).  Here q enters as a bf16 high part plus residual, on warp MMAs: a CTA has 32 tokens of a KV
// head, their keys in shared memory (at most 32 sinks and 64 + 31 window rows), a warp 16 query rows on M at a time and 8
// keys on N, with the head dimension in the order in which it lies in memory (16 bytes a lane).  Rows with few keys are
// all rows, or the first 64 of each sequence, where this is one short launch behind the forward's (4 x 16384 tokens of
// 32/8 heads, d = 128: 10 us).  For all rows of the same at window 33 it takes 410 us: a warp's chain of fragments, which
// the queries' two parts mostly are.
#include "bwd_util.cuh"
#include "kernels.cuh"
#include "xattn.cuh"

namespace orthros {

namespace {

constexpr int SL_TOK = 32, SL_SLOTS = 128;

template <int D>
__global__ void __launch_bounds__(256, 2) sink_lse_kernel(const SinkLseParams p)
{
    constexpr int KK = D / 32, PITCH = D + 32;  // the pitch keeps eight lanes' 16 bytes in banks of their own
    __shared__ __align__(16) uint16_t ks[SL_SLOTS * PITCH];
    asm volatile("griddepcontrol.wait;" ::: "memory");  // for the forward's kernel, which writes lse too
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane & 3, rq = lane >> 2;
    const int G = p.Hq / p.Hkv;
    // ranges begin at multiples of 128, so a row's tile, and its bits, do not depend on them
    const long long per = (p.row_end - p.row_begin + SL_TOK - 1) / SL_TOK, bg = blockIdx.x / per;
    const int g = static_cast<int>(bg % p.Hkv), b = static_cast<int>(bg / p.Hkv);
    const int t0 = p.row_begin + static_cast<int>(blockIdx.x % per) * SL_TOK, t1 = min(t0 + SL_TOK, p.row_end) - 1;
    const int lo0 = max(0, t0 - p.window + 1);    // the first window key of token t0
    const int ns = min(p.sinks, lo0);             // sinks before it
    const int count = ns + t1 - lo0 + 1;          // slots: sinks 0 .. ns - 1, keys lo0 .. t1
    const orthros_bf16 *kb = p.k + b * p.kv_bstride + static_cast<long long>(g) * D;
    for (int x = threadIdx.x; x < count * (D / 8); x += 256) {
        const int slot = x / (D / 8), part = x % (D / 8) * 8, j = slot < ns ? slot : lo0 + slot - ns;
        *reinterpret_cast<uint4 *>(ks + slot * PITCH + part) =
            __ldg(reinterpret_cast<const uint4 *>(kb + static_cast<long long>(j) * p.Hkv * D + part));
    }
    __syncthreads();
    const int rows = (t1 - t0 + 1) * G;
    for (int r0 = 16 * warp; r0 < rows; r0 += 128) {
        uint32_t hi[2 * KK][4], lo[2 * KK][4];  // A fragments of rows r0 + rq and r0 + rq + 8
        int t[2], h[2];
        const orthros_bf16 *x[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const int r = min(r0 + rq + 8 * y, rows - 1);
            t[y] = t0 + r / G;
            h[y] = g * G + r % G;
            x[y] = p.q + b * p.q_bstride + (static_cast<long long>(t[y]) * p.Hq + h[y]) * D + 8 * c;
        }
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            __align__(16) float al[8], be[8];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                if (y == 0 || h[1] != h[0]) {  // eight rows further it is the same head but for G = 16 and the last row
                    const float *a = p.alpha + h[y] * D + 8 * c + 32 * kk, *s = p.beta + h[y] * D + 8 * c + 32 * kk;
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        *reinterpret_cast<float4 *>(al + e) = __ldg(reinterpret_cast<const float4 *>(a + e));
                        *reinterpret_cast<float4 *>(be + e) = __ldg(reinterpret_cast<const float4 *>(s + e));
                    }
                }
                const uint4 u = __ldg(reinterpret_cast<const uint4 *>(x[y] + 32 * kk));
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 v = unpack_bf16x2(w[e]);
                    const int kt = 2 * kk + e / 2, at = y + 2 * (e & 1);
                    split_q_pair(fmaf(v.x, al[2 * e], be[2 * e]), fmaf(v.y, al[2 * e + 1], be[2 * e + 1]), hi[kt][at],
                                 lo[kt][at]);
                }
            }
        }
        // tokens of the tile; window keys that one of them sees
        const int ta = t0 + r0 / G, tb = t0 + min(r0 + 15, rows - 1) / G, first = max(lo0, ta - p.window + 1);
        float m[2] = {-3e38f, -3e38f}, sum[2] = {0.f, 0.f};
        for (int n = 0; n < count; n += 8) {
            const int key = lo0 + n - ns;  // of slot n, behind the sinks' slots
            if (n >= ns && (key > tb || (key + 7 < first && key >= p.sinks)))
                continue;
            float part[4][4] = {};  // four chains of MMAs
            const uint16_t *kr = ks + min(n + rq, count - 1) * PITCH + 8 * c;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                const uint4 u = *reinterpret_cast<const uint4 *>(kr + 32 * kk);
                mma_16816(part[0], hi[2 * kk], u.x, u.y);
                mma_16816(part[1], lo[2 * kk], u.x, u.y);
                mma_16816(part[2], hi[2 * kk + 1], u.z, u.w);
                mma_16816(part[3], lo[2 * kk + 1], u.z, u.w);
            }
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int slot = n + 2 * c + e, j = slot < ns ? slot : lo0 + slot - ns;
                    if (slot < count && j <= t[y] && (j > t[y] - p.window || j < p.sinks)) {
                        const int at = 2 * y + e;
                        const float x = ((part[0][at] + part[2][at]) + (part[1][at] + part[3][at])) * p.qscale;
                        const float big = fmaxf(m[y], x);
                        sum[y] = fmaf(sum[y], fast_exp2(m[y] - big), fast_exp2(x - big));
                        m[y] = big;
                    }
                }
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
#pragma unroll
            for (int off = 1; off <= 2; off <<= 1) {
                const float om = __shfl_xor_sync(0xffffffffu, m[y], off), os = __shfl_xor_sync(0xffffffffu, sum[y], off);
                const float big = fmaxf(m[y], om);
                sum[y] = sum[y] * fast_exp2(m[y] - big) + os * fast_exp2(om - big);
                m[y] = big;
            }
            if (c == 0 && r0 + rq + 8 * y < rows)
                p.lse[(static_cast<long long>(b) * p.T + t[y]) * p.Hq + h[y]] = (m[y] + log2f(sum[y])) * 0.6931471805599453f;
        }
    }
}

template <int D>
cudaError_t launch_t(const SinkLseParams &p, cudaStream_t stream)
{
    const long long per = (p.row_end - p.row_begin + SL_TOK - 1) / SL_TOK;
    return launch_dependent(sink_lse_kernel<D>, dim3(static_cast<unsigned>(per * p.B * p.Hkv)), 256, 0, stream, p);
}

}  // namespace

cudaError_t launch_sink_lse(int D, SinkLseParams p, cudaStream_t stream)
{
    if (p.window > 64 - p.sinks && p.row_end > 64)
        p.row_end = 64;  // only a sequence's first rows see so few keys
    if (p.row_begin >= p.row_end)
        return cudaSuccess;
    return D == 128 ? launch_t<128>(p, stream) : launch_t<64>(p, stream);
}

}  // namespace orthros
