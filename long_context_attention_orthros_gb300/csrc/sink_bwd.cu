// sink_bwd.cu -- gradient of the base stream with attention sinks (row t sees keys j <= t with j > t - window or
// j < sinks), given the forward's log-sum-exp and output.  With x = Q_raw, q = x alpha + beta,
//   p_tj = exp(scale q_t . k_j - lse_t),  D_t = dO_t . o_t,  dS_tj = p_tj (dO_t . v_j - D_t)
//   dq_t = scale sum_j dS_tj k_j,  dq_raw = dq alpha,  dalpha = sum_t x_t dq_t,  dbeta = sum_t dq_t
//   dk_j = scale sum_t dS_tj q_t,  dv_j = sum_t p_tj dO_t
// Everything leaves in fp32 and is computed to match: k, v, x and dO are bf16 and enter the products as they are;
// q, dS and P enter as a bf16 high part plus residual (their product's relative error some 2^-17, where one
// bf16 would give 2^-9); sums, exponents and D are fp32.  Launches:
//   sink_keys_kernel    q's two parts, D and the log-sum-exp in log2 units, one pass over x, o, dO; in the same pass
//                       the sinks' share of dk, dv from the rows behind their window: every row adds to the same few
//                       keys, so the tokens are split over CTAs, which leave partial sums
//   sink_rows_kernel    the pass alone, where no row has a sink behind its window
//   sink_dq_tc_kernel   dq over a row's window and the sinks; dalpha, dbeta by atomics (sink_dq.cu)
//   sink_dkv_tc_kernel  dk, dv of the window's part (sink_dkv.cu)
//   sink_join_kernel    adds the partial sums to dk, dv in order
#include "bwd_util.cuh"
#include "kernels.cuh"
#include "xattn.cuh"

namespace orthros {

namespace {

// ------------------------------------------------------------------ prepared rows

// D / 8 lanes a row, 16 bytes of each of x, o and dO a lane.  The first CTAs also zero dalpha and dbeta.
template <int D>
__global__ void __launch_bounds__(256) sink_rows_kernel(const SinkBwdParams p)
{
    constexpr int LPR = D / 8;
    const long long rows = static_cast<long long>(p.B) * p.T * p.Hq;
    const long long id = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x, row = id / LPR;
    const int sub = static_cast<int>(id % LPR);
    for (long long i = id; i < p.Hq * D; i += static_cast<long long>(gridDim.x) * blockDim.x)
        p.dalpha[i] = p.dbeta[i] = 0.f;
    float acc = 0.f;
    if (row < rows) {
        const long long off = row * D + sub * 8;
        const uint4 xa = __ldg(reinterpret_cast<const uint4 *>(p.q + off));
        const uint4 oa = __ldg(reinterpret_cast<const uint4 *>(p.o + off));
        const uint4 ga = __ldg(reinterpret_cast<const uint4 *>(p.dO + off));
        const int col = static_cast<int>(row % p.Hq) * D + sub * 8;
        const uint32_t xw[4] = {xa.x, xa.y, xa.z, xa.w}, ow[4] = {oa.x, oa.y, oa.z, oa.w}, gw[4] = {ga.x, ga.y, ga.z, ga.w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 a = __ldg(reinterpret_cast<const float2 *>(p.alpha + col) + e);
            const float2 b = __ldg(reinterpret_cast<const float2 *>(p.beta + col) + e);
            const float2 x = unpack_bf16x2(xw[e]), u = unpack_bf16x2(ow[e]), v = unpack_bf16x2(gw[e]);
            split_q_pair(fmaf(x.x, a.x, b.x), fmaf(x.y, a.y, b.y), hi[e], lo[e]);
            acc = fmaf(u.x, v.x, fmaf(u.y, v.y, acc));
        }
        *reinterpret_cast<uint4 *>(p.q_hi + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(p.q_lo + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1)
        acc += __shfl_xor_sync(0xffffffffu, acc, off);
    if (row < rows && sub == 0) {
        p.Drow[row] = acc;
        p.lse[row] = p.lse_in[row] * kLog2eF;
    }
}

// ------------------------------------------------------------------ the sinks' dk, dv

// The prepared rows, and rows t against sinks j <= t - window.  A CTA has one (sequence, query head) and a run of
// tokens, a warp 16 tokens at a time: the (up to 16) sinks on M and the tokens on N for S^T = K q^T and dP^T = V dO^T,
// whose fragments are then the operands of Y = dS^T q and dV = P^T dO (tokens on K).  Operands are taken 16 bytes a
// lane, with the head dimension in the order in which it lies in memory; a lane copies what it will itself use into
// its places of a ring while the 16 tokens before are worked on (two CTAs an SM hold some 100 KB on their way).  A
// token's heads lie together in memory, so their CTAs follow one another.  More than 16 sinks: blockIdx.y (the first
// 16 write the prepared rows).
// It moves 670 MB for 1 x 16384 tokens of 32/8 heads, d = 128, in 172 us (3.9 TB/s; 220 with loads where they are used
// and the warps' sums one after the other).  What it waits for is the chain of a warp's 16 tokens, two warps a
// scheduler.
constexpr int SK_M = 16;

template <int D>
constexpr int sk_ring = 2 * 4 * (3 * 2 * D / 32) * 32 * 16;  // stages, warps, pieces of x, o and dO, lanes, bytes

template <int D>
__global__ void __launch_bounds__(128, 2) sink_keys_kernel(const SinkBwdParams p, int chunks, int count)
{
    constexpr int KK = D / 32;  // runs of 32 values: a lane has 8 of each row
    __shared__ __align__(16) uint4 ka_s[D / 16][32], va_s[D / 16][32];  // K, V as A fragments
    __shared__ __align__(16) float ab[2 * D];
    extern __shared__ __align__(16) uint8_t ring[];  // sk_ring<D> bytes, at the end the warps' sums
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane & 3, rq = lane >> 2;
    const int h = blockIdx.x % p.Hq, chunk = blockIdx.x / p.Hq % chunks, b = blockIdx.x / p.Hq / chunks;
    const int bh = b * p.Hq + h, g = h / (p.Hq / p.Hkv);
    const int s0 = SK_M * blockIdx.y, ns = min(SK_M, count - s0);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int T = p.T;

    auto pair = [&](const orthros_bf16 *src, int j, int d) -> uint32_t {  // two values of a sink (zero behind the last)
        return j < ns ? *reinterpret_cast<const uint32_t *>(src + ((static_cast<long long>(b) * T + s0 + j) * p.Hkv + g) * D + d)
                      : 0u;
    };
    for (int x = threadIdx.x; x < D / 16 * 32; x += 128) {
        const int kt = x / 32, l = x % 32, d = 32 * (kt / 2) + 8 * (l & 3) + 4 * (kt & 1), j = l >> 2;
        ka_s[kt][l] = make_uint4(pair(p.k, j, d), pair(p.k, j + 8, d), pair(p.k, j, d + 2), pair(p.k, j + 8, d + 2));
        va_s[kt][l] = make_uint4(pair(p.v, j, d), pair(p.v, j + 8, d), pair(p.v, j, d + 2), pair(p.v, j + 8, d + 2));
    }
    for (int x = threadIdx.x; x < D; x += 128) {
        ab[x] = p.alpha[h * D + x];
        ab[D + x] = p.beta[h * D + x];
        if (chunk == 0 && b == 0 && blockIdx.y == 0)
            p.dalpha[h * D + x] = p.dbeta[h * D + x] = 0.f;
    }
    __syncthreads();

    const int per = ((T + chunks - 1) / chunks + 63) / 64 * 64;
    const int t_begin = chunk * per, t_end = min(T, t_begin + per);
    const float c2 = p.scale * kLog2eF;
    float y[D / 8][4], dv[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            y[i][e] = dv[i][e] = 0.f;
    const long long stride = static_cast<long long>(p.Hq) * D;  // between tokens
    const long long row0 = static_cast<long long>(b) * T * p.Hq + h;
    const uint4 *mine = reinterpret_cast<const uint4 *>(ring) + (warp * 2 * 3 * 2 * KK) * 32 + lane;  // [stage][array][r][kk][lane]
    const uint32_t mine_at = smem_u32(mine);
    float lse_next = 0.f;  // of token t0 + lane, log2 units
    auto fetch = [&](int t0, int s) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int t = t0 + rq + 8 * r;
            const long long at = row0 * D + (t < t_end ? t * stride : 0) + 8 * c;
            const uint32_t to = mine_at + (s * 3 * 2 * KK + r * KK) * 512;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                cp_async16(to + kk * 512, p.q + at + 32 * kk, t < t_end);
                cp_async16(to + (2 * KK + kk) * 512, p.o + at + 32 * kk, t < t_end);
                cp_async16(to + (4 * KK + kk) * 512, p.dO + at + 32 * kk, t < t_end);
            }
        }
        cp_async_commit();
        lse_next = lane < 16 && t0 + lane < t_end ? p.lse_in[row0 + static_cast<long long>(t0 + lane) * p.Hq] * kLog2eF : 0.f;
    };
    int st = 0;
    if (t_begin + 16 * warp < t_end)
        fetch(t_begin + 16 * warp, 0);
    for (int t0 = t_begin + 16 * warp; t0 < t_end; t0 += 64, st ^= 1) {
        const float lse_now = lse_next;
        if (t0 + 64 < t_end) {
            fetch(t0 + 64, st ^ 1);
            cp_async_wait<1>();
        } else {
            cp_async_wait<0>();
        }
        const bool used = t0 + 15 - p.window >= s0;  // else no row of these sees a sink behind its window
        uint4 Q[2][KK], L[2][KK];
        const uint4 *O[2] = {mine + (st * 3 + 2) * 2 * KK * 32, mine + ((st * 3 + 2) * 2 + 1) * KK * 32};
        float Dq[2];  // D of row rq + 8 r
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int t = t0 + rq + 8 * r;
            const bool in = t < t_end;
            const long long at = row0 * D + t * stride + 8 * c;
            const uint4 *from = mine + (st * 3 * 2 * KK + r * KK) * 32;
            float acc = 0.f;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                const uint4 X = from[kk * 32], F = from[(2 * KK + kk) * 32], G = O[r][kk * 32];
                const uint32_t xw[4] = {X.x, X.y, X.z, X.w}, ow[4] = {F.x, F.y, F.z, F.w};
                const uint32_t gw[4] = {G.x, G.y, G.z, G.w};
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 al = *reinterpret_cast<const float2 *>(ab + 32 * kk + 8 * c + 2 * e);
                    const float2 be = *reinterpret_cast<const float2 *>(ab + D + 32 * kk + 8 * c + 2 * e);
                    const float2 x = unpack_bf16x2(xw[e]), u = unpack_bf16x2(ow[e]), v = unpack_bf16x2(gw[e]);
                    split_q_pair(fmaf(x.x, al.x, be.x), fmaf(x.y, al.y, be.y), hi[e], lo[e]);
                    acc = fmaf(u.x, v.x, fmaf(u.y, v.y, acc));
                }
                // a row behind the last would be beta, which may be infinite: zero, as its weight
                Q[r][kk] = in ? make_uint4(hi[0], hi[1], hi[2], hi[3]) : make_uint4(0, 0, 0, 0);
                L[r][kk] = in ? make_uint4(lo[0], lo[1], lo[2], lo[3]) : make_uint4(0, 0, 0, 0);
                if (in && blockIdx.y == 0) {
                    *reinterpret_cast<uint4 *>(p.q_hi + at + 32 * kk) = Q[r][kk];
                    *reinterpret_cast<uint4 *>(p.q_lo + at + 32 * kk) = L[r][kk];
                }
            }
            acc += __shfl_xor_sync(0xffffffffu, acc, 1);
            Dq[r] = acc + __shfl_xor_sync(0xffffffffu, acc, 2);
        }
        float s[2][4], dp[2][4], lse[2][2], Dr[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[r][e] = dp[r][e] = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = t0 + 8 * r + 2 * c + i;
                lse[r][i] = __shfl_sync(0xffffffffu, lse_now, 8 * r + 2 * c + i);
                Dr[r][i] = __shfl_sync(0xffffffffu, Dq[r], 4 * (2 * c + i));
                if (rq == 0 && t < t_end && blockIdx.y == 0) {
                    p.lse[row0 + static_cast<long long>(t) * p.Hq] = lse[r][i];
                    p.Drow[row0 + static_cast<long long>(t) * p.Hq] = Dr[r][i];
                }
            }
        }
        if (!used)
            continue;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            const uint4 k0 = ka_s[2 * kk][lane], k1 = ka_s[2 * kk + 1][lane];
            const uint4 v0 = va_s[2 * kk][lane], v1 = va_s[2 * kk + 1][lane];
            const uint32_t ka0[4] = {k0.x, k0.y, k0.z, k0.w}, ka1[4] = {k1.x, k1.y, k1.z, k1.w};
            const uint32_t va0[4] = {v0.x, v0.y, v0.z, v0.w}, va1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                mma_16816(s[r], ka0, Q[r][kk].x, Q[r][kk].y);
                mma_16816(s[r], ka1, Q[r][kk].z, Q[r][kk].w);
                mma_16816(s[r], ka0, L[r][kk].x, L[r][kk].y);
                mma_16816(s[r], ka1, L[r][kk].z, L[r][kk].w);
                const uint4 G = O[r][kk * 32];
                mma_16816(dp[r], va0, G.x, G.y);
                mma_16816(dp[r], va1, G.z, G.w);
            }
        }
        uint32_t ph[4], pl[4], sh[4], sl[4];  // P and dS with the sinks on M, tokens on K
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int j = rq + 8 * hf;
                float pr[2], ds[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int t = t0 + 8 * r + 2 * c + i;
                    const bool seen = j < ns && t < t_end && s0 + j <= t - p.window;
                    const float e = fast_exp2(s[r][2 * hf + i] * c2 - lse[r][i]);
                    pr[i] = seen ? e : 0.f;
                    ds[i] = seen ? e * (dp[r][2 * hf + i] - Dr[r][i]) : 0.f;
                }
                split_q_pair(pr[0], pr[1], ph[2 * r + hf], pl[2 * r + hf]);
                split_q_pair(ds[0], ds[1], sh[2 * r + hf], sl[2 * r + hf]);
            }
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            const uint4 G0 = O[0][kk * 32], G1 = O[1][kk * 32];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                auto word = [e](uint4 u) { return e == 0 ? u.x : e == 1 ? u.y : e == 2 ? u.z : u.w; };
                const uint32_t x0 = movmatrix_trans(word(Q[0][kk])), x1 = movmatrix_trans(word(Q[1][kk]));
                mma_16816(y[4 * kk + e], sh, x0, x1);
                mma_16816(y[4 * kk + e], sl, x0, x1);
                mma_16816(y[4 * kk + e], sh, movmatrix_trans(word(L[0][kk])), movmatrix_trans(word(L[1][kk])));
                const uint32_t g0 = movmatrix_trans(word(G0)), g1 = movmatrix_trans(word(G1));
                mma_16816(dv[4 * kk + e], ph, g0, g1);
                mma_16816(dv[4 * kk + e], pl, g0, g1);
            }
        }
    }
    // the four warps' sums, added up in order
    __syncthreads();
    constexpr int PITCH = 2 * D + 8;  // the eight rows of a store in banks of their own
    static_assert(4 * SK_M * PITCH * 4 <= sk_ring<D>);
    float *red = reinterpret_cast<float *>(ring);  // [warp][SK_M][PITCH]: dk, dv
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        float *row = red + (warp * SK_M + rq + 8 * hf) * PITCH;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            const int d = 32 * (i / 4) + 8 * c + 2 * (i % 4);
            *reinterpret_cast<float2 *>(row + d) = make_float2(y[i][2 * hf], y[i][2 * hf + 1]);
            *reinterpret_cast<float2 *>(row + D + d) = make_float2(dv[i][2 * hf], dv[i][2 * hf + 1]);
        }
    }
    __syncthreads();
    float *out = p.part + ((static_cast<long long>(blockIdx.y) * p.B * p.Hq + bh) * chunks + chunk) * SK_M * 2 * D;
    for (int x = threadIdx.x; x < ns * 2 * D; x += 128) {
        const float *at = red + x / (2 * D) * PITCH + x % (2 * D);
        out[x] = ((at[0] + at[SK_M * PITCH]) + at[2 * SK_M * PITCH]) + at[3 * SK_M * PITCH];
    }
}

// one CTA a sink of a (sequence, KV head), a thread a column of dk and of dv
template <int D>
__global__ void __launch_bounds__(2 * D) sink_join_kernel(const SinkBwdParams p, int chunks)
{
    const int j = blockIdx.x, bg = blockIdx.y, b = bg / p.Hkv, g = bg % p.Hkv, G = p.Hq / p.Hkv, d = threadIdx.x;
    const float *src = p.part + (((static_cast<long long>(j / SK_M) * p.B + b) * p.Hq + g * G) * chunks * SK_M + j % SK_M) * 2 * D + d;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // it waits for all grids before it
    float sum = 0.f;
    for (int i0 = 0; i0 < G * chunks; i0 += 16) {  // the heads' chunks follow one another
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            x[i] = i0 + i < G * chunks ? src[static_cast<long long>(i0 + i) * SK_M * 2 * D] : 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            sum += x[i];
    }
    const long long at = ((static_cast<long long>(b) * p.T + j) * p.Hkv + g) * D;
    if (d < D)
        p.dk[at + d] += p.scale * sum;
    else
        p.dv[at + d - D] += sum;
}

// ------------------------------------------------------------------ host side

// four waves of two CTAs on each of 152 SMs, from 64 tokens a CTA to 4096 (64 a warp's step: the accumulators are
// truncated at each)
int sink_chunks(int B, int T, int Hq)
{
    const int most = (T + 63) / 64, least = (T + 4095) / 4096, want = 1216 / (B * Hq);
    return want < least ? least : (want < most ? want : most);
}

template <int D>
cudaError_t launch_t(const SinkDqMaps &qmaps, const SinkBwdMaps &maps, const SinkBwdParams &p, cudaStream_t stream)
{
    const int count = p.sinks < p.T - p.window ? p.sinks : p.T - p.window;  // sinks that some row sees behind its window
    const int chunks = sink_chunks(p.B, p.T, p.Hq);
    if (count > 0) {
        const cudaError_t e = cudaFuncSetAttribute(sink_keys_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, sk_ring<D>);
        if (e != cudaSuccess)
            return e;
        sink_keys_kernel<D><<<dim3(chunks * p.B * p.Hq, (count + SK_M - 1) / SK_M), 128, sk_ring<D>, stream>>>(p, chunks, count);
    } else {
        const long long lanes = static_cast<long long>(p.B) * p.T * p.Hq * (D / 8);
        sink_rows_kernel<D><<<static_cast<unsigned>((lanes + 255) / 256), 256, 0, stream>>>(p);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    if ((e = launch_sink_dq(D, qmaps, p, stream)) != cudaSuccess || (e = launch_sink_dkv(D, maps, p, stream)) != cudaSuccess ||
        count <= 0)
        return e;
    return launch_dependent(sink_join_kernel<D>, dim3(count, p.B * p.Hkv), 2 * D, 0, stream, p, chunks);
}

size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

}  // namespace

size_t sink_bwd_workspace_bytes(int B, int T, int Hq, int D)
{
    const size_t rows = static_cast<size_t>(B) * T * Hq;
    return 2 * up256(2 * rows * D) + 2 * up256(4 * rows) +
           2 * static_cast<size_t>(B) * Hq * sink_chunks(B, T, Hq) * SK_M * 2 * D * sizeof(float);
}

void sink_bwd_workspace(SinkBwdParams &p, int D, void *workspace)
{
    const size_t rows = static_cast<size_t>(p.B) * p.T * p.Hq;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.q_hi = reinterpret_cast<uint16_t *>(ws);
    p.q_lo = reinterpret_cast<uint16_t *>(ws += up256(2 * rows * D));
    p.lse = reinterpret_cast<float *>(ws += up256(2 * rows * D));
    p.Drow = reinterpret_cast<float *>(ws += up256(4 * rows));
    p.part = reinterpret_cast<float *>(ws + up256(4 * rows));
}

cudaError_t launch_sink_bwd(int D, const SinkDqMaps &qmaps, const SinkBwdMaps &maps, const SinkBwdParams &p,
                            cudaStream_t stream)
{
    return D == 128 ? launch_t<128>(qmaps, maps, p, stream) : launch_t<64>(qmaps, maps, p, stream);
}

}  // namespace orthros
