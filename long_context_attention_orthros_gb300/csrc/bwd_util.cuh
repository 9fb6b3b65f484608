// bwd_util.cuh -- shared-memory tiles, asynchronous copies and waits of the gradient kernels.
#pragma once

#include "common.cuh"

namespace orthros {

namespace {

constexpr float kLog2eF = 1.4426950408889634f;

// [rows][D] bf16 tile in shared memory as D/64 slabs of rows x 128 bytes, 128-byte swizzle
__device__ __forceinline__ uint32_t tile_off(int row, int col, int slab_bytes)
{
    return static_cast<uint32_t>((col / 64) * slab_bytes) + sw128_offset(row, (col % 64) / 8);
}

// 16-byte asynchronous copy global -> shared; valid = false writes zeros (nothing is read)
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint8_t *align1024(uint8_t *p)
{
    return p + ((1024u - (smem_u32(p) & 1023u)) & 1023u);
}

// wait on an mbarrier as a whole warp (lane 0 polls); false after the time limit
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity)
{
    bool ok = true;
    if ((threadIdx.x & 31) == 0)
        ok = mbar_wait(bar, parity);
    return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}

// two fp32 values as a bf16 high part and a bf16 residual each
__device__ __forceinline__ void split_pair2(float2 x, uint32_t &hi, uint32_t &lo)
{
    hi = pack_bf16x2(x.x, x.y);
    const float2 r = ffma2(unpack_bf16x2(hi), make_float2(-1.f, -1.f), x);
    lo = pack_bf16x2(r.x, r.y);
}

// Launch as the programmatic dependent of the kernel before it in the stream.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace
}  // namespace orthros
