// 8-bit checkpoints of maps: one power-of-two step per w x w window of a
// channel, codes in window order ([C][windows][w*w], windows in (b, i, j)
// order), so that a run of windows of one channel is one contiguous run of
// bytes for the table gradient that reads them.
#include <cuda_bf16.h>

#include "ckpt_common.cuh"
#include "ptx_sm100.cuh"
#include "wbmm_internal.h"

namespace wbmm {

namespace {

__device__ __forceinline__ float ld_f(const float* p) { return *p; }
__device__ __forceinline__ float ld_f(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void st_f(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Element offset of window n (of channel c) in the map.
__device__ __forceinline__ long long window_base(long long n, int c, int C, int H, int W, int w,
                                                 int nh, int nw)
{
    const long long g = n / nw;
    const int j = (int)(n - g * nw);
    const long long b = g / nh;
    const int i = (int)(g - b * nh);
    return ((b * C + c) * H + (long long)i * w) * W + (long long)j * w;
}

// One warp per window.
template <typename T>
__global__ void ckpt_store_kernel(const T* __restrict__ x, uint8_t* __restrict__ codes,
                                  uint8_t* __restrict__ exps, int C, int H, int W, int w, int nh,
                                  int nw, long long nwin)
{
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31, d = w * w;
    const long long total = nwin * C, nwarps = (long long)gridDim.x * (blockDim.x >> 5);
    for (long long k = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); k < total;
         k += nwarps) {
        const int c = (int)(k / nwin);
        const T* src = x + window_base(k - c * nwin, c, C, H, W, w, nh, nw);
        uint32_t top = 0;
        for (int u = lane; u < d; u += 32) {
            const int r = u / w;
            const uint32_t bits =
                __float_as_uint(ld_f(src + (long long)r * W + (u - r * w))) & kAbsMask;
            top = bits > top ? bits : top;
        }
        top = __reduce_max_sync(0xffffffffu, top);
        const uint32_t e = group_exp(top);
        const float inv = inv_step_of(e);
        uint8_t* dst = codes + k * d;
        for (int u = lane; u < d; u += 32) {
            const int r = u / w;
            float v = ld_f(src + (long long)r * W + (u - r * w));
            if (e >= kExpTop)
                v = group_fix(v, e);
            dst[u] = (uint8_t)quant_code(v, inv);
        }
        if (lane == 0)
            exps[k] = (uint8_t)e;
    }
}

template <typename T>
__global__ void ckpt_restore_kernel(const uint8_t* __restrict__ codes,
                                    const uint8_t* __restrict__ exps, T* __restrict__ x, int C,
                                    int H, int W, int w, int nh, int nw, long long nwin)
{
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31, d = w * w;
    const long long total = nwin * C, nwarps = (long long)gridDim.x * (blockDim.x >> 5);
    for (long long k = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); k < total;
         k += nwarps) {
        const int c = (int)(k / nwin);
        T* dst = x + window_base(k - c * nwin, c, C, H, W, w, nh, nw);
        const float step = step_of(exps[k]);
        const uint8_t* src = codes + k * d;
        for (int u = lane; u < d; u += 32) {
            const int r = u / w;
            st_f(dst + (long long)r * W + (u - r * w), code_value(src[u], step));
        }
    }
}

unsigned warp_grid(long long warps, const Launch& L)
{
    const long long blocks = (warps + 3) / 4, most = (long long)L.num_sms * 16;
    return (unsigned)(blocks < most ? blocks : most);
}

}  // namespace

cudaError_t checkpoint_launch(const Geom& g, bool is_bf16, const void* x, uint8_t* codes,
                              uint8_t* exps, const Launch& L)
{
    const long long nwin = g.bands * g.nw;
    const dim3 grid(warp_grid(nwin * g.C, L)), block(128);
    cudaError_t e =
        is_bf16 ? launch_pdl(ckpt_store_kernel<__nv_bfloat16>, grid, block, 0, L.stream,
                             static_cast<const __nv_bfloat16*>(x), codes, exps, g.C, g.H, g.W, g.w,
                             g.nh, g.nw, nwin)
                : launch_pdl(ckpt_store_kernel<float>, grid, block, 0, L.stream,
                             static_cast<const float*>(x), codes, exps, g.C, g.H, g.W, g.w, g.nh,
                             g.nw, nwin);
    if (e != cudaSuccess)
        return e;
    note_launches(1);
    return cudaGetLastError();
}

cudaError_t checkpoint_restore_launch(const Geom& g, bool is_bf16, const uint8_t* codes,
                                      const uint8_t* exps, void* x, const Launch& L)
{
    const long long nwin = g.bands * g.nw;
    const dim3 grid(warp_grid(nwin * g.C, L)), block(128);
    cudaError_t e =
        is_bf16 ? launch_pdl(ckpt_restore_kernel<__nv_bfloat16>, grid, block, 0, L.stream, codes,
                             exps, static_cast<__nv_bfloat16*>(x), g.C, g.H, g.W, g.w, g.nh, g.nw,
                             nwin)
                : launch_pdl(ckpt_restore_kernel<float>, grid, block, 0, L.stream, codes, exps,
                             static_cast<float*>(x), g.C, g.H, g.W, g.w, g.nh, g.nw, nwin);
    if (e != cudaSuccess)
        return e;
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace wbmm
