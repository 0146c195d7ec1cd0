// 8-bit checkpoints of maps: one power-of-two step per w x w window of a
// channel, codes in window order ([C][windows][w*w], windows in (b, i, j)
// order), so that a run of windows of one channel is one contiguous run of
// bytes for the table gradient that reads them.
//
// Bands (the w image rows of one window row of a plane) follow each other in
// the map, and a band's windows follow each other in the codes, so both
// directions move whole bands with contiguous accesses and permute within a
// band in shared memory: a block takes the next bands, at most 512 window rows,
// a thread some of the rows.  The bytes are 3 an element in bf16 and 5 in fp32;
// the instructions, 16 an element in both directions at w = 14 and 28 and 25 at
// w = 7 (bf16, ncu), take 67 to 82% of the issue slots, and the barriers between
// a block's three passes are among its warps' longest waits.  128 x 256 maps of
// 28 x 28 in windows of 14: bf16 stored in 19.4 us (62% of the measured copy
// rate), restored in 17.9 us (67%); fp32 28.8 us (69%) and 28.2 us (71%).  4 rows a
// thread in 128 threads store faster than 2 in 256 (22.0 us) or 8 in 128 (25.6
// us), and restore slower (19.6 us), hence the two block sizes.
#include <cuda_bf16.h>

#include <type_traits>

#include "ckpt_common.cuh"
#include "f32x2.cuh"
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

// One warp per window: bands beyond the block kernels' shared memory.
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

// ------------------------------------------------------------ block kernels
constexpr int kStoreThreads = 128;
constexpr int kRestoreThreads = 256;
constexpr int kBandRows = 512;          // window rows a block, at most (WS > 0)
constexpr int kStoreRows = kBandRows / kStoreThreads;
constexpr int kBandElems = 8192;        // elements of a block's bands, at most

struct BandArgs {
    int B, C, nh, nw, w, W;
    int nb;                 // bands a block
    unsigned bands;         // of all planes
    unsigned div_row;       // ceil(2^32 / (nw w)) and / nw, 0 for a divisor of 1
    unsigned div_nw;
    int unit, units;        // bytes a copy of codes moves, copies a band
    unsigned div_units;
};

// n / d for n d < 2^32, m = ceil(2^32 / d).
__device__ __forceinline__ int fast_div(int n, unsigned m)
{
    return m ? (int)__umulhi((unsigned)n, m) : n;
}

// A window row of the block's bands.
struct WinRow {
    int band, r, j;
    __device__ __forceinline__ WinRow(const BandArgs& P, int k)
    {
        band = fast_div(k, P.div_row);
        const int in = k - band * P.nw * P.w;
        r = fast_div(in, P.div_nw);
        j = in - r * P.nw;
    }
};

// The band's place among the bands in checkpoint order (channels first).
__device__ __forceinline__ unsigned band_place(const BandArgs& P, unsigned f)
{
    const unsigned plane = f / (unsigned)P.nh, i = f - plane * P.nh;
    const unsigned b = plane / (unsigned)P.C, c = plane - b * P.C;
    return (c * P.B + b) * P.nh + i;
}

// The WS values of a window row.  bf16 rows start at an even or an odd
// element: of an odd one the words from the element before are read (within
// the image, which has room in front) and shifted.
template <typename T, int WS>
struct RowVals {
    static constexpr bool F32 = std::is_same<T, float>::value;
    static constexpr int N = F32 ? WS : (WS + 1) / 2;
    uint32_t u[N];      // fp32 bits, or bf16 pairs (a last odd half is zero)

    __device__ __forceinline__ void load(const T* e)
    {
        if constexpr (F32) {
#pragma unroll
            for (int t = 0; t < N; ++t)
                u[t] = __float_as_uint(e[t]);
        } else if constexpr (WS % 2 == 0) {
#pragma unroll
            for (int t = 0; t < N; ++t)
                u[t] = reinterpret_cast<const uint32_t*>(e)[t];
        } else {
            const bool odd = reinterpret_cast<uintptr_t>(e) & 2;
            const uint32_t* p = reinterpret_cast<const uint32_t*>(e - (odd ? 1 : 0));
#pragma unroll
            for (int t = 0; t < N; ++t)
                u[t] = p[t];
            if (odd) {
#pragma unroll
                for (int t = 0; t + 1 < N; ++t)
                    u[t] = __funnelshift_r(u[t], u[t + 1], 16);
                u[N - 1] >>= 16;
            }
            u[N - 1] &= 0xffffu;
        }
    }
    __device__ __forceinline__ uint32_t top() const
    {
        uint32_t m = 0;
#pragma unroll
        for (int t = 0; t < N; ++t)
            m = F32 ? max(m, u[t] & kAbsMask) : max_abs2(m, u[t] & 0x7fff7fffu);
        return F32 ? m : max(m & 0xffff0000u, m << 16);
    }
    __device__ __forceinline__ float value(int t) const
    {
        if constexpr (F32)
            return __uint_as_float(u[t]);
        else
            return __uint_as_float(t & 1 ? u[t / 2] & 0xffff0000u : u[t / 2] << 16);
    }
    // group_fix of every value: exact in bf16 too (127 steps are)
    __device__ __forceinline__ void fix(uint32_t e)
    {
#pragma unroll
        for (int t = 0; t < WS; ++t) {
            const uint32_t b = __float_as_uint(group_fix(value(t), e));
            if constexpr (F32)
                u[t] = b;
            else
                u[t / 2] = t & 1 ? (u[t / 2] & 0xffffu) | (b & 0xffff0000u)
                                 : (u[t / 2] & 0xffff0000u) | (b >> 16);
        }
    }
    __device__ __forceinline__ void store(uint8_t* d, float inv) const
    {
#pragma unroll
        for (int t = 0; t < WS; t += 2) {
            const F2 q = fma2({value(t), t + 1 < WS ? value(t + 1) : 0.0f}, {inv, inv},
                              {12583040.0f, 12583040.0f});
            const uint32_t a = __float_as_uint(q.x), b = __float_as_uint(q.y);
            if constexpr (WS % 2 == 0) {
                reinterpret_cast<uint16_t*>(d)[t / 2] = (uint16_t)__byte_perm(a, b, 0x0040);
            } else {
                d[t] = (uint8_t)a;
                if (t + 1 < WS)
                    d[t + 1] = (uint8_t)b;
            }
        }
    }
};

template <typename T, int WS>
__device__ __forceinline__ void restore_row(T* e, const uint8_t* c, float st)
{
    constexpr bool F32 = std::is_same<T, float>::value;
#pragma unroll
    for (int t = 0; t < WS; t += 2) {
        uint32_t a, b;
        if constexpr (WS % 2 == 0) {
            const uint32_t u = reinterpret_cast<const uint16_t*>(c)[t / 2];
            a = __byte_perm(u, 0x4b000000u, 0x7440);
            b = __byte_perm(u, 0x4b000000u, 0x7441);
        } else {
            a = 0x4b000000u | c[t];
            b = t + 1 < WS ? 0x4b000000u | c[t + 1] : a;
        }
        // 2^23 + code, less 2^23 + 128, times the step: all exact
        const F2 v = mul2(add2({__uint_as_float(a), __uint_as_float(b)}, {-8388736.0f, -8388736.0f}),
                          {st, st});
        if constexpr (F32) {
            e[t] = v.x;
            if (t + 1 < WS)
                e[t + 1] = v.y;
        } else if constexpr (WS % 2 == 0) {
            // exact in bf16: the upper halves
            reinterpret_cast<uint32_t*>(e)[t / 2] =
                __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632);
        } else {
            reinterpret_cast<uint16_t*>(e)[t] = (uint16_t)(__float_as_uint(v.x) >> 16);
            if (t + 1 < WS)
                reinterpret_cast<uint16_t*>(e)[t + 1] = (uint16_t)(__float_as_uint(v.y) >> 16);
        }
    }
}

// WS: the window size, 2 to 16 or 28 as the tensor-core kernels compile for,
// or 0 for any other (w as given).
template <typename T, int WS>
__global__ void __launch_bounds__(kStoreThreads)
    ckpt_store_bands_kernel(const T* __restrict__ x, uint8_t* __restrict__ codes,
                            uint8_t* __restrict__ exps, const BandArgs P)
{
    extern __shared__ __align__(16) uint8_t smem[];
    const int w = WS ? WS : P.w, tid = threadIdx.x;
    const int bn = w * P.W;                                 // elements a band
    const unsigned f0 = blockIdx.x * (unsigned)P.nb;
    const int nb = (int)min(P.bands - f0, (unsigned)P.nb);
    const int windows = nb * P.nw, rows = windows * w;
    // the map's elements, with their offset from a 16-byte boundary; codes;
    // the windows' largest magnitudes
    uint8_t* img = smem + 16;
    uint8_t* cds = img + (P.nb * bn * (int)sizeof(T) + 31) / 16 * 16;
    uint32_t* top = reinterpret_cast<uint32_t*>(cds + (P.nb * bn + 15) / 16 * 16);
    unsigned* place = reinterpret_cast<unsigned*>(top + P.nb * P.nw);
    for (int k = tid; k < nb; k += kStoreThreads)
        place[k] = band_place(P, f0 + k);
    for (int k = tid; k < windows; k += kStoreThreads)
        top[k] = 0u;
    grid_dep_wait();
    grid_dep_launch();
    const T* src = x + (long long)f0 * bn;
    const int off = (int)(reinterpret_cast<uintptr_t>(src) & 15);
    const int bytes = nb * bn * (int)sizeof(T);
    for (int lo = 16 * tid - off; lo < bytes; lo += 16 * kStoreThreads) {
        const uint8_t* from = reinterpret_cast<const uint8_t*>(src) + lo;
        if (lo >= 0 && lo + 16 <= bytes) {
            cp_async_16z(smem_u32(img + off + lo), from, 16u);
        } else {
            // the first and last partial 16 bytes, by elements
            for (int q = 0; q < 16; q += (int)sizeof(T))
                if (lo + q >= 0 && lo + q < bytes)
                    *reinterpret_cast<T*>(img + off + lo + q) = *reinterpret_cast<const T*>(from + q);
        }
    }
    cp_async_wait_all();
    __syncthreads();
    const T* map = reinterpret_cast<const T*>(img + off);
    if constexpr (WS > 0) {
        // each thread's window rows stay in registers between the two passes
        RowVals<T, WS> val[kStoreRows];
        int win[kStoreRows], at[kStoreRows];
#pragma unroll
        for (int m = 0; m < kStoreRows; ++m) {
            const int k = tid + m * kStoreThreads;
            if (k < rows) {
                const WinRow q(P, k);
                win[m] = q.band * P.nw + q.j;
                at[m] = q.band * bn + (q.j * WS + q.r) * WS;
                val[m].load(map + q.band * bn + q.r * P.W + q.j * WS);
                atomicMax(&top[win[m]], val[m].top());
            }
        }
        __syncthreads();
#pragma unroll
        for (int m = 0; m < kStoreRows; ++m) {
            if (tid + m * kStoreThreads < rows) {
                const uint32_t ex = group_exp(top[win[m]]);
                if (ex >= kExpTop)
                    val[m].fix(ex);
                val[m].store(cds + at[m], inv_step_of(ex));
            }
        }
    } else {
        for (int k = tid; k < rows; k += kStoreThreads) {
            const WinRow q(P, k);
            const T* e = map + q.band * bn + q.r * P.W + q.j * w;
            uint32_t m = 0;
            for (int t = 0; t < w; ++t)
                m = max(m, __float_as_uint(ld_f(e + t)) & kAbsMask);
            atomicMax(&top[q.band * P.nw + q.j], m);
        }
        __syncthreads();
        for (int k = tid; k < rows; k += kStoreThreads) {
            const WinRow q(P, k);
            const T* e = map + q.band * bn + q.r * P.W + q.j * w;
            const uint32_t ex = group_exp(top[q.band * P.nw + q.j]);
            const float inv = inv_step_of(ex);
            uint8_t* d = cds + q.band * bn + (q.j * w + q.r) * w;
            for (int t = 0; t < w; ++t) {
                float v = ld_f(e + t);
                if (ex >= kExpTop)
                    v = group_fix(v, ex);
                d[t] = (uint8_t)quant_code(v, inv);
            }
        }
    }
    __syncthreads();
    for (int k = tid; k < nb * P.units; k += kStoreThreads) {
        const int band = fast_div(k, P.div_units);
        const int at = (k - band * P.units) * P.unit;
        uint8_t* out = codes + (long long)place[band] * bn + at;
        const uint8_t* in = cds + band * bn + at;
        if (P.unit == 8)
            *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(in);
        else if (P.unit == 4)
            *reinterpret_cast<uint32_t*>(out) = *reinterpret_cast<const uint32_t*>(in);
        else
            *out = *in;
    }
    for (int k = tid; k < windows; k += kStoreThreads) {
        const int band = fast_div(k, P.div_nw);
        exps[(long long)place[band] * P.nw + (k - band * P.nw)] = (uint8_t)group_exp(top[k]);
    }
}

template <typename T, int WS>
__global__ void __launch_bounds__(kRestoreThreads)
    ckpt_restore_bands_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ exps,
                              T* __restrict__ x, const BandArgs P)
{
    extern __shared__ __align__(16) uint8_t smem[];
    const int w = WS ? WS : P.w, tid = threadIdx.x;
    const int bn = w * P.W;
    const unsigned f0 = blockIdx.x * (unsigned)P.nb;
    const int nb = (int)min(P.bands - f0, (unsigned)P.nb);
    const int windows = nb * P.nw, rows = windows * w;
    uint8_t* img = smem + 16;
    uint8_t* cds = img + (P.nb * bn * (int)sizeof(T) + 31) / 16 * 16;
    float* step = reinterpret_cast<float*>(cds + (P.nb * bn + 15) / 16 * 16);
    unsigned* place = reinterpret_cast<unsigned*>(step + P.nb * P.nw);
    for (int k = tid; k < nb; k += kRestoreThreads)
        place[k] = band_place(P, f0 + k);
    __syncthreads();
    grid_dep_wait();
    grid_dep_launch();
    for (int k = tid; k < nb * P.units; k += kRestoreThreads) {
        const int band = fast_div(k, P.div_units);
        const int at = (k - band * P.units) * P.unit;
        const uint8_t* in = codes + (long long)place[band] * bn + at;
        uint8_t* to = cds + band * bn + at;
        if (P.unit == 8)
            cp_async_8(smem_u32(to), in);
        else if (P.unit == 4)
            cp_async_4(smem_u32(to), in);
        else
            *to = *in;
    }
    for (int k = tid; k < windows; k += kRestoreThreads) {
        const int band = fast_div(k, P.div_nw);
        step[k] = step_of(exps[(long long)place[band] * P.nw + (k - band * P.nw)]);
    }
    cp_async_wait_all();
    __syncthreads();
    T* dst = x + (long long)f0 * bn;
    const int off = (int)(reinterpret_cast<uintptr_t>(dst) & 15);
    T* map = reinterpret_cast<T*>(img + off);
    for (int k = tid; k < rows; k += kRestoreThreads) {
        const WinRow q(P, k);
        T* e = map + q.band * bn + q.r * P.W + q.j * w;
        const float st = step[q.band * P.nw + q.j];
        const uint8_t* c = cds + q.band * bn + (q.j * w + q.r) * w;
        if constexpr (WS > 0) {
            restore_row<T, WS>(e, c, st);
        } else {
            for (int t = 0; t < w; ++t)
                st_f(e + t, code_value(c[t], st));
        }
    }
    __syncthreads();
    const int bytes = nb * bn * (int)sizeof(T);
    for (int lo = 16 * tid - off; lo < bytes; lo += 16 * kRestoreThreads) {
        uint8_t* to = reinterpret_cast<uint8_t*>(dst) + lo;
        const uint8_t* from = img + off + lo;
        if (lo >= 0 && lo + 16 <= bytes) {
            *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(from);
        } else {
            for (int q = 0; q < 16; q += (int)sizeof(T))
                if (lo + q >= 0 && lo + q < bytes)
                    *reinterpret_cast<T*>(to + q) = *reinterpret_cast<const T*>(from + q);
        }
    }
}

unsigned ceil_recip(int d) { return d == 1 ? 0u : (unsigned)(((1ull << 32) + d - 1) / d); }

// The block kernels' arguments; false where a band does not fit.
bool band_args(const Geom& g, size_t sz, int num_sms, BandArgs* P, size_t* smem)
{
    const long long bn = (long long)g.w * g.W;
    if (bn > kBandElems)
        return false;
    P->B = g.B; P->C = g.C; P->nh = g.nh; P->nw = g.nw; P->w = g.w; P->W = g.W;
    if (g.bands * g.C >= (1ll << 31))
        return false;
    P->bands = (unsigned)(g.bands * g.C);
    const int rows = g.nw * g.w;
    // fewer rows a block where that leaves SMs without blocks
    long long nb = kBandRows / rows;
    if (P->bands < nb * 4 * num_sms)
        nb = kBandRows / 2 / rows;
    nb = nb < 1 ? 1 : nb > kBandElems / bn ? kBandElems / bn : nb;
    P->nb = (int)nb;
    P->div_row = ceil_recip(rows);
    P->div_nw = ceil_recip(g.nw);
    P->unit = bn % 8 == 0 ? 8 : bn % 4 == 0 ? 4 : 1;
    P->units = (int)bn / P->unit;
    P->div_units = ceil_recip(P->units);
    *smem = 16 + (nb * bn * sz + 31) / 16 * 16 + (nb * bn + 15) / 16 * 16 + (size_t)nb * (g.nw + 1) * 4;
    return *smem <= 48 * 1024;
}

template <template <typename, int> class KernelT, typename T, int WS>
auto pick_kernel(int w)
{
    if constexpr (WS < 2)
        return KernelT<T, 0>::get();
    else
        return w == WS ? KernelT<T, WS>::get() : pick_kernel<KernelT, T, WS - 1>(w);
}

template <template <typename, int> class KernelT, typename T, typename... Args>
cudaError_t band_launch(const BandArgs& P, int threads, size_t smem, const Launch& L, Args... args)
{
    const dim3 grid((P.bands + P.nb - 1) / P.nb), block(threads);
    // the compiled sizes hold a block's window rows in registers
    const bool fits = P.nb * P.nw * P.w <= kBandRows;
    return launch_pdl(!fits        ? KernelT<T, 0>::get()
                      : P.w == 28 ? KernelT<T, 28>::get()
                                  : pick_kernel<KernelT, T, 16>(P.w),
                      grid, block, smem, L.stream, args..., P);
}

template <typename T, int WS>
struct StoreKernel {
    static constexpr auto get() { return &ckpt_store_bands_kernel<T, WS>; }
};

template <typename T, int WS>
struct RestoreKernel {
    static constexpr auto get() { return &ckpt_restore_bands_kernel<T, WS>; }
};

unsigned warp_grid(long long warps, const Launch& L)
{
    const long long blocks = (warps + 3) / 4, most = (long long)L.num_sms * 16;
    return (unsigned)(blocks < most ? blocks : most);
}

}  // namespace

cudaError_t checkpoint_launch(const Geom& g, bool is_bf16, const void* x, uint8_t* codes,
                              uint8_t* exps, const Launch& L)
{
    BandArgs P;
    size_t smem;
    cudaError_t e;
    const long long nwin = g.bands * g.nw;
    const dim3 grid(warp_grid(nwin * g.C, L)), block(128);
    if (band_args(g, is_bf16 ? 2 : 4, L.num_sms, &P, &smem))
        e = is_bf16 ? band_launch<StoreKernel, __nv_bfloat16>(
                          P, kStoreThreads, smem, L, static_cast<const __nv_bfloat16*>(x), codes, exps)
                    : band_launch<StoreKernel, float>(P, kStoreThreads, smem, L,
                                                      static_cast<const float*>(x), codes, exps);
    else
        e = is_bf16 ? launch_pdl(ckpt_store_kernel<__nv_bfloat16>, grid, block, 0, L.stream,
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
    BandArgs P;
    size_t smem;
    cudaError_t e;
    const long long nwin = g.bands * g.nw;
    const dim3 grid(warp_grid(nwin * g.C, L)), block(128);
    if (band_args(g, is_bf16 ? 2 : 4, L.num_sms, &P, &smem))
        e = is_bf16 ? band_launch<RestoreKernel, __nv_bfloat16>(P, kRestoreThreads, smem, L, codes, exps,
                                                                static_cast<__nv_bfloat16*>(x))
                    : band_launch<RestoreKernel, float>(P, kRestoreThreads, smem, L, codes, exps,
                                                        static_cast<float*>(x));
    else
        e = is_bf16 ? launch_pdl(ckpt_restore_kernel<__nv_bfloat16>, grid, block, 0, L.stream, codes,
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
