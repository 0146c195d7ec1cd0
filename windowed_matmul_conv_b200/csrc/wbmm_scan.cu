// Gated linear recurrence along the rows of a [B, C, L] tensor:
//   f = 1 / (1 + exp(-g)),  h_t = f_t h_{t-1} + (1 - f_t) v_t,  y_t = h_t
// and its backward pass.
//
// A step is the affine map h -> f h + u, u = (1 - f) v, and maps compose:
// (A1, H1) then (A2, H2) is (A1 A2, A2 H1 + H2).  A warp takes a tile of 256
// successive positions of one row, 8 a lane: each lane composes its 8 steps,
// the lanes' maps are joined by an inclusive scan in 5 exchanges, and each
// lane replays its 8 steps from its exact starting state.  The order of every
// product and sum is fixed by the position within the row, so results are
// bit-identical from run to run.
//
// The backward pass needs h_{t-1}: it replays a tile from the state before it,
// which the forward call keeps (one fp32 value per 256 positions), beside the
// reversed recurrence of c_t = f_t (dy_t + c_{t+1}).
//
// 1 - f is e f with e = exp(-g), not a difference, so that it keeps its
// relative accuracy where f is close to 1; exp's argument is held at 80 at
// most, where f (1.8e-35) is zero for every purpose and e f is 1.
#include <cuda_bf16.h>

#include <type_traits>

#include "ckpt_common.cuh"
#include "ptx_sm100.cuh"
#include "wbmm.h"
#include "wbmm_internal.h"

namespace wbmm {

namespace {

constexpr uint32_t kFull = 0xffffffffu;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float min_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// f = sigmoid(g), i = 1 - f.
template <typename T>
__device__ __forceinline__ void gate(float g, float& f, float& i)
{
    const float a = min_nan(-g, 80.0f);
    if constexpr (std::is_same<T, float>::value) {
        const float e = expf(a);
        f = __frcp_rn(1.0f + e);
        i = e * f;
    } else {
        // the fast forms' errors, about 2^-21, are far below bf16's 2^-8
        const float e = __expf(a);
        f = __fdividef(1.0f, 1.0f + e);
        i = e * f;
    }
}

// Positions of row b*C + c that the sequence has.
__device__ __forceinline__ int row_len(const int* lengths, long long row, int C, int L)
{
    if (!lengths)
        return L;
    const int n = lengths[row / C];
    return n < 0 ? 0 : n > L ? L : n;
}

// Elements [t, t + cnt) of a row, zeros up to 8.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int cnt, float (&x)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        x[j] = j < cnt ? to_f(p[j]) : 0.0f;
}

template <typename T>
__device__ __forceinline__ void store8(T* p, int cnt, const float (&x)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < cnt)
            put(p + j, x[j]);
}

__device__ __forceinline__ int clamp8(long long n) { return n < 0 ? 0 : n > 8 ? 8 : (int)n; }

// Gates and inputs of a lane's 8 positions; the steps past cnt are the
// identity (f = 1, u = 0, i = 0).
template <typename T>
__device__ __forceinline__ void gates8(const float (&g)[8], int cnt, float (&f)[8], float (&i)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        gate<T>(g[j], f[j], i[j]);
        if (j >= cnt) {
            f[j] = 1.0f;
            i[j] = 0.0f;
        }
    }
}

// Inclusive scan of the lanes' maps (forward: lane order; reverse: from the
// last lane down), then the map of everything before the lane.
template <bool REV>
__device__ __forceinline__ void warp_scan(float& A, float& H, float& Aex, float& Hex, int lane)
{
    const int pos = REV ? 31 - lane : lane;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float a = REV ? __shfl_down_sync(kFull, A, o) : __shfl_up_sync(kFull, A, o);
        const float h = REV ? __shfl_down_sync(kFull, H, o) : __shfl_up_sync(kFull, H, o);
        if (pos >= o) {
            H = fmaf(A, h, H);
            A *= a;
        }
    }
    Aex = REV ? __shfl_down_sync(kFull, A, 1) : __shfl_up_sync(kFull, A, 1);
    Hex = REV ? __shfl_down_sync(kFull, H, 1) : __shfl_up_sync(kFull, H, 1);
    if (pos == 0) {
        Aex = 1.0f;
        Hex = 0.0f;
    }
}

// 8-bit form of 64 successive positions (8 lanes of 8).
__device__ __forceinline__ void encode8(const float (&x)[8], int cnt, bool head, uint8_t* codes,
                                        uint8_t* exp)
{
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t b = __float_as_uint(x[j]) & kAbsMask;
        top = b > top ? b : top;
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        const uint32_t b = __shfl_xor_sync(kFull, top, o);
        top = b > top ? b : top;
    }
    const uint32_t e = group_exp(top);
    const float inv = inv_step_of(e);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < cnt)
            codes[j] = (uint8_t)quant_code(e >= kExpTop ? group_fix(x[j], e) : x[j], inv);
    if (head && cnt > 0)
        *exp = (uint8_t)e;
}

__device__ __forceinline__ void decode8(const uint8_t* codes, const uint8_t* exp, int cnt,
                                        float (&x)[8])
{
    const float step = cnt > 0 ? step_of(*exp) : 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        x[j] = j < cnt ? code_value(codes[j], step) : 0.0f;
}

// One warp per row.
template <typename T>
__global__ void __launch_bounds__(128) scan_fwd_kernel(const ScanArgs P)
{
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= P.rows)
        return;
    const int n = row_len(P.lengths, row, P.C, P.L);
    const T* v = static_cast<const T*>(P.v) + row * P.L;
    const T* g = static_cast<const T*>(P.g) + row * P.L;
    T* y = static_cast<T*>(P.y) + row * P.L;
    const long long ntile = (P.L + kScanTile - 1ll) / kScanTile;
    const long long ngrp = (P.L + WBMM_SEQ_GROUP - 1ll) / WBMM_SEQ_GROUP;
    float h = P.h0 ? P.h0[row] : 0.0f;
    for (long long t = 0; t < ntile; ++t) {
        const long long t0 = t * kScanTile + lane * 8;
        const int cnt = clamp8(n - t0), all = clamp8(P.L - t0);
        float xv[8], xg[8], f[8], i[8];
        load8(v + t0, cnt, xv);
        load8(g + t0, cnt, xg);
        gates8<T>(xg, cnt, f, i);
        float A = 1.0f, H = 0.0f, Aex, Hex;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            H = fmaf(f[j], H, i[j] * xv[j]);
            A *= f[j];
        }
        warp_scan<false>(A, H, Aex, Hex, lane);
        if (P.states && lane == 0 && t * kScanTile < n)
            P.states[row * ntile + t] = h;
        float s = fmaf(Aex, h, Hex), out[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s = fmaf(f[j], s, i[j] * xv[j]);
            out[j] = j < cnt ? s : 0.0f;
        }
        store8(y + t0, all, out);
        if (P.v_codes) {
            const long long gi = row * ngrp + t0 / WBMM_SEQ_GROUP;
            encode8(xv, all, (lane & 7) == 0, P.v_codes + row * P.L + t0, P.v_exps + gi);
            encode8(xg, all, (lane & 7) == 0, P.g_codes + row * P.L + t0, P.g_exps + gi);
        }
        h = __shfl_sync(kFull, s, 31);
    }
    if (P.hT && lane == 0)
        P.hT[row] = h;
}

template <typename T, bool CODES>
__global__ void __launch_bounds__(128) scan_bwd_kernel(const ScanArgs P)
{
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= P.rows)
        return;
    const int n = row_len(P.lengths, row, P.C, P.L);
    const T* v = static_cast<const T*>(P.v) + row * P.L;
    const T* g = static_cast<const T*>(P.g) + row * P.L;
    const T* dy = static_cast<const T*>(P.dy) + row * P.L;
    T* dv = static_cast<T*>(P.dv) + row * P.L;
    T* dg = static_cast<T*>(P.dg) + row * P.L;
    const long long ntile = (P.L + kScanTile - 1ll) / kScanTile;
    const long long ngrp = (P.L + WBMM_SEQ_GROUP - 1ll) / WBMM_SEQ_GROUP;
    float c = P.h0 ? P.h0[row] : 0.0f;
    for (long long t = ntile - 1; t >= 0; --t) {
        const long long t0 = t * kScanTile + lane * 8;
        const int cnt = clamp8(n - t0), all = clamp8(P.L - t0);
        float xv[8], xg[8], d[8], f[8], i[8];
        if constexpr (CODES) {
            const long long gi = row * ngrp + t0 / WBMM_SEQ_GROUP;
            decode8(P.v_codes + row * P.L + t0, P.v_exps + gi, cnt, xv);
            decode8(P.g_codes + row * P.L + t0, P.g_exps + gi, cnt, xg);
        } else {
            load8(v + t0, cnt, xv);
            load8(g + t0, cnt, xg);
        }
        load8(dy + t0, cnt, d);
        gates8<T>(xg, cnt, f, i);
        const float h = t * kScanTile < n ? P.states[row * ntile + t] : 0.0f;
        float A = 1.0f, H = 0.0f, Aex, Hex;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            H = fmaf(f[j], H, i[j] * xv[j]);
            A *= f[j];
        }
        float Ar = A, D = 0.0f, Dex;
#pragma unroll
        for (int j = 7; j >= 0; --j)
            D = f[j] * (d[j] + D);
        warp_scan<false>(A, H, Aex, Hex, lane);
        float s = fmaf(Aex, h, Hex), before[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            before[j] = s;
            s = fmaf(f[j], s, i[j] * xv[j]);
        }
        warp_scan<true>(Ar, D, Aex, Dex, lane);
        float cc = fmaf(Aex, c, Dex), ov[8], og[8];
#pragma unroll
        for (int j = 7; j >= 0; --j) {
            const float dh = d[j] + cc;
            const float di = dh * i[j];
            cc = f[j] * dh;
            ov[j] = di;
            og[j] = di * f[j] * (before[j] - xv[j]);
        }
        // i is 0 past the sequence's end, but a state that overflowed would
        // still make NaN of it
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j >= cnt)
                ov[j] = og[j] = 0.0f;
        store8(dv + t0, all, ov);
        store8(dg + t0, all, og);
        c = __shfl_sync(kFull, cc, 0);
    }
    if (P.hT && lane == 0)
        P.hT[row] = c;
}

// One position of every row; one thread a row.
template <typename T>
__global__ void __launch_bounds__(128)
    scan_step_kernel(const T* __restrict__ v, const T* __restrict__ g, const float* h, T* y,
                     float* h_next, long long rows)
{
    grid_dep_wait();
    grid_dep_launch();
    const long long r = (long long)blockIdx.x * 128 + threadIdx.x;
    if (r >= rows)
        return;
    float f, i;
    gate<T>(to_f(g[r]), f, i);
    const float s = fmaf(f, h[r], i * to_f(v[r]));
    put(y + r, s);
    h_next[r] = s;
}

cudaError_t done(cudaError_t e)
{
    if (e != cudaSuccess)
        return e;
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t scan_forward_launch(const ScanArgs& A, bool is_bf16, const Launch& L)
{
    const dim3 grid((unsigned)((A.rows + 3) / 4)), block(128);
    return done(is_bf16 ? launch_pdl(scan_fwd_kernel<__nv_bfloat16>, grid, block, 0, L.stream, A)
                        : launch_pdl(scan_fwd_kernel<float>, grid, block, 0, L.stream, A));
}

cudaError_t scan_backward_launch(const ScanArgs& A, bool is_bf16, const Launch& L)
{
    const dim3 grid((unsigned)((A.rows + 3) / 4)), block(128);
    if (A.v_codes)
        return done(is_bf16
                        ? launch_pdl(scan_bwd_kernel<__nv_bfloat16, true>, grid, block, 0, L.stream, A)
                        : launch_pdl(scan_bwd_kernel<float, true>, grid, block, 0, L.stream, A));
    return done(is_bf16
                    ? launch_pdl(scan_bwd_kernel<__nv_bfloat16, false>, grid, block, 0, L.stream, A)
                    : launch_pdl(scan_bwd_kernel<float, false>, grid, block, 0, L.stream, A));
}

cudaError_t scan_step_launch(const void* v, const void* g, const float* h, void* y, float* h_next,
                             long long rows, bool is_bf16, const Launch& L)
{
    const dim3 grid((unsigned)((rows + 127) / 128)), block(128);
    return done(
        is_bf16 ? launch_pdl(scan_step_kernel<__nv_bfloat16>, grid, block, 0, L.stream,
                             static_cast<const __nv_bfloat16*>(v),
                             static_cast<const __nv_bfloat16*>(g), h,
                             static_cast<__nv_bfloat16*>(y), h_next, rows)
                : launch_pdl(scan_step_kernel<float>, grid, block, 0, L.stream,
                             static_cast<const float*>(v), static_cast<const float*>(g), h,
                             static_cast<float*>(y), h_next, rows));
}

}  // namespace wbmm
