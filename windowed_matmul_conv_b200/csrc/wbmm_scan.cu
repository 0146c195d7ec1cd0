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

__device__ __forceinline__ int clamp8(long long n) { return n < 0 ? 0 : n > 8 ? 8 : (int)n; }

// Eight successive elements as they sit in memory.  VEC: rows start at
// 16-byte boundaries and hold a multiple of 8 elements, so a lane's elements
// are whole 16-byte vectors.  Otherwise a lane takes 4-byte words (of a bf16
// row that starts at an odd element: 4 words from the element before, which
// belongs to the tensor, and the last element by itself), which costs no
// shuffles; the words of neighbouring lanes share their sectors.
template <typename T>
struct Raw {
    static constexpr int N = 2 * (int)sizeof(T);    // 32-bit words
    uint32_t w[N];
};

template <bool VEC, typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p, int cnt)
{
    Raw<T> r;
#pragma unroll
    for (int k = 0; k < Raw<T>::N; ++k)
        r.w[k] = 0u;
    if constexpr (VEC) {
        if (cnt > 0) {
#pragma unroll
            for (int k = 0; k < Raw<T>::N; k += 4) {
                const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + k / 4);
                r.w[k] = q.x; r.w[k + 1] = q.y; r.w[k + 2] = q.z; r.w[k + 3] = q.w;
            }
        }
    } else if constexpr (sizeof(T) == 4) {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < cnt)
                r.w[k] = __ldg(q + k);
    } else if (cnt == 8) {
        if ((reinterpret_cast<uintptr_t>(p) & 2) == 0) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                r.w[k] = __ldg(reinterpret_cast<const uint32_t*>(p) + k);
        } else {
            const uint32_t* q = reinterpret_cast<const uint32_t*>(p - 1);
            uint32_t u[5];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                u[k] = __ldg(q + k);
            u[4] = __ldg(reinterpret_cast<const unsigned short*>(p) + 7);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                r.w[k] = __funnelshift_r(u[k], u[k + 1], 16);
        }
    } else {
        const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < cnt)
                r.w[k / 2] |= (uint32_t)__ldg(q + k) << (16 * (k & 1));
    }
    return r;
}

// As floats, zeros from cnt on.
template <typename T>
__device__ __forceinline__ void unpack8(const Raw<T>& r, int cnt, float (&x)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if constexpr (sizeof(T) == 4)
            x[j] = __uint_as_float(r.w[j]);
        else
            x[j] = __uint_as_float(j & 1 ? r.w[j / 2] & 0xffff0000u : r.w[j / 2] << 16);
    }
    if (cnt < 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j >= cnt)
                x[j] = 0.0f;
    }
}

template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* p, int cnt, const float (&x)[8])
{
    if (cnt <= 0)
        return;
    if constexpr (sizeof(T) == 4) {
        if constexpr (VEC) {
            reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
            reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < cnt)
                    p[j] = x[j];
        }
    } else {
        // even and odd elements paired from both alignments
        if (VEC || (cnt == 8 && (reinterpret_cast<uintptr_t>(p) & 2) == 0)) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const __nv_bfloat162 q = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
                w[k] = reinterpret_cast<const uint32_t&>(q);
            }
            if constexpr (VEC) {
                *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    reinterpret_cast<uint32_t*>(p)[k] = w[k];
            }
        } else if (cnt == 8) {
            put(p, x[0]);
#pragma unroll
            for (int k = 0; k < 3; ++k)
                *reinterpret_cast<__nv_bfloat162*>(p + 1 + 2 * k) =
                    __floats2bfloat162_rn(x[2 * k + 1], x[2 * k + 2]);
            put(p + 7, x[7]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < cnt)
                    put(p + j, x[j]);
        }
    }
}

// Gates and inputs of a lane's 8 positions; the steps past cnt are the
// identity (f = 1, i = 0).
template <typename T>
__device__ __forceinline__ void gates8(const float (&g)[8], int cnt, float (&f)[8], float (&i)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        gate<T>(g[j], f[j], i[j]);
    if (cnt < 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j >= cnt) {
                f[j] = 1.0f;
                i[j] = 0.0f;
            }
    }
}

// Inclusive scan of the maps of S lanes (forward: lane order; REV: from the
// last lane down), and the map of everything before the lane.
template <int S, bool REV>
__device__ __forceinline__ void lane_scan(float& A, float& H, float& Aex, float& Hex, int sub)
{
    const int pos = REV ? S - 1 - sub : sub;
#pragma unroll
    for (int o = 1; o < S; o <<= 1) {
        const float a = REV ? __shfl_down_sync(kFull, A, o, S) : __shfl_up_sync(kFull, A, o, S);
        const float h = REV ? __shfl_down_sync(kFull, H, o, S) : __shfl_up_sync(kFull, H, o, S);
        if (pos >= o) {
            H = fmaf(A, h, H);
            A *= a;
        }
    }
    Aex = 1.0f;
    Hex = 0.0f;
    if constexpr (S > 1) {
        const float a = REV ? __shfl_down_sync(kFull, A, 1, S) : __shfl_up_sync(kFull, A, 1, S);
        const float h = REV ? __shfl_down_sync(kFull, H, 1, S) : __shfl_up_sync(kFull, H, 1, S);
        if (pos > 0) {
            Aex = a;
            Hex = h;
        }
    }
}

// 8-bit form of 64 successive positions: 8 lanes of 8 (all the row's lanes
// where it has fewer).
template <int S, bool VEC>
__device__ __forceinline__ void encode8(const float (&x)[8], int cnt, int sub, uint8_t* codes,
                                        uint8_t* exp)
{
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t b = __float_as_uint(x[j]) & kAbsMask;
        top = b > top ? b : top;
    }
#pragma unroll
    for (int o = 1; o < (S < 8 ? S : 8); o <<= 1) {
        const uint32_t b = __shfl_xor_sync(kFull, top, o);
        top = b > top ? b : top;
    }
    const uint32_t e = group_exp(top);
    const float inv = inv_step_of(e);
    uint32_t q[8];
    if (e >= kExpTop) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            q[j] = quant_code(group_fix(x[j], e), inv);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            q[j] = quant_code(x[j], inv);
    }
    if (cnt > 0 && (sub & 7) == 0)
        *exp = (uint8_t)e;
    if constexpr (VEC) {
        if (cnt > 0) {
            uint2 w;
            w.x = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
            w.y = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
            *reinterpret_cast<uint2*>(codes) = w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < cnt)
                codes[j] = (uint8_t)q[j];
    }
}

// Eight codes and their group's exponent byte as they sit in memory.
struct RawCodes {
    uint32_t w[2];
    uint32_t e;
};

template <bool VEC>
__device__ __forceinline__ RawCodes load_codes(const uint8_t* codes, const uint8_t* exp, int cnt)
{
    RawCodes r = {{0u, 0u}, 0u};
    if (cnt > 0) {
        r.e = __ldg(exp);
        if constexpr (VEC) {
            const uint2 q = __ldg(reinterpret_cast<const uint2*>(codes));
            r.w[0] = q.x;
            r.w[1] = q.y;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < cnt)
                    r.w[j / 4] |= (uint32_t)__ldg(codes + j) << (8 * (j & 3));
        }
    }
    return r;
}

__device__ __forceinline__ void decode8(const RawCodes& r, int cnt, float (&x)[8])
{
    const float step = step_of(r.e);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        x[j] = code_value(__byte_perm(r.w[j / 4], 0u, 0x4440 + (j & 3)), step);
    if (cnt < 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j >= cnt)
                x[j] = 0.0f;
    }
}

// What a lane reads of one tile, loaded a tile ahead of its use.
template <typename T, bool CODES>
struct Inputs {
    std::conditional_t<CODES, RawCodes, Raw<T>> v, g;
};

// The row that S lanes of a warp work on, and its tiles of S * 8 positions.
struct Row {
    long long row, at;      // row index; its first element
    long long ntile, ngrp;  // entries of the states array and exponent bytes a row
    int n;                  // positions of the sequence
    int L;                  // positions of the row (0: no such row)
};

__device__ __forceinline__ Row make_row(const ScanArgs& P, long long row)
{
    Row R;
    R.row = row;
    R.at = row * P.L;
    R.ntile = (P.L + kScanTile - 1ll) / kScanTile;
    R.ngrp = (P.L + WBMM_SEQ_GROUP - 1ll) / WBMM_SEQ_GROUP;
    const bool real = row < P.rows;
    R.L = real ? P.L : 0;
    R.n = real ? row_len(P.lengths, row, P.C, P.L) : 0;
    return R;
}

template <typename T, bool VEC, bool CODES>
__device__ __forceinline__ Inputs<T, CODES> load_inputs(const ScanArgs& P, const Row& R, long long t0)
{
    Inputs<T, CODES> in;
    const int cnt = clamp8(R.n - t0);
    if constexpr (CODES) {
        const long long gi = R.row * R.ngrp + t0 / WBMM_SEQ_GROUP;
        in.v = load_codes<VEC>(P.v_codes + R.at + t0, P.v_exps + gi, cnt);
        in.g = load_codes<VEC>(P.g_codes + R.at + t0, P.g_exps + gi, cnt);
    } else {
        in.v = load_raw<VEC>(static_cast<const T*>(P.v) + R.at + t0, cnt);
        in.g = load_raw<VEC>(static_cast<const T*>(P.g) + R.at + t0, cnt);
    }
    return in;
}

template <typename T>
__device__ __forceinline__ void values8(const Raw<T>& r, int cnt, float (&x)[8]) { unpack8(r, cnt, x); }
template <typename T>
__device__ __forceinline__ void values8(const RawCodes& r, int cnt, float (&x)[8]) { decode8(r, cnt, x); }

// The forward steps of a tile: gates, inputs (1 - f) v, and the composed map.
template <typename T, bool CODES>
struct Steps {
    float v[8], f[8], i[8];
    float A, H;
    __device__ __forceinline__ void make(const Inputs<T, CODES>& in, int cnt)
    {
        float g[8];
        values8<T>(in.v, cnt, v);
        values8<T>(in.g, cnt, g);
        gates8<T>(g, cnt, f, i);
        A = 1.0f;
        H = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            H = fmaf(f[j], H, i[j] * v[j]);
            A *= f[j];
        }
    }
};

// Forward, S lanes a row: 32 lanes walk a row's tiles one after the other,
// fewer lanes take rows of at most 8 * S positions in one tile.
template <typename T, int S, bool VEC, bool KEEP>
__global__ void __launch_bounds__(128) scan_fwd_kernel(const ScanArgs P)
{
    grid_dep_wait();
    grid_dep_launch();
    const int sub = threadIdx.x & (S - 1);
    const Row R = make_row(P, (long long)blockIdx.x * (128 / S) + threadIdx.x / S);
    float h = P.h0 && R.L ? P.h0[R.row] : 0.0f;
    const long long tiles = S == 32 ? R.ntile : 1;
    Inputs<T, false> nxt = load_inputs<T, VEC, false>(P, R, sub * 8);
    for (long long t = 0; t < tiles; ++t) {
        const long long t0 = t * kScanTile + sub * 8;
        const int cnt = clamp8(R.n - t0), all = clamp8(R.L - t0);
        const Inputs<T, false> in = nxt;
        if (S == 32 && t + 1 < tiles)
            nxt = load_inputs<T, VEC, false>(P, R, t0 + kScanTile);
        Steps<T, false> st;
        st.make(in, cnt);
        float A = st.A, H = st.H, Aex, Hex;
        lane_scan<S, false>(A, H, Aex, Hex, sub);
        if (P.states && sub == 0 && t * kScanTile < R.n)
            P.states[R.row * R.ntile + t] = h;
        float s = fmaf(Aex, h, Hex), out[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s = fmaf(st.f[j], s, st.i[j] * st.v[j]);
            out[j] = j < cnt ? s : 0.0f;
        }
        store8<VEC>(static_cast<T*>(P.y) + R.at + t0, all, out);
        if constexpr (KEEP) {
            const long long gi = R.row * R.ngrp + t0 / WBMM_SEQ_GROUP;
            float xg[8];
            values8<T>(in.g, cnt, xg);
            encode8<S, VEC>(st.v, all, sub, P.v_codes + R.at + t0, P.v_exps + gi);
            encode8<S, VEC>(xg, all, sub, P.g_codes + R.at + t0, P.g_exps + gi);
        }
        h = __shfl_sync(kFull, s, S - 1, S);
    }
    if (P.hT && sub == 0 && R.L)
        P.hT[R.row] = h;
}

// Backward, S lanes a row, tiles from the last to the first.
template <typename T, int S, bool VEC, bool CODES>
__global__ void __launch_bounds__(128) scan_bwd_kernel(const ScanArgs P)
{
    grid_dep_wait();
    grid_dep_launch();
    const int sub = threadIdx.x & (S - 1);
    const Row R = make_row(P, (long long)blockIdx.x * (128 / S) + threadIdx.x / S);
    const T* dy = static_cast<const T*>(P.dy) + R.at;
    float c = P.h0 && R.L ? P.h0[R.row] : 0.0f;
    const long long tiles = S == 32 ? R.ntile : 1;
    auto state_at = [&](long long t) {
        return t * kScanTile < R.n ? __ldg(P.states + R.row * R.ntile + t) : 0.0f;
    };
    long long t0 = (tiles - 1) * kScanTile + sub * 8;
    Inputs<T, CODES> nxt = load_inputs<T, VEC, CODES>(P, R, t0);
    Raw<T> nxt_dy = load_raw<VEC>(dy + t0, clamp8(R.n - t0));
    float nxt_h = state_at(tiles - 1);
    for (long long t = tiles - 1; t >= 0; --t, t0 -= kScanTile) {
        const int cnt = clamp8(R.n - t0), all = clamp8(R.L - t0);
        const Inputs<T, CODES> in = nxt;
        const Raw<T> rdy = nxt_dy;
        const float h = nxt_h;
        if (S == 32 && t > 0) {
            nxt = load_inputs<T, VEC, CODES>(P, R, t0 - kScanTile);
            nxt_dy = load_raw<VEC>(dy + t0 - kScanTile, clamp8(R.n - t0 + kScanTile));
            nxt_h = state_at(t - 1);
        }
        Steps<T, CODES> st;
        st.make(in, cnt);
        float d[8];
        unpack8(rdy, cnt, d);
        float A = st.A, H = st.H, Ar = st.A, D = 0.0f, Aex, Hex, Dex;
#pragma unroll
        for (int j = 7; j >= 0; --j)
            D = st.f[j] * (d[j] + D);
        lane_scan<S, false>(A, H, Aex, Hex, sub);
        float s = fmaf(Aex, h, Hex), before[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            before[j] = s;
            s = fmaf(st.f[j], s, st.i[j] * st.v[j]);
        }
        lane_scan<S, true>(Ar, D, Aex, Dex, sub);
        float cc = fmaf(Aex, c, Dex), ov[8], og[8];
#pragma unroll
        for (int j = 7; j >= 0; --j) {
            const float dh = d[j] + cc;
            ov[j] = dh * st.i[j];
            cc = st.f[j] * dh;
            og[j] = ov[j] * st.f[j] * (before[j] - st.v[j]);
        }
        if (cnt < 8) {
            // i is 0 past the sequence's end, but NaN of a state times 0 is not
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j >= cnt)
                    ov[j] = og[j] = 0.0f;
        }
        store8<VEC>(static_cast<T*>(P.dv) + R.at + t0, all, ov);
        store8<VEC>(static_cast<T*>(P.dg) + R.at + t0, all, og);
        c = __shfl_sync(kFull, cc, 0, S);
    }
    if (P.hT && sub == 0 && R.L)
        P.hT[R.row] = c;
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

namespace {

template <typename T, int S, bool VEC, bool AUX>
cudaError_t row_launch(const ScanArgs& A, bool backward, const Launch& L)
{
    const dim3 grid((unsigned)((A.rows + 128 / S - 1) / (128 / S))), block(128);
    return done(backward ? launch_pdl(scan_bwd_kernel<T, S, VEC, AUX>, grid, block, 0, L.stream, A)
                         : launch_pdl(scan_fwd_kernel<T, S, VEC, AUX>, grid, block, 0, L.stream, A));
}

// Lanes a row: as few as hold it in one tile of 8 positions a lane (1, 4 or
// 16), so that short rows leave no lanes idle, or a warp that walks it.
template <typename T, bool VEC, bool AUX>
cudaError_t lanes_launch(const ScanArgs& A, bool backward, const Launch& L)
{
    if (A.L <= 8)
        return row_launch<T, 1, VEC, AUX>(A, backward, L);
    if (A.L <= 32)
        return row_launch<T, 4, VEC, AUX>(A, backward, L);
    if (A.L <= 128)
        return row_launch<T, 16, VEC, AUX>(A, backward, L);
    return row_launch<T, 32, VEC, AUX>(A, backward, L);
}

// Whole 16-byte vectors everywhere: rows of a multiple of 8 elements in
// buffers that start at 16-byte boundaries (bf16 ones always do).
bool vector_rows(const ScanArgs& A)
{
    uintptr_t all = 0;
    for (const void* p : {A.v, A.g, (const void*)A.y, A.dy, (const void*)A.dv, (const void*)A.dg})
        all |= reinterpret_cast<uintptr_t>(p);
    return A.L % 8 == 0 && all % 16 == 0;
}

cudaError_t scan_launch(const ScanArgs& A, bool is_bf16, bool backward, const Launch& L)
{
    const bool vec = vector_rows(A), aux = A.v_codes != nullptr;
    if (is_bf16) {
        if (vec)
            return aux ? lanes_launch<__nv_bfloat16, true, true>(A, backward, L)
                       : lanes_launch<__nv_bfloat16, true, false>(A, backward, L);
        return aux ? lanes_launch<__nv_bfloat16, false, true>(A, backward, L)
                   : lanes_launch<__nv_bfloat16, false, false>(A, backward, L);
    }
    if (vec)
        return aux ? lanes_launch<float, true, true>(A, backward, L)
                   : lanes_launch<float, true, false>(A, backward, L);
    return aux ? lanes_launch<float, false, true>(A, backward, L)
               : lanes_launch<float, false, false>(A, backward, L);
}

}  // namespace

cudaError_t scan_forward_launch(const ScanArgs& A, bool is_bf16, const Launch& L)
{
    return scan_launch(A, is_bf16, false, L);
}

cudaError_t scan_backward_launch(const ScanArgs& A, bool is_bf16, const Launch& L)
{
    return scan_launch(A, is_bf16, true, L);
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
