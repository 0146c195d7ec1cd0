// Gated linear recurrence along the rows of a [B, C, L] tensor:
//   f = 1 / (1 + exp(-g)),  h_t = f_t h_{t-1} + (1 - f_t) v_t,  y_t = h_t
// and its backward pass.
//
// A step is the affine map h -> f h + u, u = (1 - f) v, and maps compose:
// (A1, H1) then (A2, H2) is (A1 A2, A2 H1 + H2).  A warp takes a tile of 256
// successive positions of one row, 8 a lane: each lane composes its 8 steps,
// the lanes' maps are joined by an inclusive scan in 5 exchanges, and each
// lane replays its 8 steps from its exact starting state.  The order of every
// product and sum is fixed by the position within the row and the call's
// sizes, so results are bit-identical from run to run.
//
// The backward pass needs h_{t-1}: it replays a tile from the state before it,
// which the forward call keeps (one fp32 value per 256 positions), beside the
// reversed recurrence of c_t = f_t (dy_t + c_{t+1}).
//
// 1 - f is e f with e = exp(-g), not a difference, so that it keeps its
// relative accuracy where f is close to 1; -g is held at about 79.6 at most, so
// that e stays finite: e f is 1 there, and 3e-35 of the state before remains.
//
// The bytes of a call (6 an element forward, 10 backward, in bf16) take the
// memory 0.9 and 1.6 ps an element; the kernels issue 25 and 40 instructions an
// element (ncu; 44 and 45 with 8-bit forms) and reach 87% and 90% of the measured
// copy rate (27.5 and 44.0 us on 8192 rows of 3136; 75% and 72% with 8-bit forms,
// 42.8 and 44.5 us).  Two thirds of the issue slots are taken, with a third of the
// warps resident: both the instructions and the latency that so few warps hide
// are in the way.  So the code around the arithmetic is kept short: paired fp32
// instructions (f32x2), one test a tile for a partial tile, states and exponent
// bytes fetched for 32 tiles at once.
#include <cuda_bf16.h>

#include <type_traits>

#include "ckpt_common.cuh"
#include "f32x2.cuh"
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

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float ex2_fast(float a)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
    return r;
}

__device__ __forceinline__ float rcp_fast(float a)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
    return r;
}

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLog2eLow = (float)(1.44269504088896340736 - (double)kLog2e);
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kGateMin = -79.5f;      // exact in bf16

// f = 1 / (1 + e), i = 1 - f = e f with e = exp(-g) = 2^(-g log2 e), for two
// gates.  ex2 is within 2^-22 and rcp within an ulp.  The rounding of the
// product t and of the constant leave an error of 1.5 |g| 2^-24 in e, far
// below bf16's 2^-8; fp32 maps take it back with the product's exact remainder
// and the constant's next bits, 2^(t + r) = 2^t (1 + r ln 2), |r| < 2^-15.
// bf16 gates have been held at kGateMin (in pairs, before they were widened),
// fp32 ones are held at t = 115; neither these nor an infinite t has a
// remainder.
template <typename T>
__device__ __forceinline__ void gate2(F2 g, F2& f, F2& i)
{
    F2 t = mul2(g, {-kLog2e, -kLog2e}), e;
    if constexpr (std::is_same<T, float>::value) {
        F2 r = fma2(g, {-kLog2e, -kLog2e}, {-t.x, -t.y});
        r = mul2(fma2(g, {-kLog2eLow, -kLog2eLow}, r), {kLn2, kLn2});
        t = {min_nan(t.x, 115.0f), min_nan(t.y, 115.0f)};
        e = {ex2_fast(t.x), ex2_fast(t.y)};
        const F2 c = fma2(e, r, e);
        e.x = fabsf(t.x) < 115.0f ? c.x : e.x;
        e.y = fabsf(t.y) < 115.0f ? c.y : e.y;
    } else {
        e = {ex2_fast(t.x), ex2_fast(t.y)};
    }
    const F2 d = add2(e, {1.0f, 1.0f});
    f = {rcp_fast(d.x), rcp_fast(d.y)};
    i = mul2(e, f);
}

// Positions of row b*C + c that the sequence has.
__device__ __forceinline__ int row_len(const int* lengths, long long row, int C, int L)
{
    if (!lengths)
        return L;
    const int n = lengths[row / C];
    return n < 0 ? 0 : n > L ? L : n;
}

// ------------------------------------------------------- eight of a lane's values
// A lane's eight elements as they sit in memory.
template <typename T>
struct Raw {
    static constexpr int N = 2 * (int)sizeof(T);    // 32-bit words
    uint32_t w[N];
};

template <typename T>
__device__ __forceinline__ void unpack8(const Raw<T>& r, F2 (&x)[4])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4)
            x[j] = {__uint_as_float(r.w[2 * j]), __uint_as_float(r.w[2 * j + 1])};
        else
            x[j] = {__uint_as_float(r.w[j] << 16), __uint_as_float(r.w[j] & 0xffff0000u)};
    }
}

// The gates' arguments: as unpack8, bf16 ones held at kGateMin (NaN stays).
template <typename T>
__device__ __forceinline__ void unpack_gates8(const Raw<T>& r, F2 (&x)[4])
{
    if constexpr (sizeof(T) == 4) {
        unpack8(r, x);
    } else {
        Raw<T> h;
        constexpr uint32_t lim = 0xc29fc29fu;   // kGateMin twice
#pragma unroll
        for (int j = 0; j < 4; ++j)
            asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(h.w[j]) : "r"(r.w[j]), "r"(lim));
        unpack8(h, x);
    }
}

template <typename T>
__device__ __forceinline__ Raw<T> pack8(const F2 (&x)[4])
{
    Raw<T> r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
            r.w[2 * j] = __float_as_uint(x[j].x);
            r.w[2 * j + 1] = __float_as_uint(x[j].y);
        } else {
            const __nv_bfloat162 q = __floats2bfloat162_rn(x[j].x, x[j].y);
            r.w[j] = reinterpret_cast<const uint32_t&>(q);
        }
    }
    return r;
}

// Replaces the values from position cnt on.
__device__ __forceinline__ void cut8(F2 (&x)[4], int cnt, float with)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[j].x = 2 * j < cnt ? x[j].x : with;
        x[j].y = 2 * j + 1 < cnt ? x[j].y : with;
    }
}

// Eight codes and their group's exponent byte.
struct RawCodes {
    uint2 w;
    uint32_t e;
};

__device__ __forceinline__ void decode8(const RawCodes& r, F2 (&x)[4])
{
    const float step = step_of(r.e);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t w = j < 2 ? r.w.x : r.w.y;
        // 2^23 + code, less 2^23 + 128, times the step: all exact
        const F2 m = {__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 + (2 * j & 3))),
                      __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 + (2 * j + 1 & 3)))};
        x[j] = mul2(add2(m, {-8388736.0f, -8388736.0f}), {step, step});
    }
}

// The codes of a lane's 8 values in a group with exponent byte e.
__device__ __forceinline__ uint2 codes8(const F2 (&x)[4], uint32_t e)
{
    const float inv = inv_step_of(e);
    uint32_t q[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        // as quant_code: the product is exact, so one rounding
        const F2 r = fma2(x[j], {inv, inv}, {12583040.0f, 12583040.0f});
        q[2 * j] = __float_as_uint(r.x);
        q[2 * j + 1] = __float_as_uint(r.y);
    }
    return make_uint2(
        __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410),
        __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410));
}

// 8-bit forms of v and g over 64 successive positions: 8 lanes of 8 (all the
// row's lanes where it has fewer); positions from cnt on count as zero.
// Exponent bytes in ev and eg.  bf16 magnitudes are compared in pairs,
// and the groups' of v and g in one word.
template <int S, typename T>
__device__ __forceinline__ void encode8(const Raw<T>& rv, const Raw<T>& rg, int cnt, uint2& cv, uint2& cg,
                                        uint32_t& ev, uint32_t& eg)
{
    F2 v[4], g[4];
    unpack8(rv, v);
    unpack8(rg, g);
    if (cnt < 8) {
        cut8(v, cnt, 0.0f);
        cut8(g, cnt, 0.0f);
    }
    constexpr int LANES = S < 8 ? S : 8;
    if constexpr (sizeof(T) == 2) {
        uint32_t mv = 0, mg = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t wv = rv.w[j], wg = rg.w[j];
            if (cnt < 8) {
                const uint32_t keep = (2 * j < cnt ? 0xffffu : 0u) | (2 * j + 1 < cnt ? 0xffff0000u : 0u);
                wv &= keep;
                wg &= keep;
            }
            mv = max_abs2(mv, wv & 0x7fff7fffu);
            mg = max_abs2(mg, wg & 0x7fff7fffu);
        }
        // v's largest in the lower half, g's in the upper
        uint32_t m = max_abs2(__byte_perm(mv, mg, 0x5410), __byte_perm(mv, mg, 0x7632));
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1)
            m = max_abs2(m, __shfl_xor_sync(kFull, m, o));
        ev = group_exp(m << 16);
        eg = group_exp(m & 0xffff0000u);
    } else {
        uint32_t mv = 0, mg = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            mv = max(mv, max(__float_as_uint(v[j].x) & kAbsMask, __float_as_uint(v[j].y) & kAbsMask));
            mg = max(mg, max(__float_as_uint(g[j].x) & kAbsMask, __float_as_uint(g[j].y) & kAbsMask));
        }
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) {
            mv = max(mv, __shfl_xor_sync(kFull, mv, o));
            mg = max(mg, __shfl_xor_sync(kFull, mg, o));
        }
        ev = group_exp(mv);
        eg = group_exp(mg);
    }
    if (max(ev, eg) >= kExpTop) {
        // rare: a bad group, or one at the top of the range
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (ev >= kExpTop)
                v[j] = {group_fix(v[j].x, ev), group_fix(v[j].y, ev)};
            if (eg >= kExpTop)
                g[j] = {group_fix(g[j].x, eg), group_fix(g[j].y, eg)};
        }
    }
    cv = codes8(v, ev);
    cg = codes8(g, eg);
}

// What a lane reads of one tile besides dy.
template <typename T, bool CODES>
struct Inputs {
    std::conditional_t<CODES, RawCodes, Raw<T>> v, g;
};

template <typename T>
__device__ __forceinline__ void values8(const Raw<T>& r, F2 (&x)[4]) { unpack8(r, x); }
template <typename T>
__device__ __forceinline__ void values8(const RawCodes& r, F2 (&x)[4]) { decode8(r, x); }
template <typename T>
__device__ __forceinline__ void gate_values8(const Raw<T>& r, F2 (&x)[4]) { unpack_gates8(r, x); }
template <typename T>
__device__ __forceinline__ void gate_values8(const RawCodes& r, F2 (&x)[4])
{
    decode8(r, x);
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x[j] = {max_nan(x[j].x, kGateMin), max_nan(x[j].y, kGateMin)};
    }
}

// ------------------------------------------------------------- maps of a tile
// Inclusive scan of the maps of S lanes (forward: lane order; REV: from the
// last lane down).
template <int S, bool REV>
__device__ __forceinline__ void lane_scan(float& A, float& H, int sub)
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
}

// The state before a lane's positions (REV: behind them) from the inclusive
// maps and the state s before all of the lanes; `end` becomes the one after
// the lane.
template <int S, bool REV>
__device__ __forceinline__ float lane_start(float A, float H, float s, int sub, float& end)
{
    end = fmaf(A, s, H);
    if constexpr (S == 1)
        return s;
    const float prev = REV ? __shfl_down_sync(kFull, end, 1, S) : __shfl_up_sync(kFull, end, 1, S);
    return sub == (REV ? S - 1 : 0) ? s : prev;
}

// The forward steps of a lane's positions: f, i = 1 - f, u = i v, and their
// composed map.  cnt < 8: the steps from cnt on are the identity.
template <typename T, bool CODES>
struct Steps {
    F2 v[4], f[4], i[4], u[4];
    float A, H;
    __device__ __forceinline__ void make(const Inputs<T, CODES>& in, int cnt)
    {
        F2 g[4];
        values8<T>(in.v, v);
        gate_values8<T>(in.g, g);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            gate2<T>(g[j], f[j], i[j]);
            u[j] = mul2(i[j], v[j]);
        }
        if (cnt < 8) {
            cut8(f, cnt, 1.0f);
            cut8(i, cnt, 0.0f);
            cut8(u, cnt, 0.0f);
        }
        A = f[0].x * f[0].y;
        H = fmaf(f[0].y, u[0].x, u[0].y);
#pragma unroll
        for (int j = 1; j < 4; ++j) {
            H = fmaf(f[j].y, fmaf(f[j].x, H, u[j].x), u[j].y);
            A = A * f[j].x * f[j].y;
        }
    }
    __device__ __forceinline__ void replay(float s, F2 (&y)[4]) const
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y[j].x = fmaf(f[j].x, s, u[j].x);
            s = y[j].y = fmaf(f[j].y, y[j].x, u[j].y);
        }
    }
};

// The reversed steps c = f (dy + c') of a lane's positions, in two parts: the
// gates and the composed map, and, once the state before and the c behind the
// lane's tile are known, the gradients, for which v is read.
template <typename T, bool CODES>
struct BackSteps {
    F2 f[4], i[4];
    float A, D;
    __device__ __forceinline__ void make(const std::conditional_t<CODES, RawCodes, Raw<T>>& g,
                                         const Raw<T>& dy, int cnt)
    {
        F2 x[4], d[4];
        gate_values8<T>(g, x);
        unpack8(dy, d);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            gate2<T>(x[j], f[j], i[j]);
        if (cnt < 8) {
            cut8(f, cnt, 1.0f);
            cut8(i, cnt, 0.0f);
            cut8(d, cnt, 0.0f);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            d[j] = mul2(f[j], d[j]);
        D = fmaf(f[3].x, d[3].y, d[3].x);
        A = f[0].x * f[0].y;
#pragma unroll
        for (int j = 2; j >= 0; --j)
            D = fmaf(f[j].x, fmaf(f[j].y, D, d[j].y), d[j].x);
#pragma unroll
        for (int j = 1; j < 4; ++j)
            A = A * f[j].x * f[j].y;
    }
    // dv and dg from the state `h` before all S lanes and the c behind this one
    template <int S>
    __device__ __forceinline__ void grads(const std::conditional_t<CODES, RawCodes, Raw<T>>& rv,
                                          const Raw<T>& dy, float h, float c, int cnt, int sub,
                                          F2 (&ov)[4], F2 (&og)[4]) const
    {
        F2 v[4], d[4], u[4];
        values8<T>(rv, v);
        unpack8(dy, d);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            u[j] = mul2(i[j], v[j]);
        if (cnt < 8) {
            cut8(u, cnt, 0.0f);
            cut8(d, cnt, 0.0f);
        }
        float a = A, H = fmaf(f[0].y, u[0].x, u[0].y), end;
#pragma unroll
        for (int j = 1; j < 4; ++j)
            H = fmaf(f[j].y, fmaf(f[j].x, H, u[j].x), u[j].y);
        lane_scan<S, false>(a, H, sub);
        float s = lane_start<S, false>(a, H, h, sub, end);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float s1 = fmaf(f[j].x, s, u[j].x);
            const F2 gap = add2({s, s1}, {-v[j].x, -v[j].y});
            og[j] = mul2(gap, f[j]);
            s = fmaf(f[j].y, s1, u[j].y);
        }
#pragma unroll
        for (int j = 3; j >= 0; --j) {
            const F2 fd = mul2(f[j], d[j]);
            const float c1 = fmaf(f[j].y, c, fd.y);
            const F2 dh = add2(d[j], {c1, c});
            ov[j] = mul2(dh, i[j]);
            og[j] = mul2(og[j], ov[j]);
            c = fmaf(f[j].x, c1, fd.x);
        }
        if (cnt < 8) {
            // i is 0 past the sequence's end, but NaN of a state times 0 is not
            cut8(ov, cnt, 0.0f);
            cut8(og, cnt, 0.0f);
        }
    }
};

// ------------------------------------------------------------- data movement
// VEC rows (bf16, a multiple of 8 elements): a lane's elements are one 16-byte
// vector.  Other rows are moved as the 16-byte blocks of memory that hold the
// tile's elements, through an image of them in shared memory, from which lanes
// take their elements at whatever offset they have; blocks that reach over the
// tile's ends are written element by element.  (fp32 rows go that way even
// where they are aligned: a lane's 32 bytes would be two 16-byte accesses 32
// bytes apart, each half of every sector; B32 C256 L1568 forward 40 us against
// 31 us through the image.)

__device__ __forceinline__ uint4 lds4(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }

// Copies the blocks that hold [at, at + bytes) into `dst`, cut at the
// tensor's ends: base, its first byte, and end, the one behind its last.
__device__ __forceinline__ void image_copy(uint8_t* dst, const uint8_t* at, int bytes,
                                           const uint8_t* base, const uint8_t* end, int lane)
{
    if (bytes <= 0)
        return;
    const uint8_t* a0 = at - (reinterpret_cast<uintptr_t>(at) & 15);
    const int blocks = (int)((at - a0) + bytes + 15) >> 4;
    for (int k = lane; k < blocks; k += 32) {
        const uint8_t* src = a0 + 16 * k;
        const uint32_t to = smem_u32(dst + 16 * k);
        if (src >= base) {
            const long long left = end - src;
            cp_async_16z(to, src, left < 16 ? (uint32_t)left : 16u);
        } else {
            // fp32 tensors may start between 16-byte boundaries
#pragma unroll
            for (int q = 0; q < 16; q += 4)
                if (src + q >= base && src + q < end)
                    cp_async_4(to + q, src + q);
        }
    }
}

// N words from byte sh on of a block of an image, sh the same for all lanes
// and even, 0 <= sh < 16.  Eight words (fp32) are taken from where they are in
// one of four uniform branches; four words are moved down in two steps, which
// costs less than the branches.
template <int N>
__device__ __forceinline__ void shifted(const uint8_t* block, int sh, uint32_t (&r)[N])
{
    uint32_t u[N + 4];
#pragma unroll
    for (int k = 0; k < N + 4; k += 4) {
        if (N == 4 || k < N || sh != 0) {
            const uint4 q = lds4(block + 4 * k);
            u[k] = q.x; u[k + 1] = q.y; u[k + 2] = q.z; u[k + 3] = q.w;
        } else {
            u[k] = u[k + 1] = u[k + 2] = u[k + 3] = 0u;
        }
    }
    if constexpr (N == 4) {
        if (sh & 8) {
#pragma unroll
            for (int k = 0; k < N + 2; ++k)
                u[k] = u[k + 2];
        }
        if (sh & 4) {
#pragma unroll
            for (int k = 0; k < N + 1; ++k)
                u[k] = u[k + 1];
        }
#pragma unroll
        for (int k = 0; k < N; ++k)
            r[k] = sh & 2 ? __funnelshift_r(u[k], u[k + 1], 16) : u[k];
    } else {
        auto take = [&](auto from) {
#pragma unroll
            for (int k = 0; k < N; ++k)
                r[k] = u[decltype(from)::value + k];
        };
        if (sh < 8) {
            if (sh < 4)
                take(std::integral_constant<int, 0>());
            else
                take(std::integral_constant<int, 1>());
        } else {
            if (sh < 12)
                take(std::integral_constant<int, 2>());
            else
                take(std::integral_constant<int, 3>());
        }
    }
}

// Eight elements at byte `off` of an image.
template <typename T>
__device__ __forceinline__ Raw<T> image_read(const uint8_t* img, int off)
{
    Raw<T> r;
    const uint32_t* p = reinterpret_cast<const uint32_t*>(img + (off & ~3));
    uint32_t u[Raw<T>::N + 1];
#pragma unroll
    for (int k = 0; k < Raw<T>::N + 1; ++k)
        u[k] = p[k];
#pragma unroll
    for (int k = 0; k < Raw<T>::N; ++k)
        r.w[k] = sizeof(T) == 2 && (off & 2) ? __funnelshift_r(u[k], u[k + 1], 16) : u[k];
    return r;
}

// The 8 codes at byte `off` of an image.
__device__ __forceinline__ uint2 image_codes(const uint8_t* img, int off)
{
    const uint32_t* p = reinterpret_cast<const uint32_t*>(img + (off & ~3));
    const int sh = 8 * (off & 3);
    const uint32_t a = p[0], b = p[1], c = p[2];
    return make_uint2(__funnelshift_r(a, b, sh), __funnelshift_r(b, c, sh));
}

// Writes the lanes' elements through the warp's image buffer: `count` from p
// on, this lane's (cnt of them) from element `mine`.
template <typename T, bool ONE_ROW>
__device__ __forceinline__ void image_store(T* p, int count, int mine, int cnt, const Raw<T>& r,
                                            uint8_t* stage, int lane)
{
    constexpr int E = 16 / (int)sizeof(T);      // elements a block
    const int s = (int)(reinterpret_cast<uintptr_t>(p) & 15) / (int)sizeof(T);
    T* img = reinterpret_cast<T*>(stage);
    __syncwarp();
    if constexpr (ONE_ROW) {
        // as they are, from the second block on: blocks are shifted when read
#pragma unroll
        for (int k = 0; k < Raw<T>::N; k += 4)
            *reinterpret_cast<uint4*>(img + E + mine + k / 4 * E) =
                make_uint4(r.w[k], r.w[k + 1], r.w[k + 2], r.w[k + 3]);
        __syncwarp();
        // whole blocks from element `head` on; single elements around them
        const int head = s != 0 ? E - s : 0, full = count > head ? (count - head) / E : 0;
#pragma unroll
        for (int m = 0; m < kScanTile / E / 32; ++m) {
            const int k = lane + 32 * m;
            if (k < full) {
                uint32_t q[4];
                shifted<4>(stage + 16 + 16 * k, head * (int)sizeof(T), q);
                *reinterpret_cast<uint4*>(p + head + k * E) = make_uint4(q[0], q[1], q[2], q[3]);
            }
        }
        const int e = lane < 16 ? lane : head + full * E + lane - 16;
        if (e < (lane < 16 && head < count ? head : count))
            p[e] = img[E + e];
    } else {
        // in the place that memory has for them
        const T* x = reinterpret_cast<const T*>(r.w);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < cnt)
                img[s + mine + j] = x[j];
        __syncwarp();
        const int blocks = (s + count + E - 1) / E;
        for (int k = lane; k < blocks; k += 32) {
            const int e0 = k * E - s;
            if (e0 >= 0 && e0 + E <= count) {
                *reinterpret_cast<uint4*>(p + e0) = lds4(stage + 16 * k);
            } else {
                for (int j = 0; j < E; ++j)
                    if (e0 + j >= 0 && e0 + j < count)
                        p[e0 + j] = img[s + e0 + j];
            }
        }
    }
}

// The same for codes: 16-byte blocks of a whole tile of one row, else words;
// single bytes at the ends.
template <bool ONE_ROW>
__device__ __forceinline__ void image_store_codes(uint8_t* p, int count, int mine, int cnt, uint2 codes,
                                                  uint8_t* stage, int lane)
{
    __syncwarp();
    if constexpr (ONE_ROW) {
        *reinterpret_cast<uint2*>(stage + 16 + mine) = codes;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < cnt)
                stage[16 + mine + j] = (uint8_t)((j < 4 ? codes.x : codes.y) >> (8 * (j & 3)));
    }
    __syncwarp();
    if constexpr (ONE_ROW) {
        const int s = (int)(reinterpret_cast<uintptr_t>(p) & 15);
        const int head = s != 0 ? 16 - s : 0, full = count > head ? (count - head) / 16 : 0;
        if (lane < full) {
            const int off = 16 + head + 16 * lane, sh = 8 * (off & 3);
            const uint32_t* w = reinterpret_cast<const uint32_t*>(stage + (off & ~3));
            uint32_t u[5];
#pragma unroll
            for (int k = 0; k < 5; ++k)
                u[k] = w[k];
            *reinterpret_cast<uint4*>(p + head + 16 * lane) =
                make_uint4(__funnelshift_r(u[0], u[1], sh), __funnelshift_r(u[1], u[2], sh),
                           __funnelshift_r(u[2], u[3], sh), __funnelshift_r(u[3], u[4], sh));
        }
        const int e = lane < 16 ? lane : head + full * 16 + lane - 16;
        if (e < (lane < 16 && head < count ? head : count))
            p[e] = stage[16 + e];
        return;
    }
    const int s = (int)(reinterpret_cast<uintptr_t>(p) & 3);
    const int words = (s + count + 3) / 4;
    for (int k = lane; k < words; k += 32) {
        const int e0 = 4 * k - s;
        if (e0 >= 0 && e0 + 4 <= count) {
            const int off = 16 + e0;
            const uint32_t* w = reinterpret_cast<const uint32_t*>(stage + (off & ~3));
            *reinterpret_cast<uint32_t*>(p + e0) = __funnelshift_r(w[0], w[1], 8 * (off & 3));
        } else {
            for (int j = 0; j < 4; ++j)
                if (e0 + j >= 0 && e0 + j < count)
                    p[e0 + j] = stage[16 + e0 + j];
        }
    }
}

// Bytes of an image of 256 elements, with room for the reads past its end.
template <typename T>
constexpr int kImage = 256 * (int)sizeof(T) + 48;

// ---------------------------------------------------------- rows of many tiles
// A warp, or a team of warps, walks a row's tiles with the inputs of its next
// tiles in flight as asynchronous copies into a ring of stages of its own.
constexpr int kWarps = 4;

// One stage: v and g (maps or codes), dy.
template <typename T, bool VEC, bool CODES, bool BACK, bool TEAM>
struct Stage {
    static constexpr int MAP = VEC ? 256 * (int)sizeof(T) : kImage<T>;
    static constexpr int ARR = !CODES ? MAP : VEC ? 256 : 304;
    static constexpr int DY = 2 * ARR;
    static constexpr int BYTES = DY + (BACK ? MAP : 0);
    // four stages; three of the larger fp32 ones where a warp works alone
    // (more warps fit an SM: B32 C256 L1568 forward 32.0 us, 34.0 with four)
    // and where four would not fit (fp32 backward)
    static constexpr int DEPTH = BYTES > (TEAM ? 3000 : 2048) ? 3 : 4;
    // tiles a round: a team's warp takes two, whose arithmetic overlaps and
    // which share the round's barrier, where the ring holds two rounds (768
    // rows of 50176 forward 43.0 us, 57.5 with one)
    static constexpr int PER = TEAM && DEPTH == 4 ? 2 : 1;
    static constexpr int OUT = VEC ? 0 : kImage<T>;     // image of an output
    static constexpr int WARP = DEPTH * BYTES + OUT;
};

// One input array of a row as the warp walks it.
template <int SZ, bool VEC>
struct Stream {
    const uint8_t* next;    // of the tile to fetch next: this lane's part (VEC), its first element
    __device__ __forceinline__ void start(const void* p, long long first, int lane)
    {
        next = static_cast<const uint8_t*>(p) + first * SZ + (VEC ? lane * 8 * SZ : 0);
    }
    // positions from the tile's start to the end of the sequence
    __device__ __forceinline__ void fetch(uint8_t* dst, int left, bool inner, const void* base,
                                          long long elems, int lane) const
    {
        if constexpr (VEC) {
            if (left > lane * 8) {
                if constexpr (SZ == 1) {
                    cp_async_8(smem_u32(dst + 8 * lane), next);
                } else {
#pragma unroll
                    for (int k = 0; k < SZ / 2; ++k)
                        cp_async_16z(smem_u32(dst + 512 * k + 16 * lane), next + 16 * k, 16u);
                }
            }
        } else if (inner && next - 12 >= base) {
            // a whole tile with a block's worth of the row behind it (and of
            // the tensor before it: fp32 ones may start anywhere): 16, 32 or
            // 64 blocks, and one more for the shift
            const int s = (int)(reinterpret_cast<uintptr_t>(next) & 15);
            const uint8_t* src = next - s + 16 * lane;
            if (lane < 16 * SZ)
                cp_async_16z(smem_u32(dst + 16 * lane), src, 16u);
            if constexpr (SZ == 4)
                cp_async_16z(smem_u32(dst + 512 + 16 * lane), src + 512, 16u);
            if (s != 0 && lane == 0)
                cp_async_16z(smem_u32(dst + 256 * SZ), src + 256 * SZ, 16u);
        } else {
            const uint8_t* b = static_cast<const uint8_t*>(base);
            image_copy(dst, next, (left < kScanTile ? left : kScanTile) * SZ, b, b + elems * SZ, lane);
        }
    }
    __device__ __forceinline__ void advance(int tiles) { next += (long long)tiles * (kScanTile * SZ); }
};

// Where several warps take one row: a team of the 4 warps of a CTA, or of all
// CTAs of a cluster.  In each round warp k of the team has the round's k-th
// tile or pair of tiles, publishes its composed map in the shared memory of
// every CTA of the team, and, after one barrier, applies the maps of the warps
// before its own to the state that all of them carry from round to round.  Rounds
// alternate between two slot arrays, so one barrier a round is enough: a warp
// overwrites a slot only after the next barrier, which its readers have passed
// by then.  A CTA's last remote access comes before the last barrier, so none
// reaches a CTA that has ended.
constexpr int kTeamMax = 8 * kWarps;

struct Team {
    int ctas, size, me;     // CTAs of the cluster, warps of the team, this warp
    float2 (*slot)[kTeamMax];

    __device__ __forceinline__ void init(float2 (*s)[kTeamMax])
    {
        ctas = (int)cluster_nctarank();
        size = ctas * kWarps;
        me = (int)cluster_ctarank() * kWarps + (int)(threadIdx.x >> 5);
        slot = s;
        if (ctas > 1)
            cluster_sync();     // every CTA of the cluster has started
    }
    // A and H are the warp's map of the round, on every lane.
    __device__ __forceinline__ void publish(int buf, float A, float H, int lane)
    {
        if (ctas == 1) {
            if (lane == 0)
                slot[buf][me] = make_float2(A, H);
            __syncthreads();
        } else {
            if (lane < ctas)
                st_cluster_f2(smem_u32(&slot[buf][me]), (uint32_t)lane, A, H);
            __syncwarp();
            cluster_sync();
        }
    }
    // The state before this warp's tiles, from the one before the round's
    // first (REV: behind its last); `s` becomes the one after the round.
    template <bool REV>
    __device__ __forceinline__ float join(int buf, float& s) const
    {
        float mine = s;
        for (int k = 0; k < size; k += 4) {
            float2 m[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                m[q] = slot[buf][REV ? size - 1 - k - q : k + q];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if ((REV ? size - 1 - k - q : k + q) == me)
                    mine = s;
                s = fmaf(m[q].x, s, m[q].y);
            }
        }
        return mine;
    }
};

// The four exponent bytes of tile t (0 past the row's last).
__device__ __forceinline__ uint32_t tile_exps(const uint8_t* row, int t, int ngrp)
{
    uint32_t w = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b)
        if (t >= 0 && 4ll * t + b < ngrp)
            w |= (uint32_t)__ldg(row + 4ll * t + b) << (8 * b);
    return w;
}

// A row and the warp's walk along it.
struct RowWalk {
    long long row;
    int n;              // positions of the sequence
    int ntile, ngrp;    // of the row
    int step, from;     // a round's tiles: from every step-th on, the first of them the from-th
    int rounds;
};

template <bool TEAM, int PER>
__device__ __forceinline__ RowWalk row_walk(const ScanArgs& P, const Team& M)
{
    RowWalk w;
    w.row = TEAM ? (long long)(blockIdx.x / M.ctas)
                 : (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    w.n = w.row < P.rows ? row_len(P.lengths, w.row, P.C, P.L) : 0;
    w.ntile = (int)((P.L + kScanTile - 1ll) / kScanTile);
    w.ngrp = (int)((P.L + WBMM_SEQ_GROUP - 1ll) / WBMM_SEQ_GROUP);
    w.step = (TEAM ? M.size : 1) * PER;
    w.from = TEAM ? M.me * PER : 0;
    w.rounds = (w.ntile + w.step - 1) / w.step;
    return w;
}

template <typename T, bool VEC>
__device__ __forceinline__ Raw<T> stage_map(const uint8_t* st, int off, int lane)
{
    Raw<T> r;
    if constexpr (VEC) {
#pragma unroll
        for (int k = 0; k < Raw<T>::N; k += 4) {
            const uint4 q = lds4(st + 128 * k + 16 * lane);
            r.w[k] = q.x; r.w[k + 1] = q.y; r.w[k + 2] = q.z; r.w[k + 3] = q.w;
        }
    } else {
        shifted<Raw<T>::N>(st + lane * 8 * (int)sizeof(T), off, r.w);
    }
    return r;
}

// Offset of a row's elements from 16-byte boundaries, the same for all of its
// tiles.
template <int SZ, bool VEC>
__device__ __forceinline__ int shift_of(const void* p, long long first)
{
    return VEC ? 0 : (int)((reinterpret_cast<uintptr_t>(p) + (unsigned long long)first * SZ) & 15);
}

// One element type's output of a tile: `count` positions of the row, cnt of
// them this lane's.
template <typename T, bool VEC>
__device__ __forceinline__ void tile_store(T* p, int count, const F2 (&x)[4], uint8_t* out, int lane)
{
    const Raw<T> r = pack8<T>(x);
    if constexpr (VEC) {
        if (count > lane * 8) {
#pragma unroll
            for (int k = 0; k < Raw<T>::N; k += 4)
                reinterpret_cast<uint4*>(p + lane * 8)[k / 4] =
                    make_uint4(r.w[k], r.w[k + 1], r.w[k + 2], r.w[k + 3]);
        }
    } else if (count > 0) {
        image_store<T, true>(p, count < kScanTile ? count : kScanTile, lane * 8, 8, r, out, lane);
    }
}

__device__ __forceinline__ int lane_count(int left, int lane)
{
    const int c = left - lane * 8;
    return c < 0 ? 0 : c > 8 ? 8 : c;
}

// Blocks an SM that the register allocation has to leave room for: measured on
// 8192 rows of 3136 (forward 27.6 us with 8, 28.4 unconstrained; with
// checkpoints 43.0 with 8; backward 44.0 with 6, 45.1 with 7), 768 rows of
// 50176 (a team's forward 44.4 us with 6, 52.5 with 4) and 128 rows of 65536
// (with checkpoints 23.8 us with 4, 27.3 with 5; backward 23.6 and 26.7).
constexpr int fwd_blocks(bool vec, bool keep, bool team)
{
    return team ? (vec && !keep ? 6 : 4) : vec || !keep ? 8 : 6;
}
constexpr int bwd_blocks(bool vec, bool team) { return team ? 4 : vec ? 6 : 5; }

// Forward: one row a warp, or (TEAM) a CTA or cluster.  KEEP: the 8-bit forms
// of v and g are written too.
template <typename T, bool VEC, bool KEEP, bool TEAM>
__global__ void __launch_bounds__(32 * kWarps, fwd_blocks(VEC, KEEP, TEAM))
    scan_fwd_kernel(const ScanArgs P)
{
    using G = Stage<T, VEC, false, false, TEAM>;
    constexpr int SZ = (int)sizeof(T), PER = G::PER;
    __shared__ __align__(16) uint8_t ring[kWarps][G::WARP];
    __shared__ float2 slots[2][TEAM ? kTeamMax : 1];
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31;
    uint8_t* const mine = ring[threadIdx.x >> 5];
    uint8_t* const out = mine + G::DEPTH * G::BYTES;
    Team M = {};
    if constexpr (TEAM)
        M.init(reinterpret_cast<float2(*)[kTeamMax]>(slots));
    const RowWalk w = row_walk<TEAM, PER>(P, M);
    if (w.row >= P.rows)
        return;         // no teams: they have a row each
    const long long base = w.row * P.L, elems = P.rows * P.L;
    long long at = base + (long long)w.from * kScanTile;    // the round's first element
    const int off_v = shift_of<SZ, VEC>(P.v, at), off_g = shift_of<SZ, VEC>(P.g, at);
    Stream<SZ, VEC> fv, fg;
    fv.start(P.v, at, lane);
    fg.start(P.g, at, lane);
    const int hop = w.step * kScanTile;
    int left = w.n - w.from * kScanTile;        // from the round's start to the sequence's end
    int far = left, stored = P.L - w.from * kScanTile;
    int turn = 0;                               // tile of its round that is fetched next
    uint8_t* into = mine;                       // the stage to fetch into
    const uint8_t* const last = mine + (G::DEPTH - 1) * G::BYTES;
    auto prefetch = [&] {
        if (far > 0) {
            fv.fetch(into, far, far >= kScanTile + 16, P.v, elems, lane);
            fg.fetch(into + G::ARR, far, far >= kScanTile + 16, P.g, elems, lane);
        }
        const int go = PER == 1 || turn == PER - 1 ? w.step - (PER - 1) : 1;
        turn = turn == PER - 1 ? 0 : turn + 1;
        fv.advance(go);
        fg.advance(go);
        far -= go * kScanTile;
        into = into == last ? mine : into + G::BYTES;
        cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < G::DEPTH - PER; ++k)
        prefetch();
    float h = P.h0 ? P.h0[w.row] : 0.0f;
    float kept = 0.0f;      // lane k: the state before the k-th of 32 tiles
    const uint8_t* st = mine;
    for (int k = 0; k < w.rounds; ++k) {
        if constexpr (!VEC)
            __syncwarp();       // every lane has read the stages that are fetched into next
#pragma unroll
        for (int m = 0; m < PER; ++m)
            prefetch();
        cp_async_wait_group<G::DEPTH - PER>();
        if constexpr (!VEC)
            __syncwarp();
        Inputs<T, false> in[PER];
        Steps<T, false> s8[PER];
        float A[PER], H[PER];
        int cnt[PER];
#pragma unroll
        for (int m = 0; m < PER; ++m) {
            cnt[m] = left >= (m + 1) * kScanTile ? 8 : lane_count(left - m * kScanTile, lane);
            in[m].v = stage_map<T, VEC>(st, off_v, lane);
            in[m].g = stage_map<T, VEC>(st + G::ARR, off_g, lane);
            st = st == last ? mine : st + G::BYTES;
            s8[m].make(in[m], cnt[m]);
            A[m] = s8[m].A;
            H[m] = s8[m].H;
        }
#pragma unroll
        for (int m = 0; m < PER; ++m)
            lane_scan<32, false>(A[m], H[m], lane);
        float hin = h;
        if constexpr (TEAM) {
            static_assert(PER == 2, "forward stages are small enough for four");
            const float a0 = __shfl_sync(kFull, A[0], 31), h0 = __shfl_sync(kFull, H[0], 31);
            const float a1 = __shfl_sync(kFull, A[1], 31), h1 = __shfl_sync(kFull, H[1], 31);
            M.publish(k & 1, a0 * a1, fmaf(a1, h0, h1), lane);
            hin = M.join<false>(k & 1, h);
        }
#pragma unroll
        for (int m = 0; m < PER; ++m) {
            const int here = stored - m * kScanTile;
            float end;
            const float s = lane_start<32, false>(A[m], H[m], hin, lane, end);
            const float hnext = !TEAM || m + 1 < PER ? __shfl_sync(kFull, end, 31) : 0.0f;
            F2 y[4];
            s8[m].replay(s, y);
            if (cnt[m] < 8)
                cut8(y, cnt[m], 0.0f);
            tile_store<T, VEC>(static_cast<T*>(P.y) + at + m * kScanTile, here, y, out, lane);
            const int t = k * w.step + w.from + m;
            if constexpr (KEEP) {
                if (here > 0) {
                    const int all = lane_count(here, lane);
                    const long long to = at + m * kScanTile;
                    uint2 cv, cg;
                    uint32_t ev, eg;
                    encode8<32>(in[m].v, in[m].g, cnt[m], cv, cg, ev, eg);
                    if constexpr (VEC) {
                        if (all > 0) {
                            *reinterpret_cast<uint2*>(P.v_codes + to + lane * 8) = cv;
                            *reinterpret_cast<uint2*>(P.g_codes + to + lane * 8) = cg;
                        }
                    } else {
                        const int n = here < kScanTile ? here : kScanTile;
                        image_store_codes<true>(P.v_codes + to, n, lane * 8, 8, cv, out, lane);
                        image_store_codes<true>(P.g_codes + to, n, lane * 8, 8, cg, out, lane);
                    }
                    if (all > 0 && (lane & 7) == 0) {
                        const long long grp = w.row * w.ngrp + (long long)t * 4 + lane / 8;
                        P.v_exps[grp] = (uint8_t)ev;
                        P.g_exps[grp] = (uint8_t)eg;
                    }
                }
            }
            if (P.states) {
                const int q = k * PER + m;
                if (lane == (q & 31))
                    kept = hin;
                if ((q & 31) == 31 || (k == w.rounds - 1 && m == PER - 1)) {
                    const int i = (q & ~31) + lane;
                    const int ti = i / PER * w.step + w.from + i % PER;
                    if (lane <= (q & 31) && (long long)ti * kScanTile < w.n)
                        P.states[w.row * w.ntile + ti] = kept;
                }
            }
            hin = hnext;
        }
        if constexpr (!TEAM)
            h = hin;
        left -= hop;
        stored -= hop;
        at += hop;
    }
    if (P.hT && lane == 0 && (!TEAM || M.me == 0))
        P.hT[w.row] = h;
}

// Backward, tiles from the last to the first.  CODES: v and g from their
// 8-bit forms.
template <typename T, bool VEC, bool CODES, bool TEAM>
__global__ void __launch_bounds__(32 * kWarps, bwd_blocks(VEC, TEAM))
    scan_bwd_kernel(const ScanArgs P)
{
    using G = Stage<T, VEC, CODES, true, TEAM>;
    constexpr int SZ = (int)sizeof(T), IN = CODES ? 1 : SZ, PER = G::PER;
    __shared__ __align__(16) uint8_t ring[kWarps][G::WARP];
    __shared__ float2 slots[2][TEAM ? kTeamMax : 1];
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31;
    uint8_t* const mine = ring[threadIdx.x >> 5];
    uint8_t* const out = mine + G::DEPTH * G::BYTES;
    Team M = {};
    if constexpr (TEAM)
        M.init(reinterpret_cast<float2(*)[kTeamMax]>(slots));
    const RowWalk w = row_walk<TEAM, PER>(P, M);
    if (w.row >= P.rows)
        return;         // no teams: they have a row each
    const long long base = w.row * P.L, elems = P.rows * P.L;
    // the last tile of the round that is taken first
    const int t_last = (w.rounds - 1) * w.step + w.from + PER - 1;
    long long at = base + (long long)t_last * kScanTile;
    const void* const sv = CODES ? P.v_codes : P.v;
    const void* const sg = CODES ? P.g_codes : P.g;
    const int off_v = shift_of<IN, VEC>(sv, at), off_g = shift_of<IN, VEC>(sg, at);
    const int off_d = shift_of<SZ, VEC>(P.dy, at);
    Stream<IN, VEC> fv, fg;
    Stream<SZ, VEC> fd;
    fv.start(sv, at, lane);
    fg.start(sg, at, lane);
    fd.start(P.dy, at, lane);
    const int hop = w.step * kScanTile;
    int left = (int)(w.n - (long long)t_last * kScanTile);
    int far = left, stored = (int)(P.L - (long long)t_last * kScanTile);
    int togo = w.rounds * PER;                      // tiles to fetch
    int turn = 0;                                   // tile of its round that is fetched next
    uint8_t* into = mine;
    const uint8_t* const last = mine + (G::DEPTH - 1) * G::BYTES;
    auto prefetch = [&] {
        if (togo > 0 && far > 0) {
            fv.fetch(into, far, far >= kScanTile + 16, sv, elems, lane);
            fg.fetch(into + G::ARR, far, far >= kScanTile + 16, sg, elems, lane);
            fd.fetch(into + G::DY, far, far >= kScanTile + 16, P.dy, elems, lane);
        }
        const int go = PER == 1 || turn == PER - 1 ? w.step - (PER - 1) : 1;
        turn = turn == PER - 1 ? 0 : turn + 1;
        fv.advance(-go);
        fg.advance(-go);
        fd.advance(-go);
        far += togo > 0 ? go * kScanTile : 0;
        --togo;
        into = into == last ? mine : into + G::BYTES;
        cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < G::DEPTH - PER; ++k)
        prefetch();
    float c = P.h0 ? P.h0[w.row] : 0.0f;
    // lane k: the state before the tile, and the exponent bytes, of the k-th of
    // 32 tiles
    float states = 0.0f;
    uint32_t ve = 0, ge = 0;
    const uint8_t* st = mine;
    for (int k = 0; k < w.rounds; ++k) {
        if ((k * PER & 31) == 0) {
            const int q = k * PER + lane, t = t_last - q / PER * w.step - q % PER;
            states = t >= 0 && (long long)t * kScanTile < w.n ? __ldg(P.states + w.row * w.ntile + t) : 0.0f;
            if constexpr (CODES) {
                ve = tile_exps(P.v_exps + w.row * w.ngrp, t, w.ngrp);
                ge = tile_exps(P.g_exps + w.row * w.ngrp, t, w.ngrp);
            }
        }
        if constexpr (!VEC)
            __syncwarp();       // every lane has read the stages that are fetched into next
#pragma unroll
        for (int m = 0; m < PER; ++m)
            prefetch();
        cp_async_wait_group<G::DEPTH - PER>();
        if constexpr (!VEC)
            __syncwarp();
        BackSteps<T, CODES> s8[PER];
        float A[PER], D[PER];
        int cnt[PER];
        const uint8_t* from[PER] = {};
        Raw<T> dy[PER];
        auto input = [&](int m, bool gates) {
            std::conditional_t<CODES, RawCodes, Raw<T>> r;
            const uint8_t* p = from[m] + (gates ? G::ARR : 0);
            const int off = gates ? off_g : off_v;
            if constexpr (CODES) {
                if constexpr (VEC)
                    r.w = *reinterpret_cast<const uint2*>(p + 8 * lane);
                else
                    r.w = image_codes(p, off + 8 * lane);
                r.e = __byte_perm(__shfl_sync(kFull, gates ? ge : ve, (k * PER + m) & 31), 0u,
                                  0x4440 + lane / 8);
            } else {
                r = stage_map<T, VEC>(p, off, lane);
            }
            return r;
        };
#pragma unroll
        for (int m = 0; m < PER; ++m) {
            const int here = left + m * kScanTile;
            cnt[m] = here >= kScanTile ? 8 : lane_count(here, lane);
            from[m] = st;
            st = st == last ? mine : st + G::BYTES;
            dy[m] = stage_map<T, VEC>(from[m] + G::DY, off_d, lane);
            s8[m].make(input(m, true), dy[m], cnt[m]);
            A[m] = s8[m].A;
            D[m] = s8[m].D;
        }
#pragma unroll
        for (int m = 0; m < PER; ++m)
            lane_scan<32, true>(A[m], D[m], lane);
        float cin = c;
        if constexpr (TEAM) {
            const float a0 = __shfl_sync(kFull, A[0], 0), d0 = __shfl_sync(kFull, D[0], 0);
            if constexpr (PER == 1) {
                M.publish(k & 1, a0, d0, lane);
            } else {
                const float a1 = __shfl_sync(kFull, A[PER - 1], 0), d1 = __shfl_sync(kFull, D[PER - 1], 0);
                M.publish(k & 1, a0 * a1, fmaf(a1, d0, d1), lane);
            }
            cin = M.join<true>(k & 1, c);
        }
#pragma unroll
        for (int m = 0; m < PER; ++m) {
            float end;
            const float cc = lane_start<32, true>(A[m], D[m], cin, lane, end);
            cin = !TEAM || m + 1 < PER ? __shfl_sync(kFull, end, 0) : 0.0f;
            const float h = __shfl_sync(kFull, states, (k * PER + m) & 31);
            F2 ov[4], og[4];
            s8[m].template grads<32>(input(m, false), dy[m], h, cc, cnt[m], lane, ov, og);
            const long long to = at - m * kScanTile;
            const int here = stored + m * kScanTile;
            tile_store<T, VEC>(static_cast<T*>(P.dv) + to, here, ov, out, lane);
            tile_store<T, VEC>(static_cast<T*>(P.dg) + to, here, og, out, lane);
        }
        if constexpr (!TEAM)
            c = cin;
        left += hop;
        stored += hop;
        at -= hop;
    }
    if (P.hT && lane == 0 && (!TEAM || M.me == 0))
        P.hT[w.row] = c;
}

// ---------------------------------------------------------------- short rows
// Rows of at most 8 S positions: S = 1, 2, 4, 8, 16 or 32 lanes a row, 32 / S
// rows a warp, which are neighbours in memory.  No ring: 131072 bf16 rows of 256
// take 35.7 and 63.8 us forward and backward, 42.2 and 75.4 us as rows of many
// tiles would.
template <int S>
struct Group {
    long long row0, row;    // the warp's first row; this lane's
    int sub, n, L;          // lane within the row; its positions (sequence, row)
    int count, mine;        // elements of the warp's rows; this lane's first among them
    int cnt, all;           // this lane's positions (sequence, row)
    __device__ __forceinline__ void init(const ScanArgs& P, int lane)
    {
        row0 = ((long long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * (32 / S);
        row = row0 + lane / S;
        sub = lane & (S - 1);
        const bool real = row < P.rows;
        L = real ? P.L : 0;
        n = real ? row_len(P.lengths, row, P.C, P.L) : 0;
        const long long rows = P.rows - row0;
        count = (rows < 0 ? 0 : rows > 32 / S ? 32 / S : (int)rows) * P.L;
        mine = lane / S * P.L + sub * 8;
        cnt = min(max(n - sub * 8, 0), 8);
        all = min(max(L - sub * 8, 0), 8);
    }
};

template <typename T, bool VEC>
__device__ __forceinline__ void group_fetch(uint8_t* img, const void* base, long long first, int count,
                                            long long elems, int lane)
{
    if constexpr (!VEC) {
        const uint8_t* b = static_cast<const uint8_t*>(base);
        image_copy(img, b + first * (long long)sizeof(T), count * (int)sizeof(T), b,
                   b + elems * (long long)sizeof(T), lane);
    }
}

template <typename T, bool VEC, int S>
__device__ __forceinline__ Raw<T> group_map(const uint8_t* img, const void* base, long long first, int mine,
                                            int cnt)
{
    Raw<T> r = {};
    const T* p = static_cast<const T*>(base) + first;
    if constexpr (VEC) {
        if (cnt > 0) {
#pragma unroll
            for (int k = 0; k < Raw<T>::N; k += 4) {
                const uint4 q = __ldg(reinterpret_cast<const uint4*>(p + mine) + k / 4);
                r.w[k] = q.x; r.w[k + 1] = q.y; r.w[k + 2] = q.z; r.w[k + 3] = q.w;
            }
        }
    } else {
        const int sh = (int)(reinterpret_cast<uintptr_t>(p) & 15);
        if constexpr (S == 32)
            shifted<Raw<T>::N>(img + mine * (int)sizeof(T), sh, r.w);
        else
            r = image_read<T>(img, sh + mine * (int)sizeof(T));
    }
    return r;
}

template <bool VEC>
__device__ __forceinline__ RawCodes group_codes(const uint8_t* img, const uint8_t* base, const uint8_t* exp,
                                                long long first, int mine, int cnt)
{
    RawCodes r = {};
    if (cnt > 0)
        r.e = __ldg(exp);
    const uint8_t* p = base + first;
    if constexpr (VEC) {
        if (cnt > 0)
            r.w = __ldg(reinterpret_cast<const uint2*>(p + mine));
    } else {
        r.w = image_codes(img, (int)(reinterpret_cast<uintptr_t>(p) & 15) + mine);
    }
    return r;
}

template <typename T, bool VEC, int S>
__device__ __forceinline__ void group_store(T* base, const Group<S>& w, long long first, const F2 (&x)[4],
                                            uint8_t* img, int lane)
{
    const Raw<T> r = pack8<T>(x);
    if constexpr (VEC) {
        if (w.all > 0) {
#pragma unroll
            for (int k = 0; k < Raw<T>::N; k += 4)
                reinterpret_cast<uint4*>(base + first + w.mine)[k / 4] =
                    make_uint4(r.w[k], r.w[k + 1], r.w[k + 2], r.w[k + 3]);
        }
    } else {
        image_store<T, S == 32>(base + first, w.count, w.mine, w.all, r, img, lane);
    }
}

template <typename T, int S, bool VEC, bool KEEP>
__global__ void __launch_bounds__(32 * kWarps) scan_fwd_short_kernel(const ScanArgs P)
{
    __shared__ __align__(16) uint8_t images[kWarps][VEC ? 16 : 2 * kImage<T>];
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31;
    uint8_t* const img = images[threadIdx.x >> 5];
    Group<S> w;
    w.init(P, lane);
    const long long first = w.row0 * P.L, elems = P.rows * P.L;
    group_fetch<T, VEC>(img, P.v, first, w.count, elems, lane);
    group_fetch<T, VEC>(img + kImage<T>, P.g, first, w.count, elems, lane);
    cp_async_wait_all();
    __syncwarp();
    Inputs<T, false> in;
    in.v = group_map<T, VEC, S>(img, P.v, first, w.mine, w.cnt);
    in.g = group_map<T, VEC, S>(img + kImage<T>, P.g, first, w.mine, w.cnt);
    const float h = P.h0 && w.L > 0 ? P.h0[w.row] : 0.0f;
    Steps<T, false> s8;
    s8.make(in, w.cnt);
    float A = s8.A, H = s8.H, end;
    lane_scan<S, false>(A, H, w.sub);
    const float s = lane_start<S, false>(A, H, h, w.sub, end);
    F2 y[4];
    s8.replay(s, y);
    if (w.cnt < 8)
        cut8(y, w.cnt, 0.0f);
    group_store<T, VEC>(static_cast<T*>(P.y), w, first, y, img, lane);
    if constexpr (KEEP) {
        uint2 cv, cg;
        uint32_t ev, eg;
        encode8<S>(in.v, in.g, w.cnt, cv, cg, ev, eg);
        if constexpr (VEC) {
            if (w.all > 0) {
                *reinterpret_cast<uint2*>(P.v_codes + first + w.mine) = cv;
                *reinterpret_cast<uint2*>(P.g_codes + first + w.mine) = cg;
            }
        } else {
            image_store_codes<S == 32>(P.v_codes + first, w.count, w.mine, w.all, cv, img, lane);
            image_store_codes<S == 32>(P.g_codes + first, w.count, w.mine, w.all, cg, img, lane);
        }
        if (w.all > 0 && (w.sub & 7) == 0) {
            const int ngrp = (P.L + WBMM_SEQ_GROUP - 1) / WBMM_SEQ_GROUP;
            const long long grp = w.row * ngrp + w.sub / 8;
            P.v_exps[grp] = (uint8_t)ev;
            P.g_exps[grp] = (uint8_t)eg;
        }
    }
    if (P.states && w.sub == 0 && w.n > 0)
        P.states[w.row] = h;
    if (P.hT && w.sub == S - 1 && w.L > 0)
        P.hT[w.row] = end;
}

template <typename T, int S, bool VEC, bool CODES>
__global__ void __launch_bounds__(32 * kWarps) scan_bwd_short_kernel(const ScanArgs P)
{
    __shared__ __align__(16) uint8_t images[kWarps][VEC ? 16 : 3 * kImage<T>];
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31;
    uint8_t* const img = images[threadIdx.x >> 5];
    Group<S> w;
    w.init(P, lane);
    const long long first = w.row0 * P.L, elems = P.rows * P.L;
    if constexpr (CODES) {
        group_fetch<uint8_t, VEC>(img, P.v_codes, first, w.count, elems, lane);
        group_fetch<uint8_t, VEC>(img + kImage<T>, P.g_codes, first, w.count, elems, lane);
    } else {
        group_fetch<T, VEC>(img, P.v, first, w.count, elems, lane);
        group_fetch<T, VEC>(img + kImage<T>, P.g, first, w.count, elems, lane);
    }
    group_fetch<T, VEC>(img + 2 * kImage<T>, P.dy, first, w.count, elems, lane);
    cp_async_wait_all();
    __syncwarp();
    Inputs<T, CODES> in;
    if constexpr (CODES) {
        const int ngrp = (P.L + WBMM_SEQ_GROUP - 1) / WBMM_SEQ_GROUP;
        const long long grp = w.row * ngrp + w.sub / 8;
        in.v = group_codes<VEC>(img, P.v_codes, P.v_exps + grp, first, w.mine, w.cnt);
        in.g = group_codes<VEC>(img + kImage<T>, P.g_codes, P.g_exps + grp, first, w.mine, w.cnt);
    } else {
        in.v = group_map<T, VEC, S>(img, P.v, first, w.mine, w.cnt);
        in.g = group_map<T, VEC, S>(img + kImage<T>, P.g, first, w.mine, w.cnt);
    }
    const Raw<T> dy = group_map<T, VEC, S>(img + 2 * kImage<T>, P.dy, first, w.mine, w.cnt);
    const float c = P.h0 && w.L > 0 ? P.h0[w.row] : 0.0f;
    const float h = w.n > 0 ? __ldg(P.states + w.row) : 0.0f;
    BackSteps<T, CODES> s8;
    s8.make(in.g, dy, w.cnt);
    float A = s8.A, D = s8.D, end;
    lane_scan<S, true>(A, D, w.sub);
    const float cc = lane_start<S, true>(A, D, c, w.sub, end);
    F2 ov[4], og[4];
    s8.template grads<S>(in.v, dy, h, cc, w.cnt, w.sub, ov, og);
    group_store<T, VEC>(static_cast<T*>(P.dv), w, first, ov, img, lane);
    group_store<T, VEC>(static_cast<T*>(P.dg), w, first, og, img, lane);
    if (P.hT && w.sub == 0 && w.L > 0)
        P.hT[w.row] = end;
}

// ------------------------------------------------------------- one position
// One position of every row, V rows a thread: 1, or 8 as 16-byte vectors.
template <typename T, int V>
__global__ void __launch_bounds__(128)
    scan_step_kernel(const T* __restrict__ v, const T* __restrict__ g, const float* h, T* y,
                     float* h_next, long long rows)
{
    const long long r = ((long long)blockIdx.x * 128 + threadIdx.x) * V;
    grid_dep_wait();
    grid_dep_launch();
    if (r >= rows)
        return;
    if constexpr (V == 1) {
        F2 f, i;
        const float a = sizeof(T) == 2 ? max_nan(to_f(g[r]), kGateMin) : to_f(g[r]);
        gate2<T>({a, a}, f, i);
        const float s = fmaf(f.x, h[r], i.x * to_f(v[r]));
        put(y + r, s);
        h_next[r] = s;
    } else {
        Raw<T> rv, rg;
        F2 xv[4], xg[4], s[4];
#pragma unroll
        for (int k = 0; k < Raw<T>::N; k += 4) {
            const uint4 a = __ldg(reinterpret_cast<const uint4*>(v + r) + k / 4);
            const uint4 b = __ldg(reinterpret_cast<const uint4*>(g + r) + k / 4);
            rv.w[k] = a.x; rv.w[k + 1] = a.y; rv.w[k + 2] = a.z; rv.w[k + 3] = a.w;
            rg.w[k] = b.x; rg.w[k + 1] = b.y; rg.w[k + 2] = b.z; rg.w[k + 3] = b.w;
        }
        const float4 h0 = *reinterpret_cast<const float4*>(h + r);
        const float4 h1 = *reinterpret_cast<const float4*>(h + r + 4);
        const F2 was[4] = {{h0.x, h0.y}, {h0.z, h0.w}, {h1.x, h1.y}, {h1.z, h1.w}};
        unpack8(rv, xv);
        unpack_gates8(rg, xg);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            F2 f, i;
            gate2<T>(xg[j], f, i);
            s[j] = fma2(f, was[j], mul2(i, xv[j]));
        }
        const Raw<T> out = pack8<T>(s);
#pragma unroll
        for (int k = 0; k < Raw<T>::N; k += 4)
            reinterpret_cast<uint4*>(y + r)[k / 4] =
                make_uint4(out.w[k], out.w[k + 1], out.w[k + 2], out.w[k + 3]);
        *reinterpret_cast<float4*>(h_next + r) = make_float4(s[0].x, s[0].y, s[1].x, s[1].y);
        *reinterpret_cast<float4*>(h_next + r + 4) = make_float4(s[2].x, s[2].y, s[3].x, s[3].y);
    }
}

cudaError_t done(cudaError_t e)
{
    if (e != cudaSuccess)
        return e;
    note_launches(1);
    return cudaGetLastError();
}

template <typename T, int S, bool VEC, bool AUX>
cudaError_t short_launch(const ScanArgs& A, bool backward, const Launch& L)
{
    const long long per = 32 / S * kWarps;
    const dim3 grid((unsigned)((A.rows + per - 1) / per)), block(32 * kWarps);
    return done(backward ? launch_pdl(scan_bwd_short_kernel<T, S, VEC, AUX>, grid, block, 0, L.stream, A)
                         : launch_pdl(scan_fwd_short_kernel<T, S, VEC, AUX>, grid, block, 0, L.stream, A));
}

// A warp a row.
template <typename T, bool VEC, bool AUX>
cudaError_t row_launch(const ScanArgs& A, bool backward, const Launch& L)
{
    const dim3 grid((unsigned)((A.rows + kWarps - 1) / kWarps)), block(32 * kWarps);
    return done(backward ? launch_pdl(scan_bwd_kernel<T, VEC, AUX, false>, grid, block, 0, L.stream, A)
                         : launch_pdl(scan_fwd_kernel<T, VEC, AUX, false>, grid, block, 0, L.stream, A));
}

// The warps of `ctas` CTAs (a cluster) a row.
template <typename T, bool VEC, bool AUX>
cudaError_t team_launch(const ScanArgs& A, bool backward, int ctas, const Launch& L)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(A.rows * ctas));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return done(cudaLaunchKernelEx(&cfg,
                                   backward ? scan_bwd_kernel<T, VEC, AUX, true>
                                            : scan_fwd_kernel<T, VEC, AUX, true>,
                                   A));
}

// Warps a row: one where that gives an SM 10 of them, else a team of 4 for rows
// of 2 tiles or more, of 8, 16 and 32 while that gives an SM fewer than 10 and a
// row has two tiles for each warp of the team that is doubled (so one for each
// of the doubled one).  Measured, forward and backward, bf16: 8192 rows of 3136
// positions 28 and 43 us with a warp each, 39 and 64 us with teams of 4; 1600
// rows of 4096 10.0 and 15.6 us, 9.7 and 16.4 us; of 16384 31.7 and 49.8 us, 27.6
// and 46.0 us; 768 rows of 50176 81 and 128 us with a warp each, 43 and 79 us with
// teams of 4, 54 and 95 us with teams of 8; 128 rows of 65536 25 and 33 us with
// teams of 8, 20 and 24 us with 16, 22 and 28 us with 32.  Near the rule's edges:
// 64 rows of 4096 2.8 and 3.6 us with teams of 4, 3.0 and 3.3 with 8, 3.0 and 3.6
// with 16 (taken), 6.4 and 9.7 with a warp each; 64 rows of 2048 2.1 and 2.5 us
// with 4, 2.8 and 3.3 with 8 (taken), 3.8 and 5.6 with a warp each.  Where many
// rows have 2 tiles a team's idle warps cost: 1024 rows of 512 2.3 and 2.8 us with
// a warp each, 4.5 and 6.4 us with teams of 4 (taken).
int team_for(long long rows, int L, int num_sms)
{
    const long long tiles = ((long long)L + kScanTile - 1) / kScanTile;
    int team = 1;
    while (team < kTeamMax && rows * team < 10ll * num_sms && 2 * team <= tiles)
        team = team == 1 ? 4 : 2 * team;
    return team;
}

template <typename T, bool VEC, bool AUX>
cudaError_t lanes_launch(const ScanArgs& A, bool backward, const Launch& L)
{
    // as few lanes as hold a row in one tile
    if (A.L <= 8)
        return short_launch<T, 1, VEC, AUX>(A, backward, L);
    if (A.L <= 16)
        return short_launch<T, 2, VEC, AUX>(A, backward, L);
    if (A.L <= 32)
        return short_launch<T, 4, VEC, AUX>(A, backward, L);
    if (A.L <= 64)
        return short_launch<T, 8, VEC, AUX>(A, backward, L);
    if (A.L <= 128)
        return short_launch<T, 16, VEC, AUX>(A, backward, L);
    if (A.L <= kScanTile)
        return short_launch<T, 32, VEC, AUX>(A, backward, L);
    const int team = team_for(A.rows, A.L, L.num_sms);
    if (team > 1)
        return team_launch<T, VEC, AUX>(A, backward, team / kWarps, L);
    return row_launch<T, VEC, AUX>(A, backward, L);
}

cudaError_t scan_launch(const ScanArgs& A, bool is_bf16, bool backward, const Launch& L)
{
    const bool aux = A.v_codes != nullptr;
    if (!is_bf16)
        return aux ? lanes_launch<float, false, true>(A, backward, L)
                   : lanes_launch<float, false, false>(A, backward, L);
    if (A.L % 8 == 0)
        return aux ? lanes_launch<__nv_bfloat16, true, true>(A, backward, L)
                   : lanes_launch<__nv_bfloat16, true, false>(A, backward, L);
    return aux ? lanes_launch<__nv_bfloat16, false, true>(A, backward, L)
               : lanes_launch<__nv_bfloat16, false, false>(A, backward, L);
}

}  // namespace


cudaError_t scan_backward_launch(const ScanArgs& A, bool is_bf16, const Launch& L)
{
    return scan_launch(A, is_bf16, true, L);
}

namespace {

template <typename T>
cudaError_t step_launch(const void* v, const void* g, const float* h, void* y, float* h_next,
                        long long rows, const Launch& L)
{
    // 8 rows a thread once that leaves an SM two blocks of threads, where the
    // buffers allow it: 256 x 8192 bf16 rows take 6.3 us (17.9 one a thread), fp32
    // ones 10.8 us.  A thread's 32 bytes of an fp32 array (the states; in fp32 all
    // five) are two accesses 32 bytes apart, each half of every sector
    uintptr_t all = 0;
    for (const void* p : {v, g, (const void*)h, (const void*)y, (const void*)h_next})
        all |= reinterpret_cast<uintptr_t>(p);
    const bool wide = rows % 8 == 0 && all % 16 == 0 && rows >= 2048ll * L.num_sms;
    const long long threads = wide ? rows / 8 : rows;
    const dim3 grid((unsigned)((threads + 127) / 128)), block(128);
    const T *pv = static_cast<const T*>(v), *pg = static_cast<const T*>(g);
    T* py = static_cast<T*>(y);
    return done(wide ? launch_pdl(scan_step_kernel<T, 8>, grid, block, 0, L.stream, pv, pg, h, py, h_next, rows)
                     : launch_pdl(scan_step_kernel<T, 1>, grid, block, 0, L.stream, pv, pg, h, py, h_next, rows));
}

}  // namespace

cudaError_t scan_step_launch(const void* v, const void* g, const float* h, void* y, float* h_next,
                             long long rows, bool is_bf16, const Launch& L)
{
    return is_bf16 ? step_launch<__nv_bfloat16>(v, g, h, y, h_next, rows, L)
                   : step_launch<float>(v, g, h, y, h_next, rows, L);
}

cudaError_t scan_forward_launch(const ScanArgs& A, bool is_bf16, const Launch& L)
{
    // one position of every row is a step (256 x 8192 bf16 rows 6.3 us, 30 as
    // rows of one position), unless it is masked or kept for a backward pass
    if (A.L == 1 && A.h0 && A.hT && !A.lengths && !A.states && !A.v_codes)
        return scan_step_launch(A.v, A.g, A.h0, A.y, A.hT, A.rows, is_bf16, L);
    return scan_launch(A, is_bf16, false, L);
}

}  // namespace wbmm
