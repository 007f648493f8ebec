// k_norm.cu -- root-mean-square norm of rows, with the residual's addition, an
// 8-bit output and the gradient (sm_100a).
//
//   s = x + r,  y = w s (mean s^2 + eps)^(-1/2)
//   y8 = e4m3(y / scale), scale = max|y| / 448 over the row or over 128 columns
// Gradient at the norm's input s (rs = (mean s^2 + eps)^(-1/2), s^ = s rs):
//   dx = d_sum + rs (w dy - s^ mean(w dy s^)),   dw = sum over rows of dy s^
//
// Bound by memory: every element is read and written once.  A row belongs to
// TPR threads (8 consecutive elements a thread and vector, up to NV vectors),
// whose loads are all issued before any arithmetic.  The reduction is shuffles
// (TPR <= 32) or shuffles and one exchange through shared memory.  Sums are
// float32.  A 128-column scale is the maximum over 16 lanes that hold one block,
// so 8-bit output needs no second pass.  The weight's gradient stays in
// registers over the rows that a thread group walks; the CTAs' parts are added
// by a second kernel in a fixed order.  Rows whose width is not a multiple of 8
// start anywhere: their threads load single elements, a warp 32 neighbours, and a
// warp has whole blocks of 128 columns, so that scales and the weight's gradient
// need no other layout.  Rows too wide for registers, and most rows of odd width
// above 384 columns, take kernels that read the row again from cache.
#include <cuda_fp8.h>

#define M3_BOUNDS_FILE 11
#include "m3_bounds.cuh"
#include "m3_common.cuh"
#include "m3_kernels.h"
#include "m3_norm.h"

namespace m3 {
namespace norm {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kE4M3Max = 448.f;
constexpr float kTiny = 1e-30f;      // floor of a scale's maximum: an all-zero block has a finite scale

// 8 elements as loaded (kept packed until they are used) and as float
template <typename T> struct Vec8;
template <> struct Vec8<__nv_bfloat16> {
    struct Raw { uint4 v; };
    static __device__ __forceinline__ Raw fetch(const void* base, size_t o) {
        return {__ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + o))};
    }
    static __device__ __forceinline__ Raw none() { return {make_uint4(0u, 0u, 0u, 0u)}; }
    static __device__ __forceinline__ void open(const Raw& r, float* f) {
        const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = __uint_as_float(w[j] << 16);
            f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(void* base, size_t o, const float* f) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
            memcpy(&w[j], &v, 4);
        }
        __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + o), make_uint4(w[0], w[1], w[2], w[3]));
    }
};
template <> struct Vec8<float> {
    struct Raw { float4 a, b; };
    static __device__ __forceinline__ Raw fetch(const void* base, size_t o) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + o);
        return {__ldcs(p), __ldcs(p + 1)};
    }
    static __device__ __forceinline__ Raw none() { return {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)}; }
    static __device__ __forceinline__ void open(const Raw& r, float* f) {
        f[0] = r.a.x; f[1] = r.a.y; f[2] = r.a.z; f[3] = r.a.w;
        f[4] = r.b.x; f[5] = r.b.y; f[6] = r.b.z; f[7] = r.b.w;
    }
    static __device__ __forceinline__ void store(void* base, size_t o, const float* f) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + o);
        __stcs(p, make_float4(f[0], f[1], f[2], f[3]));
        __stcs(p + 1, make_float4(f[4], f[5], f[6], f[7]));
    }
};

// elements j and j + 1 as a pair (two lanes of one float32x2 instruction)
__device__ __forceinline__ float2 pair(const float* f, int j) { return make_float2(f[j], f[j + 1]); }
__device__ __forceinline__ void put(float* f, int j, float2 v) {
    f[j] = v.x;
    f[j + 1] = v.y;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// NA arrays' elements of a row that a thread holds, NV vectors of each
template <typename T, int NV, int NA>
struct RowRegs {
    typename Vec8<T>::Raw r[NA][NV];
    __device__ __forceinline__ void fetch(const void* const (&src)[NA], const NormParams& q, long long row, int lane, int tpr) {
        const bool live = row < q.rows;
        const size_t base = live ? (size_t)row * q.width : 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + tpr * i) * 8;
            const bool in = live && c < q.width && M3_SPAN(1, base + c, 8, q.rows * q.width);
#pragma unroll
            for (int a = 0; a < NA; ++a) r[a][i] = in && src[a] ? Vec8<T>::fetch(src[a], base + c) : Vec8<T>::none();
        }
    }
};

__device__ __forceinline__ void load_weight8(const float* w, int c, float* f) {
    if (!w) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = 1.f;
        return;
    }
    const float4 a = __ldg(reinterpret_cast<const float4*>(w + c)), b = __ldg(reinterpret_cast<const float4*>(w + c) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

__device__ __forceinline__ uint2 e4m3x8(const float* f, float inv) {
    uint32_t w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const __nv_fp8x2_storage_t lo =
            __nv_cvt_float2_to_fp8x2(make_float2(f[4 * j] * inv, f[4 * j + 1] * inv), __NV_SATFINITE, __NV_E4M3);
        const __nv_fp8x2_storage_t hi =
            __nv_cvt_float2_to_fp8x2(make_float2(f[4 * j + 2] * inv, f[4 * j + 3] * inv), __NV_SATFINITE, __NV_E4M3);
        w[j] = (uint32_t)lo | ((uint32_t)hi << 16);
    }
    return make_uint2(w[0], w[1]);
}

// NaN-keeping maximum: a row with a NaN gets a NaN scale, not a finite one
__device__ __forceinline__ float nmax(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// sum (or maximum) over the TPR threads of a row; `buf` holds one value a warp
// of the CTA.  Every thread of the CTA calls it.
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, int tpr, float* buf) {
    for (int o = min(tpr, 32) >> 1; o; o >>= 1) {
        const float u = __shfl_xor_sync(kFull, v, o);
        v = MAX ? nmax(v, u) : v + u;
    }
    if (tpr > 32) {
        const int warp = threadIdx.x >> 5, per = tpr >> 5, first = warp / per * per;
        __syncthreads();
        if ((threadIdx.x & 31) == 0) buf[warp] = v;
        __syncthreads();
        v = buf[first];
        for (int i = 1; i < per; ++i) v = MAX ? nmax(v, buf[first + i]) : v + buf[first + i];
    }
    return v;
}

// Both sums of a row in one reduction; `buf` has two sets of a pair a warp,
// taken in turn, so that one barrier a row is enough.
__device__ __forceinline__ float2 row_reduce2(float2 v, int tpr, float2* buf) {
    for (int o = min(tpr, 32) >> 1; o; o >>= 1) {
        v.x += __shfl_xor_sync(kFull, v.x, o);
        v.y += __shfl_xor_sync(kFull, v.y, o);
    }
    if (tpr > 32) {
        const int warp = threadIdx.x >> 5, per = tpr >> 5, first = warp / per * per;
        if ((threadIdx.x & 31) == 0) buf[warp] = v;
        __syncthreads();
        v = buf[first];
        for (int i = 1; i < per; ++i) {
            v.x += buf[first + i].x;
            v.y += buf[first + i].y;
        }
    }
    return v;
}

// RES: a residual is added; Q8: an 8-bit output is written.  At most 40 registers
// a thread (three CTAs of 512 an SM), so that enough loads are in flight:
// 32768 x 2048 with residual and 8-bit output takes 88 us (5.3 TB/s, 83 % of the
// copy rate), 99 without the bound; arithmetic in pairs, 94 without.
template <typename T, int NV, bool RES, bool Q8>
__global__ void __launch_bounds__(512, NV <= 2 ? 3 : 1) norm_kernel(NormParams q, int tpr) {
    __shared__ float buf[16];
    const int lane = threadIdx.x & (tpr - 1), per = blockDim.x / tpr;
    const long long row = (long long)blockIdx.x * per + threadIdx.x / tpr;
    const long long ext = q.rows * q.width;
    const void* src[RES ? 2 : 1];
    src[0] = q.x;
    if constexpr (RES) src[1] = q.residual;
    const bool live = row < q.rows;
    const size_t base = live ? (size_t)row * q.width : 0;
    RowRegs<T, NV, RES ? 2 : 1> cur;
    cur.fetch(src, q, row, lane, tpr);
    {
        float s[NV][8];
        float2 ss2 = both(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Vec8<T>::open(cur.r[0][i], s[i]);
            if constexpr (RES) {
                float r[8];
                Vec8<T>::open(cur.r[1][i], r);
#pragma unroll
                for (int j = 0; j < 8; j += 2) put(s[i], j, __fadd2_rn(pair(s[i], j), pair(r, j)));
            }
#pragma unroll
            for (int j = 0; j < 8; j += 2) ss2 = __ffma2_rn(pair(s[i], j), pair(s[i], j), ss2);
        }
        const float ss = row_reduce<false>(ss2.x + ss2.y, tpr, buf);
        const float rs = rsqrtf(ss / (float)q.width + q.eps);
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + tpr * i) * 8;
            const bool in = live && c < q.width && M3_SPAN(3, base + c, 8, ext);
            if (in && q.sum) Vec8<T>::store(q.sum, base + c, s[i]);
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 0.f;
            if (in) load_weight8(q.weight, c, w);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                put(s[i], j, __fmul2_rn(__fmul2_rn(pair(s[i], j), both(rs)), pair(w, j)));
                if (Q8 && in) top = nmax(nmax(top, fabsf(s[i][j])), fabsf(s[i][j + 1]));
            }
            if (in && q.y) Vec8<T>::store(q.y, base + c, s[i]);
            if (Q8 && q.block) {          // 16 lanes hold the 128 columns of one scale
                for (int o = 8; o; o >>= 1) top = nmax(top, __shfl_xor_sync(kFull, top, o));
                top = nmax(top, kTiny);
                const int nb = (q.width + 127) >> 7;
                if (in) __stcs(reinterpret_cast<uint2*>(q.y8 + base + c), e4m3x8(s[i], __fdiv_rn(kE4M3Max, top)));
                if (in && (c & 127) == 0 && M3_IN(7, row * nb + (c >> 7), q.rows * nb)) q.scale[row * nb + (c >> 7)] = top * (1.f / kE4M3Max);
                top = 0.f;
            }
        }
        if (Q8 && !q.block) {
            top = nmax(row_reduce<true>(top, tpr, buf), kTiny);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (lane + tpr * i) * 8;
                if (live && c < q.width && M3_SPAN(8, base + c, 8, ext))
                    __stcs(reinterpret_cast<uint2*>(q.y8 + base + c), e4m3x8(s[i], __fdiv_rn(kE4M3Max, top)));
            }
            if (live && lane == 0 && M3_IN(9, row, q.rows)) q.scale[row] = top * (1.f / kE4M3Max);
        }
    }
}

// Rows of any width up to 8192.  Warp w of the WPR warps of a row has the blocks
// of 128 columns w, w + WPR, ... (NB of them), lane l the columns l, l + 32, l + 64
// and l + 96 of each; all loads go out before any arithmetic.
template <typename T, int NB>
__global__ void __launch_bounds__(512) norm_odd_kernel(NormParams q, int wpr) {
    __shared__ float buf[16];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w0 = warp & (wpr - 1), tpr = 32 * wpr;
    const long long row = (long long)blockIdx.x * (blockDim.x / tpr) + warp / wpr;
    const long long ext = q.rows * q.width;
    const bool live = row < q.rows;
    const size_t base = live ? (size_t)row * q.width : 0;
    const T* x = static_cast<const T*>(q.x);
    const T* r = static_cast<const T*>(q.residual);
    float s[4 * NB], v[4 * NB];
    auto col = [&](int e) { return (w0 + wpr * (e >> 2)) * 128 + (e & 3) * 32 + lane; };
#pragma unroll
    for (int e = 0; e < 4 * NB; ++e) {
        const bool in = live && col(e) < q.width && M3_IN(30, base + col(e), ext);
        s[e] = in ? ld_io(x + base + col(e)) : 0.f;
        v[e] = in && r ? ld_io(r + base + col(e)) : 0.f;
    }
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 4 * NB; ++e) {
        s[e] += v[e];
        ss = fmaf(s[e], s[e], ss);
    }
    ss = row_reduce<false>(ss, tpr, buf);
    const float rs = rsqrtf(ss / (float)q.width + q.eps);
#pragma unroll
    for (int e = 0; e < 4 * NB; ++e) {
        const bool in = live && col(e) < q.width && M3_IN(31, base + col(e), ext);
        v[e] = in ? s[e] * rs * (q.weight ? __ldg(q.weight + col(e)) : 1.f) : 0.f;
        if (in && q.sum) st_io(static_cast<T*>(q.sum) + base + col(e), s[e]);
        if (in && q.y) st_io(static_cast<T*>(q.y) + base + col(e), v[e]);
    }
    if (!q.y8) return;
    const int nb = q.block ? (q.width + 127) >> 7 : 1;
    float top = 0.f;
    if (!q.block) {
#pragma unroll
        for (int e = 0; e < 4 * NB; ++e) top = nmax(top, fabsf(v[e]));
        top = nmax(row_reduce<true>(top, tpr, buf), kTiny);
        if (live && w0 == 0 && lane == 0 && M3_IN(32, row, q.rows)) q.scale[row] = top * (1.f / kE4M3Max);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        if (q.block) {
            top = nmax(nmax(fabsf(v[4 * b]), fabsf(v[4 * b + 1])), nmax(fabsf(v[4 * b + 2]), fabsf(v[4 * b + 3])));
#pragma unroll
            for (int o = 16; o; o >>= 1) top = nmax(top, __shfl_xor_sync(kFull, top, o));
            top = nmax(top, kTiny);
            const int k = w0 + wpr * b;
            if (live && lane == 0 && k < nb && M3_IN(33, row * nb + k, q.rows * nb)) q.scale[row * nb + k] = top * (1.f / kE4M3Max);
        }
        const float inv = __fdiv_rn(kE4M3Max, top);
#pragma unroll
        for (int e = 4 * b; e < 4 * b + 4; ++e)
            if (live && col(e) < q.width && M3_IN(34, base + col(e), ext))
                q.y8[base + col(e)] = __nv_cvt_float_to_fp8(v[e] * inv, __NV_SATFINITE, __NV_E4M3);
    }
}

// Rows of any width (which ones: odd_shape_of's comment): one CTA a row, elements
// strided over the threads
template <typename T>
__global__ void __launch_bounds__(256) norm_any_kernel(NormParams q) {
    __shared__ float buf[16];
    const T* x = static_cast<const T*>(q.x);
    const T* r = static_cast<const T*>(q.residual);
    const size_t base = (size_t)blockIdx.x * q.width;
    const long long ext = q.rows * q.width;
    float ss = 0.f;
    for (int c = threadIdx.x; c < q.width; c += 256) {
        if (!M3_IN(10, base + c, ext)) continue;
        const float s = ld_io(x + base + c) + (r ? ld_io(r + base + c) : 0.f);
        ss = fmaf(s, s, ss);
    }
    ss = row_reduce<false>(ss, 256, buf);
    const float rs = rsqrtf(ss / (float)q.width + q.eps);
    const int block = q.block ? q.block : q.width;
    const int nb = (q.width - 1) / block + 1;
    for (int k = 0; k < nb; ++k) {
        const int c1 = min(q.width, (k + 1) * block);
        float top = 0.f;
        if (q.y8) {
            for (int c = k * block + threadIdx.x; c < c1; c += 256) {
                if (!M3_IN(11, base + c, ext)) continue;
                const float s = ld_io(x + base + c) + (r ? ld_io(r + base + c) : 0.f);
                top = nmax(top, fabsf(s * rs * (q.weight ? q.weight[c] : 1.f)));
            }
            top = nmax(row_reduce<true>(top, 256, buf), kTiny);
            if (threadIdx.x == 0 && M3_IN(12, (long long)blockIdx.x * nb + k, q.rows * nb))
                q.scale[(size_t)blockIdx.x * nb + k] = top / kE4M3Max;
        }
        for (int c = k * block + threadIdx.x; c < c1; c += 256) {
            if (!M3_IN(13, base + c, ext)) continue;
            const float s = ld_io(x + base + c) + (r ? ld_io(r + base + c) : 0.f);
            const float y = s * rs * (q.weight ? q.weight[c] : 1.f);
            if (q.sum) st_io(static_cast<T*>(q.sum) + base + c, s);
            if (q.y) st_io(static_cast<T*>(q.y) + base + c, y);
            if (q.y8) q.y8[base + c] = __nv_cvt_float_to_fp8(y * (kE4M3Max / top), __NV_SATFINITE, __NV_E4M3);
        }
    }
}

// ---------------------------------------------------------------- gradient --
// The weight's gradient of a group's columns stays in registers; at the end the
// groups of a CTA are added through shared memory (`part` has a row a CTA).
template <typename T, int NV>
__global__ void __launch_bounds__(512) norm_bwd_kernel(NormParams q, int tpr) {
    extern __shared__ float sums[];
    __shared__ float2 buf[2][16];
    const int lane = threadIdx.x & (tpr - 1), per = blockDim.x / tpr, sub = threadIdx.x / tpr;
    const long long group = (long long)blockIdx.x * per + sub, groups = (long long)gridDim.x * per;
    const long long ext = q.rows * q.width;
    const void* const src[3] = {q.x, q.dy, q.d_sum};
    float dw[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
    // all groups of a CTA take the same number of rounds (the reduction may be CTA-wide)
    const long long rounds = (q.rows + groups - 1) / groups;
    // a row's loads are issued while the row before is reduced
    RowRegs<T, NV, 3> next;
    next.fetch(src, q, group, lane, tpr);
    for (long long k = 0; k < rounds; ++k) {
        const long long row = k * groups + group;
        const bool live = row < q.rows;
        const size_t base = live ? (size_t)row * q.width : 0;
        const RowRegs<T, NV, 3> cur = next;
        float2 ss = both(0.f), sd = both(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + tpr * i) * 8;
            float s[8], d[8], w[8];
            Vec8<T>::open(cur.r[0][i], s);
            Vec8<T>::open(cur.r[1][i], d);
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 0.f;
            if (c < q.width && M3_SPAN(15, c, 8, q.width)) load_weight8(q.weight, c, w);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                ss = __ffma2_rn(pair(s, j), pair(s, j), ss);
                sd = __ffma2_rn(__fmul2_rn(pair(s, j), pair(w, j)), pair(d, j), sd);
            }
        }
        if (k + 1 < rounds) next.fetch(src, q, row + groups, lane, tpr);
        const float2 sum = row_reduce2(make_float2(ss.x + ss.y, sd.x + sd.y), tpr, buf[k & 1]);
        const float rs = rsqrtf(sum.x / (float)q.width + q.eps);
        const float m = sum.y * rs * rs / (float)q.width;          // mean(w dy s^) rs
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + tpr * i) * 8;
            if (!(live && c < q.width && M3_SPAN(16, base + c, 8, ext))) continue;
            float s[8], d[8], w[8], e[8];
            Vec8<T>::open(cur.r[0][i], s);
            Vec8<T>::open(cur.r[1][i], d);
            Vec8<T>::open(cur.r[2][i], e);
            load_weight8(q.weight, c, w);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float2 s2 = pair(s, j), d2 = pair(d, j);
                put(dw[i], j, __ffma2_rn(d2, __fmul2_rn(s2, both(rs)), pair(dw[i], j)));
                put(e, j, __ffma2_rn(both(rs), __ffma2_rn(pair(w, j), d2, __fmul2_rn(s2, both(-m))), pair(e, j)));
            }
            Vec8<T>::store(q.dx, base + c, e);
        }
    }
    if (!q.dweight) return;
    // group by group into the CTA's sums
    for (int g = 0; g < per; ++g) {
        if (sub == g) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (lane + tpr * i) * 8;
                if (c < q.width && M3_SPAN(17, c, 8, dyn_smem_bytes() / 4)) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) sums[c + j] = g ? sums[c + j] + dw[i][j] : dw[i][j];
                }
            }
        }
        __syncthreads();
    }
    for (int c = threadIdx.x; c < q.width; c += blockDim.x)
        if (M3_IN(24, (long long)blockIdx.x * q.width + c, (long long)q.parts * q.width))
            q.part[(size_t)blockIdx.x * q.width + c] = sums[c];
}

// Rows of any width up to 8192, in the layout of norm_odd_kernel
template <typename T, int NB>
__global__ void __launch_bounds__(512) norm_bwd_odd_kernel(NormParams q, int wpr) {
    extern __shared__ float sums[];
    __shared__ float2 buf[2][16];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w0 = warp & (wpr - 1), tpr = 32 * wpr;
    const int per = blockDim.x / tpr, sub = warp / wpr;
    const long long group = (long long)blockIdx.x * per + sub, groups = (long long)gridDim.x * per;
    const long long ext = q.rows * q.width, rounds = (q.rows + groups - 1) / groups;
    const T* x = static_cast<const T*>(q.x);
    const T* dy = static_cast<const T*>(q.dy);
    const T* ds = static_cast<const T*>(q.d_sum);
    auto col = [&](int e) { return (w0 + wpr * (e >> 2)) * 128 + (e & 3) * 32 + lane; };
    float w[4 * NB], dw[4 * NB];
#pragma unroll
    for (int e = 0; e < 4 * NB; ++e) {
        w[e] = col(e) >= q.width ? 0.f : q.weight ? __ldg(q.weight + col(e)) : 1.f;
        dw[e] = 0.f;
    }
    for (long long k = 0; k < rounds; ++k) {
        const long long row = k * groups + group;
        const bool live = row < q.rows;
        const size_t base = live ? (size_t)row * q.width : 0;
        float s[4 * NB], d[4 * NB], g[4 * NB];
#pragma unroll
        for (int e = 0; e < 4 * NB; ++e) {
            const bool in = live && col(e) < q.width && M3_IN(35, base + col(e), ext);
            s[e] = in ? ld_io(x + base + col(e)) : 0.f;
            d[e] = in ? ld_io(dy + base + col(e)) : 0.f;
            g[e] = in && ds ? ld_io(ds + base + col(e)) : 0.f;
        }
        float2 sum = both(0.f);
#pragma unroll
        for (int e = 0; e < 4 * NB; ++e) {
            sum.x = fmaf(s[e], s[e], sum.x);
            sum.y = fmaf(s[e] * w[e], d[e], sum.y);
        }
        sum = row_reduce2(sum, tpr, buf[k & 1]);
        const float rs = rsqrtf(sum.x / (float)q.width + q.eps);
        const float m = sum.y * rs * rs / (float)q.width;
#pragma unroll
        for (int e = 0; e < 4 * NB; ++e) {
            if (!(live && col(e) < q.width && M3_IN(36, base + col(e), ext))) continue;
            dw[e] = fmaf(d[e], s[e] * rs, dw[e]);
            st_io(static_cast<T*>(q.dx) + base + col(e), fmaf(rs, fmaf(w[e], d[e], -s[e] * m), g[e]));
        }
    }
    if (!q.dweight) return;
    for (int g = 0; g < per; ++g) {                // group by group into the CTA's sums
        if (sub == g)
#pragma unroll
            for (int e = 0; e < 4 * NB; ++e)
                if (col(e) < q.width && M3_IN(37, col(e), dyn_smem_bytes() / 4)) sums[col(e)] = g ? sums[col(e)] + dw[e] : dw[e];
        __syncthreads();
    }
    for (int c = threadIdx.x; c < q.width; c += blockDim.x)
        if (M3_IN(38, (long long)blockIdx.x * q.width + c, (long long)q.parts * q.width))
            q.part[(size_t)blockIdx.x * q.width + c] = sums[c];
}

template <typename T>
__global__ void __launch_bounds__(256) norm_bwd_any_kernel(NormParams q) {
    __shared__ float buf[16];
    const T* x = static_cast<const T*>(q.x);
    const T* dy = static_cast<const T*>(q.dy);
    const T* ds = static_cast<const T*>(q.d_sum);
    const long long ext = q.rows * q.width;
    float* part = q.part + (size_t)blockIdx.x * q.width;
    if (q.dweight)
        for (int c = threadIdx.x; c < q.width; c += 256)
            if (M3_IN(18, (long long)blockIdx.x * q.width + c, (long long)q.parts * q.width)) part[c] = 0.f;
    for (long long row = blockIdx.x; row < q.rows; row += gridDim.x) {
        const size_t base = (size_t)row * q.width;
        float ss = 0.f, dot = 0.f;
        for (int c = threadIdx.x; c < q.width; c += 256) {
            if (!M3_IN(19, base + c, ext)) continue;
            const float s = ld_io(x + base + c), w = q.weight ? q.weight[c] : 1.f;
            ss = fmaf(s, s, ss);
            dot = fmaf(s * w, ld_io(dy + base + c), dot);
        }
        ss = row_reduce<false>(ss, 256, buf);
        dot = row_reduce<false>(dot, 256, buf);
        const float rs = rsqrtf(ss / (float)q.width + q.eps);
        const float m = dot * rs * rs / (float)q.width;
        for (int c = threadIdx.x; c < q.width; c += 256) {
            if (!M3_IN(20, base + c, ext)) continue;
            const float s = ld_io(x + base + c), w = q.weight ? q.weight[c] : 1.f, d = ld_io(dy + base + c);
            if (q.dweight && M3_IN(21, (long long)blockIdx.x * q.width + c, (long long)q.parts * q.width))
                part[c] = fmaf(d, s * rs, part[c]);      // a thread's own columns
            st_io(static_cast<T*>(q.dx) + base + c, (ds ? ld_io(ds + base + c) : 0.f) + rs * fmaf(w, d, -s * m));
        }
    }
}

// dw[c] = sum of the parts: 32 columns a CTA, 32 threads a column
__global__ void __launch_bounds__(1024) norm_dw_kernel(NormParams q) {
    __shared__ float t[32][33];
    const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5, c = blockIdx.x * 32 + cx;
    float v = 0.f;
    if (c < q.width)
#pragma unroll 16
        for (int i = ry; i < q.parts; i += 32)
            if (M3_IN(22, (long long)i * q.width + c, (long long)q.parts * q.width)) v += q.part[(size_t)i * q.width + c];
    t[ry][cx] = v;
    __syncthreads();
    v = t[cx][ry];                    // column ry of the block, part cx
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    const int cc = blockIdx.x * 32 + ry;
    if (cx == 0 && cc < q.width && M3_IN(23, cc, q.width)) q.dweight[cc] = v;
}

// Threads a row and vectors a thread.  Many rows: as many vectors a thread as
// keep its loads at 64 bytes (two where two arrays are read, else four: a norm
// without residual of 32768 x 2048 takes 49 us with four, 54 with two; one with
// residual 82 with two, 86 with one).  Few rows (fewer than 256, at most two
// CTAs an SM): one vector a thread, so that a row's latency is one load's.
struct Shape {
    int tpr, nv, threads;
    long long groups;                    // CTAs that the rows fill
};
static Shape shape_of(long long rows, int width, int most_nv) {
    const int nvec = width / 8;
    const int want = rows < 256 ? 1 : most_nv;
    Shape s;
    s.tpr = 16;                          // a scale's 16 lanes in one warp
    while (s.tpr < 512 && s.tpr * want < nvec) s.tpr *= 2;
    s.nv = 1;
    while (s.tpr * s.nv < nvec) s.nv *= 2;
    s.threads = s.tpr > 128 ? s.tpr : 128;
    s.groups = (rows + s.threads / s.tpr - 1) / (s.threads / s.tpr);
    return s;
}
static bool vec_ok(int width) { return width % 8 == 0 && width <= 512 * 4 * 8; }

// Warps a row and blocks of 128 columns a warp, for widths that vec_ok leaves: as
// few warps as have at most `most` blocks each, so that CTAs are small and many
// rows are on their way; few rows: a block a warp.  Rows (256 and more) without an 8-bit
// output go to norm_any_kernel from 385 columns on.  Measured with residual and sum, us there
// and here:
//   24 M elements, bfloat16: 118 columns 317 and 78, 250 184 and 84, 380 131 and 121, 450
//     119 and 119, 515 104 and 139, 1026 66 and 139, 2340 62 and 148;
//   24 M elements, float32: 118 columns 334 and 76, 386 135 and 76, 700 88 and 76, 902 80
//     and 84, 2340 78 and 86;
//   4000 rows: 386 columns 14 and 14, 700 16 and 25 (float32 20), 1026 18 and 32 (24);
//   300 rows: 386 columns 6 and 14, 1026 7 and 12.
// (So float32 rows of 386 to 800 columns would be better off here where there are tens of
// thousands of them, up to 1.8 times, and worse where there are fewer.)  With scales a block
// of 128 columns 10256 x 2340 take 224 and 188, and the gradient 189 and 127.
struct OddShape {
    int wpr, nb, threads;
    long long groups;
};
static OddShape odd_shape_of(long long rows, int width, int most) {
    const int blocks = (width + 127) / 128;
    OddShape s;
    if (rows < 256) most = 1;
    s.wpr = 1;
    while (s.wpr < 16 && (blocks + s.wpr - 1) / s.wpr > most) s.wpr *= 2;
    s.nb = (blocks + s.wpr - 1) / s.wpr;
    s.threads = s.wpr > 4 ? 32 * s.wpr : 128;
    const int per = s.threads / (32 * s.wpr);
    s.groups = (rows + per - 1) / per;
    return s;
}
constexpr int kOddFwd = 4, kOddBwd = 4;
static bool odd_ok(int width) { return width <= 8192; }

template <typename T, int NV>
static cudaError_t fwd_nv(const NormParams& q, const Shape& s, cudaStream_t st) {
    const unsigned grid = (unsigned)s.groups;
    if (q.residual && q.y8) norm_kernel<T, NV, true, true><<<grid, s.threads, 0, st>>>(q, s.tpr);
    else if (q.residual) norm_kernel<T, NV, true, false><<<grid, s.threads, 0, st>>>(q, s.tpr);
    else if (q.y8) norm_kernel<T, NV, false, true><<<grid, s.threads, 0, st>>>(q, s.tpr);
    else norm_kernel<T, NV, false, false><<<grid, s.threads, 0, st>>>(q, s.tpr);
    return cudaGetLastError();
}

template <typename T>
static cudaError_t fwd(const NormParams& q, cudaStream_t st) {
    if (!vec_ok(q.width)) {
        if (!odd_ok(q.width) || (!q.y8 && q.rows >= 256 && q.width > 384)) {
            norm_any_kernel<T><<<(unsigned)q.rows, 256, 0, st>>>(q);
            return cudaGetLastError();
        }
        const OddShape s = odd_shape_of(q.rows, q.width, kOddFwd);
        switch (s.nb) {
            case 1: norm_odd_kernel<T, 1><<<(unsigned)s.groups, s.threads, 0, st>>>(q, s.wpr); break;
            case 2: norm_odd_kernel<T, 2><<<(unsigned)s.groups, s.threads, 0, st>>>(q, s.wpr); break;
            case 3: norm_odd_kernel<T, 3><<<(unsigned)s.groups, s.threads, 0, st>>>(q, s.wpr); break;
            default: norm_odd_kernel<T, 4><<<(unsigned)s.groups, s.threads, 0, st>>>(q, s.wpr);
        }
        return cudaGetLastError();
    }
    const Shape s = shape_of(q.rows, q.width, q.residual ? 2 : 4);
    return s.nv == 1 ? fwd_nv<T, 1>(q, s, st) : s.nv == 2 ? fwd_nv<T, 2>(q, s, st) : fwd_nv<T, 4>(q, s, st);
}

// CTAs of the gradient: as many as its 120 registers let run together, so that a
// row's loads can go ahead of the row before and few parts are left to add
// (16384 x 2048: 59 us with four an SM, 5 of them the parts' sums; 118 without loads ahead)
static unsigned bwd_grid(long long rows, int width) {
    const long long sms = device_sm_count();
    if (!vec_ok(width)) {
        if (!odd_ok(width)) return (unsigned)(rows < 4 * sms ? rows : 4 * sms);
        const OddShape s = odd_shape_of(rows, width, kOddBwd);     // (loads of one row at a time: more CTAs)
        const long long most = (s.threads <= 128 ? 8 : s.threads <= 256 ? 4 : 2) / (s.nb <= 2 ? 1 : 2) * sms;
        return (unsigned)(s.groups < most ? s.groups : most);
    }
    const Shape s = shape_of(rows, width, 2);
    const long long most = (s.threads <= 128 ? 4 : s.threads <= 256 ? 2 : 1) * sms;
    return (unsigned)(s.groups < most ? s.groups : most);
}

template <typename T, int NV>
static cudaError_t bwd_nv(const NormParams& q, const Shape& s, cudaStream_t st) {
    const int smem = q.dweight ? q.width * 4 : 0;
    if (smem > 40 * 1024) {              // (the kernel has a little static shared memory too)
        const cudaError_t e = cudaFuncSetAttribute(norm_bwd_kernel<T, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    norm_bwd_kernel<T, NV><<<bwd_grid(q.rows, q.width), s.threads, smem, st>>>(q, s.tpr);
    return cudaGetLastError();
}

template <typename T>
static cudaError_t bwd(const NormParams& q, cudaStream_t st) {
    cudaError_t e;
    if (!vec_ok(q.width) && odd_ok(q.width)) {
        const OddShape s = odd_shape_of(q.rows, q.width, kOddBwd);
        const unsigned grid = bwd_grid(q.rows, q.width);
        const int smem = q.dweight ? q.width * 4 : 0;      // (32 KB at most)
        if (s.nb == 1) norm_bwd_odd_kernel<T, 1><<<grid, s.threads, smem, st>>>(q, s.wpr);
        else if (s.nb == 2) norm_bwd_odd_kernel<T, 2><<<grid, s.threads, smem, st>>>(q, s.wpr);
        else if (s.nb == 3) norm_bwd_odd_kernel<T, 3><<<grid, s.threads, smem, st>>>(q, s.wpr);
        else norm_bwd_odd_kernel<T, 4><<<grid, s.threads, smem, st>>>(q, s.wpr);
        e = cudaGetLastError();
    } else if (!vec_ok(q.width)) {
        norm_bwd_any_kernel<T><<<bwd_grid(q.rows, q.width), 256, 0, st>>>(q);
        e = cudaGetLastError();
    } else {
        const Shape s = shape_of(q.rows, q.width, 2);
        e = s.nv == 1 ? bwd_nv<T, 1>(q, s, st) : s.nv == 2 ? bwd_nv<T, 2>(q, s, st) : bwd_nv<T, 4>(q, s, st);
    }
    if (e == cudaSuccess && q.dweight) {
        norm_dw_kernel<<<(unsigned)((q.width + 31) / 32), 1024, 0, st>>>(q);
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace norm

int norm_bwd_parts(long long rows, int width, int) {
    return rows <= 0 ? 0 : (int)norm::bwd_grid(rows, width);
}

cudaError_t launch_norm(int io_dtype, const NormParams& q, cudaStream_t st) {
    return io_dtype == M3_BF16 ? norm::fwd<__nv_bfloat16>(q, st) : norm::fwd<float>(q, st);
}

cudaError_t launch_norm_bwd(int io_dtype, const NormParams& q, cudaStream_t st) {
    return io_dtype == M3_BF16 ? norm::bwd<__nv_bfloat16>(q, st) : norm::bwd<float>(q, st);
}

}  // namespace m3

M3_BOUNDS_EXPORT(norm)
