// k_norm.cu -- root-mean-square norm of rows, with the residual's addition, an
// 8-bit output and the gradient (sm_100a).
//
//   s = x + r,  y = w s (mean s^2 + eps)^(-1/2)
//   y8 = e4m3(y / scale), scale = max|y| / 448 over the row or over 128 columns
// Gradient at the norm's input s (rs = (mean s^2 + eps)^(-1/2), s^ = s rs):
//   dx = d_sum + rs (w dy - s^ mean(w dy s^)),   dw = sum over rows of dy s^
//
// Bound by memory: every element is read and written once.  A row lives in the
// registers of TPR threads (8 consecutive elements a thread and vector, up to
// NV vectors), all its loads are issued before the reduction, and the
// reduction is shuffles (TPR <= 32) or shuffles and one exchange through shared
// memory.  Sums are float32.  A 128-column scale is the maximum over 16 lanes
// that hold one block, so 8-bit output needs no second pass.  The weight's
// gradient stays in registers over the rows that a thread group walks; the
// groups' parts are added by a second kernel in a fixed order.  Rows whose
// width is not a multiple of 8 (or too wide for registers) take scalar
// kernels that read the row twice (the second time from cache).
#include <cuda_fp8.h>

#define M3_BOUNDS_FILE 11
#include "m3_bounds.cuh"
#include "m3_common.cuh"
#include "m3_kernels.h"

namespace m3 {
namespace norm {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kE4M3Max = 448.f;
constexpr float kTiny = 1e-30f;      // floor of a scale's maximum: an all-zero block has a finite scale

template <typename T> struct Vec8;   // 8 elements as float
template <> struct Vec8<__nv_bfloat16> {
    static __device__ __forceinline__ void load(const void* base, size_t o, float* f) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + o));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
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
    static __device__ __forceinline__ void load(const void* base, size_t o, float* f) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + o);
        const float4 a = __ldcs(p), b = __ldcs(p + 1);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    static __device__ __forceinline__ void store(void* base, size_t o, const float* f) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + o);
        __stcs(p, make_float4(f[0], f[1], f[2], f[3]));
        __stcs(p + 1, make_float4(f[4], f[5], f[6], f[7]));
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
__device__ __forceinline__ float nmax(float a, float b) { return (a > b || a != a) ? a : b; }

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

template <typename T, int NV>
__global__ void __launch_bounds__(512) norm_kernel(NormParams q, int tpr) {
    __shared__ float buf[16];
    const int lane = threadIdx.x & (tpr - 1), nvec = q.width >> 3;
    const long long row = (long long)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
    const bool live = row < q.rows;
    const size_t base = live ? (size_t)row * q.width : 0;
    const long long ext = q.rows * q.width;
    float s[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (lane + tpr * i) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) s[i][j] = 0.f;
        if (live && lane + tpr * i < nvec && M3_SPAN(1, base + c, 8, ext)) Vec8<T>::load(q.x, base + c, s[i]);
    }
    if (q.residual) {
        float r[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + tpr * i) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) r[i][j] = 0.f;
            if (live && lane + tpr * i < nvec && M3_SPAN(2, base + c, 8, ext)) Vec8<T>::load(q.residual, base + c, r[i]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[i][j] += r[i][j];
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(s[i][j], s[i][j], ss);
    ss = row_reduce<false>(ss, tpr, buf);
    const float rs = rsqrtf(ss / (float)q.width + q.eps);
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (lane + tpr * i) * 8;
        const bool in = live && lane + tpr * i < nvec;
        if (in && q.sum && M3_SPAN(3, base + c, 8, ext)) Vec8<T>::store(q.sum, base + c, s[i]);
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 0.f;
        if (in && M3_SPAN(4, c, 8, q.width)) load_weight8(q.weight, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s[i][j] = in ? s[i][j] * rs * w[j] : 0.f;
            if (q.y8) top = nmax(top, fabsf(s[i][j]));
        }
        if (in && q.y && M3_SPAN(5, base + c, 8, ext)) Vec8<T>::store(q.y, base + c, s[i]);
        if (q.y8 && q.block) {          // 16 lanes hold the 128 columns of one scale
            for (int o = min(tpr, 16) >> 1; o; o >>= 1) top = nmax(top, __shfl_xor_sync(kFull, top, o));
            top = nmax(top, kTiny);
            const int nb = (q.width + 127) >> 7;
            if (in && M3_SPAN(6, base + c, 8, ext))
                *reinterpret_cast<uint2*>(q.y8 + base + c) = e4m3x8(s[i], kE4M3Max / top);
            if (in && (c & 127) == 0 && M3_IN(7, row * nb + (c >> 7), q.rows * nb)) q.scale[row * nb + (c >> 7)] = top / kE4M3Max;
            top = 0.f;
        }
    }
    if (q.y8 && !q.block) {
        top = nmax(row_reduce<true>(top, tpr, buf), kTiny);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + tpr * i) * 8;
            if (live && lane + tpr * i < nvec && M3_SPAN(8, base + c, 8, ext))
                *reinterpret_cast<uint2*>(q.y8 + base + c) = e4m3x8(s[i], kE4M3Max / top);
        }
        if (live && lane == 0 && M3_IN(9, row, q.rows)) q.scale[row] = top / kE4M3Max;
    }
}

// any width: one CTA a row, elements strided over the threads
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
    const int nb = (q.width + block - 1) / block;
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
template <typename T, int NV>
__global__ void __launch_bounds__(512) norm_bwd_kernel(NormParams q, int tpr) {
    __shared__ float buf[16];
    const int lane = threadIdx.x & (tpr - 1), nvec = q.width >> 3, per = blockDim.x / tpr;
    const int group = blockIdx.x * per + threadIdx.x / tpr, groups = gridDim.x * per;
    const long long ext = q.rows * q.width;
    float dw[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
    // all groups of a CTA take the same number of rounds (the reduction may be CTA-wide)
    const long long rounds = (q.rows + groups - 1) / groups;
    for (long long k = 0; k < rounds; ++k) {
        const long long row = k * groups + group;
        const bool live = row < q.rows;
        const size_t base = live ? (size_t)row * q.width : 0;
        float s[NV][8], d[NV][8];
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + tpr * i) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) s[i][j] = d[i][j] = 0.f;
            if (live && lane + tpr * i < nvec && M3_SPAN(14, base + c, 8, ext)) {
                Vec8<T>::load(q.x, base + c, s[i]);
                Vec8<T>::load(q.dy, base + c, d[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + tpr * i) * 8;
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 0.f;
            if (lane + tpr * i < nvec && M3_SPAN(15, c, 8, q.width)) load_weight8(q.weight, c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                ss = fmaf(s[i][j], s[i][j], ss);
                dot = fmaf(s[i][j] * w[j], d[i][j], dot);
            }
        }
        ss = row_reduce<false>(ss, tpr, buf);
        dot = row_reduce<false>(dot, tpr, buf);
        const float rs = rsqrtf(ss / (float)q.width + q.eps);
        const float m = dot * rs * rs / (float)q.width;          // mean(w dy s^) rs
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + tpr * i) * 8;
            if (!(live && lane + tpr * i < nvec && M3_SPAN(16, base + c, 8, ext))) continue;
            float w[8], e[8];
            load_weight8(q.weight, c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = 0.f;
            if (q.d_sum) Vec8<T>::load(q.d_sum, base + c, e);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dw[i][j] = fmaf(d[i][j], s[i][j] * rs, dw[i][j]);
                e[j] += rs * fmaf(w[j], d[i][j], -s[i][j] * m);
            }
            Vec8<T>::store(q.dx, base + c, e);
        }
    }
    if (q.dweight) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + tpr * i) * 8;
            if (lane + tpr * i < nvec && M3_SPAN(17, (long long)group * q.width + c, 8, (long long)q.parts * q.width)) {
                float4* p = reinterpret_cast<float4*>(q.part + (size_t)group * q.width + c);
                p[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
                p[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
            }
        }
    }
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

// Threads a row and vectors a thread.  Many rows: 4 vectors a thread keep
// enough loads in flight with few threads in the reduction; few rows (fewer
// than a CTA for every SM): one vector a thread, so that a row's latency is
// one load's.
struct Shape {
    int tpr, nv, threads;
};
static Shape shape_of(long long rows, int width, int most_nv) {
    const int nvec = width / 8;
    const int want = rows < 256 ? 1 : most_nv;
    int tpr = 8;
    while (tpr < 512 && tpr * want < nvec) tpr *= 2;
    int nv = 1;
    while (tpr * nv < nvec) nv *= 2;
    return {tpr, nv, tpr > 128 ? tpr : 128};
}
static bool vec_ok(int width) { return width % 8 == 0 && width <= 512 * 8 * 8; }

template <typename T>
static cudaError_t fwd(const NormParams& q, cudaStream_t st) {
    if (!vec_ok(q.width)) {
        norm_any_kernel<T><<<(unsigned)q.rows, 256, 0, st>>>(q);
        return cudaGetLastError();
    }
    Shape s = shape_of(q.rows, q.width, 4);
    if (q.block && s.tpr < 16) s.tpr = 16;       // a scale's 16 lanes in one warp
    const unsigned grid = (unsigned)((q.rows + s.threads / s.tpr - 1) / (s.threads / s.tpr));
    switch (s.nv) {
        case 1: norm_kernel<T, 1><<<grid, s.threads, 0, st>>>(q, s.tpr); break;
        case 2: norm_kernel<T, 2><<<grid, s.threads, 0, st>>>(q, s.tpr); break;
        case 4: norm_kernel<T, 4><<<grid, s.threads, 0, st>>>(q, s.tpr); break;
        default: norm_kernel<T, 8><<<grid, s.threads, 0, st>>>(q, s.tpr); break;
    }
    return cudaGetLastError();
}

static unsigned bwd_grid(long long rows, int width) {
    const long long most = 4LL * device_sm_count();
    if (!vec_ok(width)) return (unsigned)(rows < most ? rows : most);
    const Shape s = shape_of(rows, width, 2);
    const long long need = (rows + s.threads / s.tpr - 1) / (s.threads / s.tpr);
    return (unsigned)(need < most ? need : most);
}

template <typename T>
static cudaError_t bwd(const NormParams& q, cudaStream_t st) {
    const unsigned grid = bwd_grid(q.rows, q.width);
    if (!vec_ok(q.width)) {
        norm_bwd_any_kernel<T><<<grid, 256, 0, st>>>(q);
    } else {
        const Shape s = shape_of(q.rows, q.width, 2);
        switch (s.nv) {
            case 1: norm_bwd_kernel<T, 1><<<grid, s.threads, 0, st>>>(q, s.tpr); break;
            case 2: norm_bwd_kernel<T, 2><<<grid, s.threads, 0, st>>>(q, s.tpr); break;
            case 4: norm_bwd_kernel<T, 4><<<grid, s.threads, 0, st>>>(q, s.tpr); break;
            default: norm_bwd_kernel<T, 8><<<grid, s.threads, 0, st>>>(q, s.tpr); break;
        }
    }
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && q.dweight) {
        norm_dw_kernel<<<(unsigned)((q.width + 31) / 32), 1024, 0, st>>>(q);
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace norm

int norm_bwd_parts(long long rows, int width, int) {
    if (rows <= 0) return 0;
    const unsigned grid = norm::bwd_grid(rows, width);
    if (!norm::vec_ok(width)) return (int)grid;
    const norm::Shape s = norm::shape_of(rows, width, 2);
    return (int)grid * (s.threads / s.tpr);
}

cudaError_t launch_norm(int io_dtype, const NormParams& q, cudaStream_t st) {
    return io_dtype == M3_BF16 ? norm::fwd<__nv_bfloat16>(q, st) : norm::fwd<float>(q, st);
}

cudaError_t launch_norm_bwd(int io_dtype, const NormParams& q, cudaStream_t st) {
    return io_dtype == M3_BF16 ? norm::bwd<__nv_bfloat16>(q, st) : norm::bwd<float>(q, st);
}

}  // namespace m3

M3_BOUNDS_EXPORT(norm)
