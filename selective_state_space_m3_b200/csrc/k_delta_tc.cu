// k_delta_tc.cu -- chunked prefill of the gated delta rule on the sm_100a
// tensor cores (tcgen05 + TMEM + TMA): bfloat16 io, N = 128, P a multiple of 64.
//
// A chunk is C = 64 tokens.  With G the inclusive sum of g in the chunk,
// Gam_ij = e^{G_i - G_j} (j <= i) and S the state before the chunk:
//   A_ij = beta_i Gam_ij k_i.k_j (j < i)      T = (I + A)^{-1}
//   R = beta o (V - e^G o K S)                U = T R
//   Y = scale (e^G o Q S + (Gam o Q K^T) U)
//   S' = e^{G_C} S + K^T (e^{G_C - G} o U)
// T and the masked Q K^T do not depend on S, so they are made ahead; the chain
// of a chunk is the three products K S, T R and K^T U.
//
// One CTA per (batch, head, 64 columns) walks the chunks of its sequence:
//   warp 0       one lane issues the chain's tcgen05.mma
//   warps 1-8    the chain's arithmetic: S lives in registers in float32 (a
//                thread has one state row and 32 columns)
//   warps 9-12   up to two chunks ahead: gates, K K^T and Q K^T (one product of
//                the stacked rows [K; Q] with K), T and the masked Q K^T
//   warp 13      one lane issues the TMA loads (three chunks of K, Q, two of V)
// Every product has M = 128 rows: [K; Q] against S gives K S and Q S at once,
// and the tile [T - I; P] (P = scale Gam o Q K^T) serves both T R (upper half
// of the accumulator) and P U (lower half); the unused half is never read.
//
// Precision.  K, Q, V are bfloat16 and enter the products as they are.  The
// chain keeps float32: S, R, U and T are split into bfloat16 parts (hi + lo, 16
// to 17 bits; the state's update of S takes three parts), the products of the
// parts add up in the float32 accumulators, and the identity of T is left out
// of the product and added in registers.  Only P and the U that it meets
// are rounded to bfloat16, since y is.  T is inverted in float32 (32 x 32
// blocks by substitution, a lane per column, then -T22 (A21 T11)).
//
// Shared memory (KB): K, Q 3 x 32, V 2 x 8, S hi/lo 32 (R and U take its place
// between the first product's end and the new state), [T - I; P] 2 x 16, T lo
// 2 x 8, scratch 16.5, gates 4: one CTA an SM.
//
// Every wait on an mbarrier is bounded (1 s); on expiry the kernel records
// M3_ERR_DEVICE_TIMEOUT in the workspace status word and runs out without
// further waiting.
#define M3_BOUNDS_FILE 12
#include "m3_bounds.cuh"
#include "m3_kernels.h"
#include "tc_ptx.cuh"

namespace m3 {

bool make_tile_map(CUtensorMap* map, const void* base, int inner, int R, int grp, int L, int batch, int T);

namespace dtc {

using namespace ptx;

constexpr int kC = 64;             // tokens a chunk
constexpr int kN = 128;
constexpr int kP = 64;             // columns a CTA
constexpr int kState = 256;        // threads of the chain
constexpr int kPrep = 128;
constexpr int kThreads = 32 + kState + kPrep + 32;
constexpr int kCols = 32;          // state columns a thread
constexpr float kLog2e = 1.4426950408889634f;
constexpr unsigned kFull = 0xffffffffu;

constexpr int OFF_KQ = 0;                       // 3 x 32 KB: two 64-column atoms, rows 0..63 K, 64..127 Q
constexpr int OFF_V = OFF_KQ + 3 * 32768;       // 2 x 8 KB
constexpr int OFF_S = OFF_V + 2 * 8192;         // S hi, S lo (16 KB each: rows n, 64 p)
constexpr int OFF_UH = OFF_S;                   // R hi, then e^{G_C-G} U hi (8 KB: rows t, 64 p)
constexpr int OFF_UL = OFF_S + 8192;            // R lo, then its lo part
constexpr int OFF_UB = OFF_S + 16384;           // U rounded, for P U
constexpr int OFF_UM = OFF_S + 24576;           // third part of e^{G_C-G} U
constexpr int OFF_X = OFF_S + 32768;            // 2 x 16 KB: [T - I hi; P]
constexpr int OFF_TL = OFF_X + 2 * 16384;       // 2 x 8 KB: T - I lo (its operand reads 64 more rows, unused)
constexpr int OFF_SCR = OFF_TL + 2 * 8192;      // A11 / T11, A22 / A21 T11, A21 (4 KB each), T22 (4.5 KB)
constexpr int SCR_BYTES = 3 * 4096 + 32 * 36 * 4;
constexpr int OFF_MISC = OFF_SCR + SCR_BYTES;

struct Gates {
    float hi[kC], lo[kC];          // G in log2 units, as a sum of two floats
    float a[kC], at[kC], beta[kC]; // e^G, e^{G_C - G}, beta (0 behind the end)
    float whole;                   // e^{G_C}
    float pad[3];
};

struct Misc {
    uint64_t kq_full[3], kq_free[3], v_full[2], v_free[2], t_full[2], x_free[2];
    uint64_t s_ready, ks, r, tr, u, s, o, g, drain_a, drain_b;
    uint32_t tmem_base;
    int abort_flag, drain_flag, pad;
    Gates gates[3];
};
constexpr int SMEM_BYTES = OFF_MISC + (int)sizeof(Misc) + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory of the delta kernel");

__device__ __forceinline__ bool wait(uint64_t* b, int phase, Misc* m, int* status, int where) {
    return mbar_wait_flag(b, (uint32_t)(phase & 1), &m->abort_flag, status, where);
}
__device__ __forceinline__ void prep_sync() { asm volatile("bar.sync 2, %0;" ::"n"(kPrep) : "memory"); }
__device__ __forceinline__ float clamp_g(float g) { return g < -1.0e4f ? -1.0e4f : g; }

// 8 floats -> 8 bfloat16 (returned), f becomes what the rounding left
__device__ __forceinline__ uint4 take_bf16(float* f) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        w[j] = pack_bf16x2(f[2 * j], f[2 * j + 1]);
        f[2 * j] -= __uint_as_float(w[j] << 16);
        f[2 * j + 1] -= __uint_as_float(w[j] & 0xffff0000u);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void put16(uint8_t* smem, int off, int row, int chunk, int limit, uint4 v) {
    if (M3_SPAN(1, sw128(row, chunk), 16, limit)) *reinterpret_cast<uint4*>(smem + off + sw128(row, chunk)) = v;
}
__device__ __forceinline__ void put2(uint8_t* smem, int off, int row, int col, float v) {
    if (M3_IN(2, row * 64 + col, 4096))
        *reinterpret_cast<__nv_bfloat16*>(smem + off + sw128(row, col >> 3) + (col & 7) * 2) = __float2bfloat16_rn(v);
}

struct Where {
    int b, h, g, p0, len, nch;
};

__device__ __forceinline__ Where where_am_i(const DeltaParams& q) {
    Where w;
    const int slices = q.headdim / kP;
    const int bh = blockIdx.x / slices;
    w.p0 = (blockIdx.x % slices) * kP;
    w.b = bh / q.nheads;
    w.h = bh % q.nheads;
    w.g = w.h / (q.nheads / q.ngroups);
    int len = q.seqlen;
    if (q.lengths && M3_IN(3, w.b, q.batch)) len = min(max(q.lengths[w.b], 0), q.seqlen);
    w.len = len;
    w.nch = (len + kC - 1) / kC;
    return w;
}

// Gates of chunk c: lane l of every prep warp holds tokens 2 l and 2 l + 1; the
// sum runs in double, so that differences of G keep float32 accuracy after
// strong decay.  Warp `pw` 0 writes.
__device__ __forceinline__ void make_gates(const DeltaParams& q, const Where& w, int c, Gates* out, bool write) {
    const int lane = threadIdx.x & 31;
    float gv[2], bv[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int t = c * kC + 2 * lane + j;
        const size_t o = ((size_t)w.b * q.seqlen + t) * q.nheads + w.h;
        const bool ok = t < w.len && M3_IN(4, o, (long long)q.batch * q.seqlen * q.nheads);
        gv[j] = (ok && q.g) ? clamp_g(__ldg(q.g + o)) : 0.f;
        bv[j] = ok ? __ldg(q.beta + o) : 0.f;
    }
    const double l2e = 1.4426950408889634074;
    double d0 = gv[0] * l2e, d1 = d0 + gv[1] * l2e, sum = d1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double u = __shfl_up_sync(kFull, sum, o);
        if (lane >= o) sum += u;
    }
    const double total = __shfl_sync(kFull, sum, 31);
    const double G[2] = {sum - d1 + d0, sum};
    if (write) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int i = 2 * lane + j;
            const float hi = (float)G[j];
            out->hi[i] = hi;
            out->lo[i] = (float)(G[j] - (double)hi);
            out->a[i] = exp2f(hi);
            out->at[i] = exp2f((float)(total - G[j]));
            out->beta[i] = bv[j];
        }
        if (lane == 0) out->whole = exp2f((float)total);
    }
}

// column `lane` of the inverse of a unit lower triangular 32 x 32 matrix whose
// strict lower part is at[col * 32 + row]: x starts as the unit vector, and a
// finished x_i takes A_ri x_i off every later x_r
__device__ __forceinline__ void invert32(const float* at, float* x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = i == lane ? 1.f : 0.f;
#pragma unroll
    for (int i = 0; i < 31; ++i) {
        const float xi = -x[i];
#pragma unroll
        for (int r4 = (i + 1) / 4; r4 < 8; ++r4) {
            const float4 v = *reinterpret_cast<const float4*>(at + i * 32 + 4 * r4);
            const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (4 * r4 + j > i) x[4 * r4 + j] = fmaf(e[j], xi, x[4 * r4 + j]);
        }
    }
}

__global__ void __launch_bounds__(kThreads, 1)
    delta_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ,
                    const __grid_constant__ CUtensorMap tmV, DeltaParams q, int* status) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (su32(smem_raw) & 1023u)) & 1023u);
    Misc* m = reinterpret_cast<Misc*>(smem + OFF_MISC);
    const uint32_t sbase = su32(smem);
    if (!M3_SPAN(5, smem - smem_raw, OFF_MISC + (int)sizeof(Misc), dyn_smem_bytes())) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Where w = where_am_i(q);
    const int P = q.headdim;
    const size_t bh = (size_t)w.b * q.nheads + w.h;

    if (tid == 0) {
        for (int i = 0; i < 3; ++i) { mbar_init(&m->kq_full[i], 1); mbar_init(&m->kq_free[i], 1); }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m->v_full[i], 1);
            mbar_init(&m->v_free[i], kState / 2);
            mbar_init(&m->t_full[i], kPrep);
            mbar_init(&m->x_free[i], 1);
        }
        mbar_init(&m->s_ready, kState);
        mbar_init(&m->ks, 1);
        mbar_init(&m->r, kState / 2);
        mbar_init(&m->tr, 1);
        mbar_init(&m->u, kState);
        mbar_init(&m->s, 1);
        mbar_init(&m->o, 1);
        mbar_init(&m->g, 1);
        mbar_init(&m->drain_a, 1);
        mbar_init(&m->drain_b, 1);
        m->abort_flag = 0;
        m->drain_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
    }
    if (warp == 0) {
        tmem_alloc(&m->tmem_base, 512);
        tmem_relinquish();
    }
    // T - I is lower triangular: its upper right blocks stay zero
    for (int e = tid; e < 2 * 32 * 4; e += kThreads) {
        const int buf = e >> 7, row = (e >> 2) & 31, ch = 4 + (e & 3);
        put16(smem, OFF_X + buf * 16384, row, ch, 16384, make_uint4(0u, 0u, 0u, 0u));
        put16(smem, OFF_TL + buf * 8192, row, ch, 8192, make_uint4(0u, 0u, 0u, 0u));
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = m->tmem_base;
    const uint32_t d_ks = tmem, d_tr = tmem + 64, d_s = tmem + 128, d_o = tmem + 192, d_g = tmem + 256;

    if (warp == 0) {
        // ------------------------------------------------ the chain's products
        if (lane == 0) {
            constexpr uint32_t idKS = idesc_bf16(128, 64, 0, 1);     // A K-major, B MN-major
            constexpr uint32_t idT = idesc_bf16(128, 64, 1, 1);      // A MN-major (K^T), B MN-major
            for (int c = 0; c < w.nch; ++c) {
                const uint32_t kq = sbase + OFF_KQ + (c % 3) * 32768, x = sbase + OFF_X + (c & 1) * 16384;
                const uint32_t tl = sbase + OFF_TL + (c & 1) * 8192;
                wait(&m->kq_full[c % 3], c / 3, m, status, 1);
                // a chunk that ends behind the sequence: its K rows are cleaned by
                // the prep warps before they hand over T
                if ((c + 1) * kC > w.len) wait(&m->t_full[c & 1], c >> 1, m, status, 2);
                wait(&m->s_ready, c, m, status, 3);
                tc_fence_after();
                for (int part = 0; part < 2; ++part)
                    for (int kk = 0; kk < 8; ++kk)
                        umma(d_ks, sdesc(kq + (kk >> 2) * 16384 + (kk & 3) * 32, 16, 1024),
                             sdesc(sbase + OFF_S + part * 16384 + kk * 2048, 8192, 1024), idKS, part + kk > 0);
                umma_commit(&m->ks);
                wait(&m->t_full[c & 1], c >> 1, m, status, 4);
                wait(&m->r, c, m, status, 5);
                tc_fence_after();
                for (int part = 0; part < 3; ++part)
                    for (int kk = 0; kk < 4; ++kk)
                        umma(d_tr, sdesc((part < 2 ? x : tl) + kk * 32, 16, 1024),
                             sdesc(sbase + (part == 1 ? OFF_UL : OFF_UH) + kk * 2048, 8192, 1024), idKS, part + kk > 0);
                umma_commit(&m->tr);
                wait(&m->u, c, m, status, 6);
                tc_fence_after();
                for (int part = 0; part < 3; ++part)
                    for (int kk = 0; kk < 4; ++kk)
                        umma(d_s, sdesc(kq + kk * 2048, 16384, 1024),
                             sdesc(sbase + (part == 0 ? OFF_UH : part == 1 ? OFF_UL : OFF_UM) + kk * 2048, 8192, 1024),
                             idT, part + kk > 0);
                umma_commit(&m->s);
                for (int kk = 0; kk < 4; ++kk)
                    umma(d_o, sdesc(x + kk * 32, 16, 1024), sdesc(sbase + OFF_UB + kk * 2048, 8192, 1024), idKS, kk > 0);
                umma_commit(&m->o);
                umma_commit(&m->kq_free[c % 3]);
                umma_commit(&m->x_free[c & 1]);
            }
            umma_commit(&m->drain_a);
            mbar_wait_flag(&m->drain_a, 0, &m->drain_flag, nullptr, 0);
        }
        __syncwarp();
    } else if (warp <= 8) {
        // ---------------------------------------------- the chain's arithmetic
        const int wk = tid - 32, wg = wk >> 7, quarter = warp & 3, row = quarter * 32 + lane, c0 = wg * kCols;
        const uint32_t tl = (uint32_t)(quarter * 32) << 16;
        const bool top = row < 64;                 // holds a token's K S and U; else its Q S and y
        const int tok = row & 63;
        const long long ext_h = (long long)q.batch * q.nheads * kN * P;
        const size_t ho = (bh * kN + row) * P + w.p0 + c0;
        float S[kCols];
#pragma unroll
        for (int c4 = 0; c4 < kCols / 4; ++c4) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (q.init_h && M3_SPAN(6, ho + 4 * c4, 4, ext_h)) v = *reinterpret_cast<const float4*>(q.init_h + ho + 4 * c4);
            S[4 * c4] = v.x; S[4 * c4 + 1] = v.y; S[4 * c4 + 2] = v.z; S[4 * c4 + 3] = v.w;
        }
        auto store_state = [&]() {                 // S hi, S lo
#pragma unroll
            for (int ch = 0; ch < kCols / 8; ++ch) {
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = S[8 * ch + j];
                put16(smem, OFF_S, row, c0 / 8 + ch, 16384, take_bf16(f));
                put16(smem, OFF_S + 16384, row, c0 / 8 + ch, 16384, take_bf16(f));
            }
            fence_async_smem();
            tc_fence_before();
            mbar_arrive(&m->s_ready);
        };
        if (w.nch > 0) store_state();
        for (int c = 0; c < w.nch; ++c) {
            const Gates* gt = &m->gates[c % 3];
            float buf[kCols];                      // top: R, then U; else Q S
            if (top) {
                // this token's V, ahead of K S
                uint4 vv[kCols / 8];
                wait(&m->v_full[c & 1], c >> 1, m, status, 10);
#pragma unroll
                for (int ch = 0; ch < kCols / 8; ++ch) {
                    const uint32_t o = sw128(tok, c0 / 8 + ch);
                    vv[ch] = M3_SPAN(7, o, 16, 8192) ? *reinterpret_cast<const uint4*>(smem + OFF_V + (c & 1) * 8192 + o)
                                                     : make_uint4(0u, 0u, 0u, 0u);
                }
                wait(&m->t_full[c & 1], c >> 1, m, status, 11);
                const float be = gt->beta[tok], ba = -be * gt->a[tok];
                const bool in = c * kC + tok < w.len;
                wait(&m->ks, c, m, status, 12);
                tc_fence_after();
                tmem_ld32(d_ks + tl + c0, buf);
#pragma unroll
                for (int ch = 0; ch < kCols / 8; ++ch) {
                    const uint32_t u[4] = {vv[ch].x, vv[ch].y, vv[ch].z, vv[ch].w};
                    float f[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float v = __uint_as_float((j & 1) ? (u[j >> 1] & 0xffff0000u) : (u[j >> 1] << 16));
                        buf[8 * ch + j] = in ? fmaf(ba, buf[8 * ch + j], be * v) : 0.f;
                        f[j] = buf[8 * ch + j];
                    }
                    put16(smem, OFF_UH, tok, c0 / 8 + ch, 8192, take_bf16(f));
                    put16(smem, OFF_UL, tok, c0 / 8 + ch, 8192, take_bf16(f));
                }
                fence_async_smem();
                tc_fence_before();
                mbar_arrive(&m->r);
                // V is free only now: R, which is stored, shows that it has been read
                // (an arrival right behind the loads let the next V overtake them)
                mbar_arrive(&m->v_free[c & 1]);
                const float at = gt->at[tok];
                wait(&m->tr, c, m, status, 13);
                tc_fence_after();
                float d[kCols];
                tmem_ld32(d_tr + tl + c0, d);
#pragma unroll
                for (int ch = 0; ch < kCols / 8; ++ch) {
                    float f[8], e[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        f[j] = buf[8 * ch + j] + d[8 * ch + j];
                        e[j] = at * f[j];
                    }
                    put16(smem, OFF_UH, tok, c0 / 8 + ch, 8192, take_bf16(e));
                    put16(smem, OFF_UL, tok, c0 / 8 + ch, 8192, take_bf16(e));
                    put16(smem, OFF_UM, tok, c0 / 8 + ch, 8192, take_bf16(e));
                    put16(smem, OFF_UB, tok, c0 / 8 + ch, 8192, take_bf16(f));
                }
                fence_async_smem();
                tc_fence_before();
                mbar_arrive(&m->u);
            } else {
                wait(&m->t_full[c & 1], c >> 1, m, status, 14);
                wait(&m->ks, c, m, status, 15);
                tc_fence_after();
                tmem_ld32(d_ks + tl + c0, buf);
                const float sa = q.scale * gt->a[tok];
#pragma unroll
                for (int j = 0; j < kCols; ++j) buf[j] *= sa;
                tc_fence_before();
                mbar_arrive(&m->u);                // the previous chunk's y has been read out
            }
            const float whole = gt->whole;
            wait(&m->s, c, m, status, 16);
            tc_fence_after();
            {
                float d[kCols];
                tmem_ld32(d_s + tl + c0, d);
#pragma unroll
                for (int j = 0; j < kCols; ++j) S[j] = fmaf(whole, S[j], d[j]);
            }
            // S lo takes the place of the U that P U reads
            wait(&m->o, c, m, status, 17);
            if (c + 1 < w.nch) store_state();
            if (!top) {
                tc_fence_after();
                const size_t o = (((size_t)w.b * q.seqlen + c * kC + tok) * q.nheads + w.h) * P + w.p0 + c0;
                float d[kCols];
                tmem_ld32(d_o + tl + c0, d);
#pragma unroll
                for (int j = 0; j < kCols; ++j) buf[j] += d[j];
                if (c * kC + tok < w.len && M3_SPAN(8, o, kCols, (long long)q.batch * q.seqlen * q.nheads * P)) {
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(q.y) + o);
#pragma unroll
                    for (int ch = 0; ch < kCols / 8; ++ch) dst[ch] = pack_chunk(buf + 8 * ch);
                }
            }
        }
        if (q.final_h && M3_SPAN(9, ho, kCols, ext_h)) {
#pragma unroll
            for (int c4 = 0; c4 < kCols / 4; ++c4)
                *reinterpret_cast<float4*>(q.final_h + ho + 4 * c4) =
                    make_float4(S[4 * c4], S[4 * c4 + 1], S[4 * c4 + 2], S[4 * c4 + 3]);
        }
    } else if (warp <= 12) {
        // ------------------------------- T and the masked Q K^T of every chunk
        const int quarter = warp & 3, row = quarter * 32 + lane, pt = tid - 32 - kState;
        const uint32_t tl = (uint32_t)(quarter * 32) << 16;
        float* a11 = reinterpret_cast<float*>(smem + OFF_SCR);
        float* a22 = a11 + 1024;
        float* a21 = a22 + 1024;
        float* t22 = a21 + 1024;
        constexpr uint32_t idG = idesc_bf16(128, 64, 0, 0);
        for (int c = 0; c < w.nch; ++c) {
            const uint32_t kqo = OFF_KQ + (c % 3) * 32768;
            const int xo = OFF_X + (c & 1) * 16384, lo = OFF_TL + (c & 1) * 8192;
            const int nt = min(kC, w.len - c * kC);
            Gates* gt = &m->gates[c % 3];
            wait(&m->kq_full[c % 3], c / 3, m, status, 20);
            // K rows behind the sequence's end (other data, possibly not numbers)
            // must be zeros: K^T U sums over all rows of the tile
            for (int e = pt; e < (kC - nt) * 16; e += kPrep) {
                const int r = nt + (e >> 4), ch = e & 15;
                put16(smem, kqo + (ch >> 3) * 16384, r, ch & 7, 16384, make_uint4(0u, 0u, 0u, 0u));
            }
            if (nt < kC) fence_async_smem();
            // this chunk's tiles and gates take the places of chunk c - 2's and c - 3's
            if (c >= 2) wait(&m->x_free[c & 1], (c >> 1) - 1, m, status, 21);
            make_gates(q, w, c, gt, warp == 9);
            tc_fence_before();
            prep_sync();
            if (pt == 0) {
                tc_fence_after();
                for (int kk = 0; kk < 8; ++kk) {
                    const uint32_t o = sbase + kqo + (kk >> 2) * 16384 + (kk & 3) * 32;
                    umma(d_g, sdesc(o, 16, 1024), sdesc(o, 16, 1024), idG, kk > 0);
                }
                umma_commit(&m->g);
            }
            __syncwarp();
            wait(&m->g, c, m, status, 22);
            tc_fence_after();
            const int tok = row & 63;
            const float gh = gt->hi[tok], gl = gt->lo[tok];
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                if (half * 32 > (tok | 31)) {      // columns behind every row of this warp
                    if (row >= 64)
#pragma unroll
                        for (int ch = 0; ch < 4; ++ch) put16(smem, xo, row, 4 + ch, 16384, make_uint4(0u, 0u, 0u, 0u));
                    continue;
                }
                float d[32];
                tmem_ld32(d_g + tl + half * 32, d);
                const float f = row < 64 ? gt->beta[tok] : q.scale;
                const int last = row < 64 ? tok - 1 : tok;
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const int col = half * 32 + j;
                    const float e = exp2f((gh - gt->hi[col]) + (gl - gt->lo[col]));
                    d[j] = col <= last ? f * e * d[j] : 0.f;
                }
                if (row < 64) {
                    float* dst = half ? a22 : (quarter == 0 ? a11 : a21);
#pragma unroll
                    for (int j = 0; j < 32; ++j) dst[j * 32 + lane] = d[j];
                } else {
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch) put16(smem, xo, row, half * 4 + ch, 16384, pack_chunk(d + 8 * ch));
                }
            }
            tc_fence_before();
            prep_sync();
            if (row < 64) {
                float x[32];
                invert32(quarter == 0 ? a11 : a22, x);
                __syncwarp();
                // T11 by rows for A21 T11; T22 by columns, padded, for T22 (A21 T11)
                if (quarter == 0) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) a11[i * 32 + lane] = x[i];
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<float4*>(t22 + lane * 36 + 4 * i) =
                            make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                }
                const int r0 = quarter * 32;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float v = i > lane ? x[i] : 0.f;
                    put2(smem, xo, r0 + i, r0 + lane, v);
                    put2(smem, lo, r0 + i, r0 + lane, v - __bfloat162float(__float2bfloat16_rn(v)));
                }
            }
            prep_sync();
            {
                const int r0 = quarter * 8;
                float acc[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = 0.f;
#pragma unroll 8
                for (int k = 0; k < 32; ++k) {
                    const float t = a11[k * 32 + lane];
                    const float4 u = *reinterpret_cast<const float4*>(a21 + k * 32 + r0);
                    const float4 v = *reinterpret_cast<const float4*>(a21 + k * 32 + r0 + 4);
                    acc[0] = fmaf(u.x, t, acc[0]); acc[1] = fmaf(u.y, t, acc[1]);
                    acc[2] = fmaf(u.z, t, acc[2]); acc[3] = fmaf(u.w, t, acc[3]);
                    acc[4] = fmaf(v.x, t, acc[4]); acc[5] = fmaf(v.y, t, acc[5]);
                    acc[6] = fmaf(v.z, t, acc[6]); acc[7] = fmaf(v.w, t, acc[7]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) a22[(r0 + i) * 32 + lane] = acc[i];
                prep_sync();
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = 0.f;
#pragma unroll 8
                for (int k = 0; k < 32; ++k) {
                    const float t = -a22[k * 32 + lane];
                    const float4 u = *reinterpret_cast<const float4*>(t22 + k * 36 + r0);
                    const float4 v = *reinterpret_cast<const float4*>(t22 + k * 36 + r0 + 4);
                    acc[0] = fmaf(u.x, t, acc[0]); acc[1] = fmaf(u.y, t, acc[1]);
                    acc[2] = fmaf(u.z, t, acc[2]); acc[3] = fmaf(u.w, t, acc[3]);
                    acc[4] = fmaf(v.x, t, acc[4]); acc[5] = fmaf(v.y, t, acc[5]);
                    acc[6] = fmaf(v.z, t, acc[6]); acc[7] = fmaf(v.w, t, acc[7]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    put2(smem, xo, 32 + r0 + i, lane, acc[i]);
                    put2(smem, lo, 32 + r0 + i, lane, acc[i] - __bfloat162float(__float2bfloat16_rn(acc[i])));
                }
            }
            fence_async_smem();
            mbar_arrive(&m->t_full[c & 1]);
        }
        if (pt == 0) {
            umma_commit(&m->drain_b);
            mbar_wait_flag(&m->drain_b, 0, &m->drain_flag, nullptr, 0);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------- loads
        if (lane == 0) {
            for (int c = 0; c < w.nch; ++c) {
                const uint32_t kq = sbase + OFF_KQ + (c % 3) * 32768;
                if (c >= 3) wait(&m->kq_free[c % 3], c / 3 - 1, m, status, 30);
                uint64_t* bar = &m->kq_full[c % 3];
                mbar_expect_tx(bar, 32768);
                tma_load_5d(kq, &tmK, bar, 0, 0, w.g, c * kC, w.b);
                tma_load_5d(kq + 16384, &tmK, bar, 64, 0, w.g, c * kC, w.b);
                tma_load_5d(kq + 8192, &tmQ, bar, 0, 0, w.g, c * kC, w.b);
                tma_load_5d(kq + 24576, &tmQ, bar, 64, 0, w.g, c * kC, w.b);
                if (c >= 2) wait(&m->v_free[c & 1], (c >> 1) - 1, m, status, 31);
                bar = &m->v_full[c & 1];
                mbar_expect_tx(bar, 8192);
                tma_load_5d(sbase + OFF_V + (c & 1) * 8192, &tmV, bar, w.p0, 0, w.h, c * kC, w.b);
            }
            // nothing may still be on its way into shared memory when the CTA ends
            for (int c = max(0, w.nch - 3); c < w.nch; ++c) {
                mbar_wait_flag(&m->kq_full[c % 3], (c / 3) & 1, &m->drain_flag, nullptr, 0);
                if (c >= w.nch - 2) mbar_wait_flag(&m->v_full[c & 1], (c >> 1) & 1, &m->drain_flag, nullptr, 0);
            }
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

}  // namespace dtc

bool delta_tc_eligible(const m3_dims& d) {
    return d.io_dtype == M3_BF16 && d.dstate == dtc::kN && d.headdim % dtc::kP == 0;
}

cudaError_t launch_delta_tc(const m3_dims& d, const DeltaParams& q, int* status, cudaStream_t st) {
    using namespace dtc;
    CUtensorMap mK, mQ, mV;
    if (!make_tile_map(&mK, q.k, kN, 1, d.ngroups, d.seqlen, d.batch, kC) ||
        !make_tile_map(&mQ, q.q, kN, 1, d.ngroups, d.seqlen, d.batch, kC) ||
        !make_tile_map(&mV, q.v, d.headdim, 1, d.nheads, d.seqlen, d.batch, kC))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(delta_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((long long)d.batch * d.nheads * (d.headdim / kP));
    delta_tc_kernel<<<grid, kThreads, SMEM_BYTES, st>>>(mK, mQ, mV, q, status);
    return cudaGetLastError();
}

}  // namespace m3

M3_BOUNDS_EXPORT(delta_tc)
