// k_delta.cu -- the gated delta rule, token by token (sm_100a): prefill and
// gradient for every supported shape and io type, and the decode step.
//
// Per batch b and head h (a_t = e^{g_t}):
//   u_t = beta_t (v_t - a_t S_{t-1}^T k_t)
//   S_t = a_t S_{t-1} + k_t u_t^T                       S in R^{N x P}
//   y_t = scale S_t^T q_t = scale (a_t S_{t-1}^T q_t + (k_t . q_t) u_t)
// The second form of y lets one pass over the state make both products with
// S_{t-1} before the update, so a token costs one reduction, not two.
//
// The columns of S never mix, so a CTA owns 16 of them; lane 16 c + j of a
// warp holds rows j, j + 16, ... of column c (two columns a warp).  A product
// with S is NR multiply-adds a thread and four shuffles.  Everything is
// float32.  The prefill brings a block of 16 tokens in through registers while the
// block before it is worked on.  The chain over tokens bounds it: 333 tokens of
// N = 40 take 64 us, 190 ns a token (99 us with the loads in the chain).
//
// Gradient, from the last token to the first, with dS the gradient of S_t:
//   dS  += q (scale dy)^T            dq = S_t (scale dy)
//   du   = dS^T k                    de = beta du = dv      dbeta = du . e
//   dk   = dS u - a S_{t-1} de       (e_t = v_t - a_t S_{t-1}^T k_t, u = beta e)
//   dS'  = dS - k de^T               dg = a <dS', S_{t-1}>  dS <- a dS'
// States are recomputed forwards in blocks of KB tokens from checkpoints that
// the prefill wrote, and kept in shared memory for the block.  dq, dk, dg and
// dbeta are sums over columns (and, for a shared group, over heads): each CTA
// writes its part, and a second kernel adds the parts in a fixed order, so
// that the result does not depend on the order in which CTAs run.
#define M3_BOUNDS_FILE 10
#include "m3_bounds.cuh"
#include "m3_common.cuh"
#include "m3_delta.h"
#include "m3_kernels.h"

namespace m3 {
namespace delta {

constexpr int kCols = 16;          // columns of S a CTA owns
constexpr int kThreads = 256;      // 8 warps x 2 columns
constexpr int kRG = 16;            // row groups (lanes that share a column)
constexpr int kTB = 16;            // tokens staged at a time
constexpr unsigned kFull = 0xffffffffu;

// log decays below this give e^g = 0 in float32; the clamp keeps -inf (a full
// reset of the state) out of differences of sums
__device__ __forceinline__ float clamp_g(float g) { return g < -1.0e4f ? -1.0e4f : g; }

__device__ __forceinline__ int seq_len(const DeltaParams& q, int b) {
    if (!q.lengths) return q.seqlen;
    const int n = M3_IN(1, b, q.batch) ? q.lengths[b] : 0;
    return min(max(n, 0), q.seqlen);
}

template <int W>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = W / 2; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// shared memory of a block of up to kTB staged tokens
struct Stage {
    float* k;      // [kTB][N]
    float* q;      // [kTB][N]
    float* v;      // [kTB][kCols]
    float* o;      // [kTB][kCols]: y (prefill), dy (gradient)
    float* a;      // [kTB] e^g
    float* beta;   // [kTB]
    float* kq;     // [kTB] k . q (prefill)
};
__device__ __forceinline__ Stage stage_at(float* p, int N) {
    Stage s;
    s.k = p;
    s.q = s.k + kTB * N;
    s.v = s.q + kTB * N;
    s.o = s.v + kTB * kCols;
    s.a = s.o + kTB * kCols;
    s.beta = s.a + kTB;
    s.kq = s.beta + kTB;
    return s;
}
__host__ __device__ constexpr int stage_floats(int N) { return kTB * (2 * N + 2 * kCols + 3); }

template <typename T>
__device__ __forceinline__ void stage_load(const DeltaParams& q, const Stage& s, int b, int h, int g, int p0, int t0,
                                           int nt, const T* dy) {
    const int N = q.dstate, P = q.headdim, tid = threadIdx.x;
    const T* kg = static_cast<const T*>(q.k);
    const T* qg = static_cast<const T*>(q.q);
    const T* vg = static_cast<const T*>(q.v);
    const long long ext_k = (long long)q.batch * q.seqlen * q.ngroups * N;
    const long long ext_v = (long long)q.batch * q.seqlen * q.nheads * P;
    for (int e = tid; e < nt * N; e += kThreads) {
        const int t = e / N, n = e - t * N;
        const size_t o = (((size_t)b * q.seqlen + t0 + t) * q.ngroups + g) * N + n;
        const bool ok = M3_IN(2, o, ext_k);
        s.k[e] = ok ? ld_io(kg + o) : 0.f;
        s.q[e] = ok ? ld_io(qg + o) : 0.f;
    }
    for (int e = tid; e < nt * kCols; e += kThreads) {
        const int t = e / kCols, c = e - t * kCols;
        const size_t o = (((size_t)b * q.seqlen + t0 + t) * q.nheads + h) * P + p0 + c;
        const bool ok = p0 + c < P && M3_IN(3, o, ext_v);
        s.v[e] = ok ? ld_io(vg + o) : 0.f;
        if (dy) s.o[e] = ok ? q.scale * ld_io(dy + o) : 0.f;
    }
    if (tid < nt) {
        const size_t o = ((size_t)b * q.seqlen + t0 + tid) * q.nheads + h;
        const bool ok = M3_IN(4, o, (long long)q.batch * q.seqlen * q.nheads);
        s.a[tid] = q.g ? expf(clamp_g(ok ? q.g[o] : 0.f)) : 1.f;
        s.beta[tid] = ok ? q.beta[o] : 0.f;
    }
}

template <typename T, int NR>
__global__ void __launch_bounds__(kThreads) delta_seq_kernel(DeltaParams q) {
    extern __shared__ float smem[];
    const int N = q.dstate, P = q.headdim, tid = threadIdx.x;
    const int tiles = (P + kCols - 1) / kCols;
    const int bh = blockIdx.x / tiles, p0 = (blockIdx.x % tiles) * kCols;
    const int b = bh / q.nheads, h = bh % q.nheads, g = h / (q.nheads / q.ngroups);
    const int rg = tid & 15, c = tid >> 4, p = p0 + c;
    const int len = seq_len(q, b);
    const long long ext_h = (long long)q.batch * q.nheads * N * P;
    const long long ext_v = (long long)q.batch * q.seqlen * q.nheads * P;
    const size_t hb = (size_t)bh * N * P;
    const Stage s = stage_at(smem, N);
    if (!M3_SPAN(5, 0, stage_floats(N) * 4, dyn_smem_bytes())) return;

    float S[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int n = rg + kRG * i;
        S[i] = 0.f;
        if (q.init_h && n < N && p < P && M3_IN(6, hb + (size_t)n * P + p, ext_h)) S[i] = q.init_h[hb + (size_t)n * P + p];
    }
    T* yg = static_cast<T*>(q.y);
    const T* kg = static_cast<const T*>(q.k);
    const T* qg = static_cast<const T*>(q.q);
    const T* vg = static_cast<const T*>(q.v);
    [[maybe_unused]] const long long ext_k = (long long)q.batch * q.seqlen * q.ngroups * N;
    [[maybe_unused]] const long long toks = (long long)q.batch * q.seqlen * q.nheads;
    // a block's operands come through registers, asked for before the previous
    // block is worked on: thread 16 t + j has rows j, j + 16, ... of token t
    static_assert(kThreads == kTB * kRG && kCols == kRG);
    const int tt = tid >> 4;
    float fk[NR], fq[NR], fv = 0.f, fg = 0.f, fb = 0.f;
    auto fetch = [&](int t0) {
        const bool in = t0 + tt < len;
        const size_t row = (size_t)b * q.seqlen + t0 + tt;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int n = rg + kRG * i;
            const size_t o = (row * q.ngroups + g) * N + n;
            const bool ok = in && n < N && M3_IN(2, o, ext_k);
            fk[i] = ok ? ld_io(kg + o) : 0.f;
            fq[i] = ok ? ld_io(qg + o) : 0.f;
        }
        const size_t o = row * q.nheads + h;
        fv = in && p0 + rg < P && M3_IN(3, o * P + p0 + rg, ext_v) ? ld_io(vg + o * P + p0 + rg) : 0.f;
        if (rg == 0) {
            const bool ok = in && M3_IN(4, o, toks);
            fg = q.g && ok ? q.g[o] : 0.f;
            fb = ok ? q.beta[o] : 0.f;
        }
    };
    fetch(0);
    for (int t0 = 0; t0 < len; t0 += kTB) {
        const int nt = min(kTB, len - t0);
        if (q.ckpt && t0 % q.KB == 0 && p < P) {
            float* ck = q.ckpt + ((size_t)bh * q.nck + t0 / q.KB) * N * P;
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int n = rg + kRG * i;
                if (n < N && M3_IN(7, ((size_t)bh * q.nck + t0 / q.KB) * N * P + (size_t)n * P + p,
                                   (long long)q.batch * q.nheads * q.nck * N * P))
                    ck[(size_t)n * P + p] = S[i];
            }
        }
        float kq = 0.f;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int n = rg + kRG * i;
            if (n < N) {
                s.k[tt * N + n] = fk[i];
                s.q[tt * N + n] = fq[i];
            }
            kq = fmaf(fk[i], fq[i], kq);
        }
        s.v[tt * kCols + rg] = fv;
        kq = group_sum<16>(kq);
        if (rg == 0) {
            s.kq[tt] = kq;
            s.a[tt] = q.g ? expf(clamp_g(fg)) : 1.f;
            s.beta[tt] = fb;
        }
        __syncthreads();
        if (t0 + kTB < len) fetch(t0 + kTB);
        float kr[NR], qr[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int n = rg + kRG * i;
            kr[i] = n < N ? s.k[n] : 0.f;
            qr[i] = n < N ? s.q[n] : 0.f;
        }
        for (int t = 0; t < nt; ++t) {
            if (q.ckpt && t > 0 && (t0 + t) % q.KB == 0 && p < P) {
                float* ck = q.ckpt + ((size_t)bh * q.nck + (t0 + t) / q.KB) * N * P;
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    const int n = rg + kRG * i;
                    if (n < N && M3_IN(8, ((size_t)bh * q.nck + (t0 + t) / q.KB) * N * P + (size_t)n * P + p,
                                       (long long)q.batch * q.nheads * q.nck * N * P))
                        ck[(size_t)n * P + p] = S[i];
                }
            }
            float sk = 0.f, sq = 0.f;
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                sk = fmaf(S[i], kr[i], sk);
                sq = fmaf(S[i], qr[i], sq);
            }
            // the next token's k and q, while the sums go round
            const int tn = min(t + 1, nt - 1);
            float kn[NR], qn[NR];
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int n = rg + kRG * i;
                kn[i] = n < N ? s.k[tn * N + n] : 0.f;
                qn[i] = n < N ? s.q[tn * N + n] : 0.f;
            }
            const float a = s.a[t], beta = s.beta[t], v = s.v[t * kCols + c], kq = s.kq[t];
            sk = group_sum<16>(sk);
            const float u = beta * fmaf(-a, sk, v);
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                S[i] = fmaf(kr[i], u, a * S[i]);
                kr[i] = kn[i];
                qr[i] = qn[i];
            }
            sq = group_sum<16>(sq);
            if (rg == 0) s.o[t * kCols + c] = q.scale * fmaf(kq, u, a * sq);
        }
        __syncthreads();
        if (yg && tt < nt && p0 + rg < P) {
            const size_t o = (((size_t)b * q.seqlen + t0 + tt) * q.nheads + h) * P + p0 + rg;
            if (M3_IN(9, o, ext_v)) st_io(yg + o, s.o[tt * kCols + rg]);
        }
    }
    if (q.final_h) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int n = rg + kRG * i;
            if (n < N && p < P && M3_IN(10, hb + (size_t)n * P + p, ext_h)) q.final_h[hb + (size_t)n * P + p] = S[i];
        }
    }
}

// ---------------------------------------------------------------- gradient --
// shared memory: stage, states before each token of the block [KB][NR][256]
// (thread-private order), u and e [KB][kCols], and the cross-warp sums of
// dq, dk [2 parities][8 warps][2][N] and of dg, dbeta [2][8][2]
constexpr int grad_floats(int N, int NR, int KB) {
    return stage_floats(N) + KB * NR * kThreads + 2 * KB * kCols + 2 * 8 * 2 * N + 2 * 8 * 2;
}

template <typename T, int NR>
__global__ void __launch_bounds__(kThreads) delta_seq_bwd_kernel(DeltaParams q) {
    extern __shared__ float smem[];
    const int N = q.dstate, P = q.headdim, tid = threadIdx.x, KB = q.KB;
    const int tiles = (P + kCols - 1) / kCols, tile = blockIdx.x % tiles;
    const int bh = blockIdx.x / tiles, p0 = tile * kCols;
    const int b = bh / q.nheads, h = bh % q.nheads, g = h / (q.nheads / q.ngroups);
    const int rg = tid & 15, c = tid >> 4, p = p0 + c, warp = tid >> 5, lane = tid & 31;
    const int len = seq_len(q, b);
    const long long ext_h = (long long)q.batch * q.nheads * N * P;
    const long long ext_v = (long long)q.batch * q.seqlen * q.nheads * P;
    const long long toks = (long long)q.batch * q.seqlen * q.nheads;
    const size_t hb = (size_t)bh * N * P;
    const Stage s = stage_at(smem, N);
    float* sS = smem + stage_floats(N);
    float* sU = sS + KB * NR * kThreads;
    float* sE = sU + KB * kCols;
    float* red = sE + KB * kCols;
    float* red2 = red + 2 * 8 * 2 * N;
    if (!M3_SPAN(11, 0, grad_floats(N, NR, KB) * 4, dyn_smem_bytes())) return;

    float dS[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int n = rg + kRG * i;
        dS[i] = 0.f;
        if (q.d_final_h && n < N && p < P && M3_IN(12, hb + (size_t)n * P + p, ext_h))
            dS[i] = q.d_final_h[hb + (size_t)n * P + p];
    }
    T* dvg = static_cast<T*>(q.dv);
    // tokens behind the end of the sequence have no gradient
    for (size_t e = (size_t)len * kCols + tid; e < (size_t)q.seqlen * kCols; e += kThreads) {
        const size_t t = e / kCols;
        const int cc = (int)(e - t * kCols);
        const size_t o = (((size_t)b * q.seqlen + t) * q.nheads + h) * P + p0 + cc;
        if (p0 + cc < P && M3_IN(13, o, ext_v)) st_io(dvg + o, 0.f);
    }
    const int nb = (len + KB - 1) / KB;
    int par = 0;
    for (int blk = nb - 1; blk >= 0; --blk) {
        const int t0 = blk * KB, nt = min(KB, len - t0);
        __syncthreads();
        stage_load<T>(q, s, b, h, g, p0, t0, nt, static_cast<const T*>(q.dy));
        float S[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int n = rg + kRG * i;
            S[i] = 0.f;
            const size_t o = ((size_t)bh * q.nck + blk) * N * P + (size_t)n * P + p;
            if (n < N && p < P && M3_IN(14, o, (long long)q.batch * q.nheads * q.nck * N * P)) S[i] = q.ckpt[o];
        }
        __syncthreads();
        for (int t = 0; t < nt; ++t) {       // states before each token of the block
            float sk = 0.f;
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int n = rg + kRG * i;
                sS[(t * NR + i) * kThreads + tid] = S[i];
                sk = fmaf(S[i], n < N ? s.k[t * N + n] : 0.f, sk);
            }
            sk = group_sum<16>(sk);
            const float a = s.a[t], e = fmaf(-a, sk, s.v[t * kCols + c]), u = s.beta[t] * e;
            if (rg == 0) {
                sU[t * kCols + c] = u;
                sE[t * kCols + c] = e;
            }
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int n = rg + kRG * i;
                S[i] = fmaf(n < N ? s.k[t * N + n] : 0.f, u, a * S[i]);
            }
        }
        __syncthreads();
        for (int t = nt - 1; t >= 0; --t) {
            const float a = s.a[t], u = sU[t * kCols + c], e = sE[t * kCols + c], dov = s.o[t * kCols + c];
            float du = 0.f;
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int n = rg + kRG * i;
                if (n < N) dS[i] = fmaf(s.q[t * N + n], dov, dS[i]);
                du = fmaf(dS[i], n < N ? s.k[t * N + n] : 0.f, du);
            }
            du = group_sum<16>(du);
            const float de = s.beta[t] * du;
            float dg = 0.f;
            float* r = red + (size_t)par * 8 * 2 * N + (size_t)warp * 2 * N;
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int n = rg + kRG * i;
                const float kv = n < N ? s.k[t * N + n] : 0.f;
                const float old = a * sS[(t * NR + i) * kThreads + tid];
                float dq = fmaf(kv, u, old) * dov, dk = fmaf(dS[i], u, -old * de);
                dq += __shfl_xor_sync(kFull, dq, 16);
                dk += __shfl_xor_sync(kFull, dk, 16);
                if (lane < 16 && n < N) {
                    r[n] = dq;
                    r[N + n] = dk;
                }
                const float dn = fmaf(-kv, de, dS[i]);
                dg = fmaf(dn, old, dg);
                dS[i] = a * dn;
            }
            dg = group_sum<32>(dg);
            float db = lane % 16 == 0 ? du * e : 0.f;
            db = group_sum<32>(db);
            if (lane == 0) {
                red2[(par * 8 + warp) * 2] = dg;
                red2[(par * 8 + warp) * 2 + 1] = db;
            }
            if (rg == 0 && p < P) {
                const size_t o = (((size_t)b * q.seqlen + t0 + t) * q.nheads + h) * P + p;
                if (M3_IN(15, o, ext_v)) st_io(dvg + o, de);
            }
            __syncthreads();
            // this CTA's part of the token's sums; the other parity is
            // written meanwhile, and the next barrier keeps it apart
            const size_t tok = ((size_t)b * q.seqlen + t0 + t) * q.nheads + h;
            for (int e2 = tid; e2 < 2 * N; e2 += kThreads) {
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < 8; ++w) v += red[(size_t)par * 8 * 2 * N + (size_t)w * 2 * N + e2];
                const size_t o = ((size_t)tile * toks + tok) * 2 * N + e2;
                if (M3_IN(16, o, (long long)tiles * toks * 2 * N)) q.part_qk[o] = v;
            }
            if (tid < 2) {
                float v = 0.f;
                for (int w = 0; w < 8; ++w) v += red2[(par * 8 + w) * 2 + tid];
                const size_t o = ((size_t)tile * toks + tok) * 2 + tid;
                if (M3_IN(17, o, (long long)tiles * toks * 2)) q.part_g[o] = v;
            }
            par ^= 1;
        }
    }
    if (q.d_init_h) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int n = rg + kRG * i;
            if (n < N && p < P && M3_IN(18, hb + (size_t)n * P + p, ext_h)) q.d_init_h[hb + (size_t)n * P + p] = dS[i];
        }
    }
}

// dq, dk [b][t][g][n] = sum over the heads of the group and the column tiles;
// dg, dbeta [b][t][h] = sum over the tiles; zero behind a sequence's end
template <typename T>
__global__ void __launch_bounds__(kThreads) delta_reduce_kernel(DeltaParams q, int tiles) {
    const int N = q.dstate, hpg = q.nheads / q.ngroups;
    const long long toks = (long long)q.batch * q.seqlen * q.nheads;
    const size_t row = blockIdx.x;                        // (b, t, g)
    const int g = (int)(row % q.ngroups);
    const size_t bt = row / q.ngroups;
    const int b = (int)(bt / q.seqlen), t = (int)(bt % q.seqlen);
    const bool live = t < seq_len(q, b);
    for (int e = threadIdx.x; e < 2 * N; e += kThreads) {
        float v = 0.f;
        if (live)
            for (int hh = 0; hh < hpg; ++hh)
                for (int tile = 0; tile < tiles; ++tile) {
                    const size_t o = ((size_t)tile * toks + bt * q.nheads + g * hpg + hh) * 2 * N + e;
                    if (M3_IN(19, o, (long long)tiles * toks * 2 * N)) v += q.part_qk[o];
                }
        const size_t o = row * N + (e < N ? e : e - N);
        if (M3_IN(20, o, (long long)q.batch * q.seqlen * q.ngroups * N))
            st_io((e < N ? static_cast<T*>(q.dq) : static_cast<T*>(q.dk)) + o, v);
    }
    for (int e = threadIdx.x; e < 2 * hpg; e += kThreads) {
        const int hh = e >> 1;
        float v = 0.f;
        if (live)
            for (int tile = 0; tile < tiles; ++tile) {
                const size_t o = ((size_t)tile * toks + bt * q.nheads + g * hpg + hh) * 2 + (e & 1);
                if (M3_IN(21, o, (long long)tiles * toks * 2)) v += q.part_g[o];
            }
        T* dst = static_cast<T*>((e & 1) ? q.dbeta : q.dg);
        if (dst && M3_IN(22, bt * q.nheads + g * hpg + hh, toks)) st_io(dst + bt * q.nheads + g * hpg + hh, v);
    }
}

// -------------------------------------------------------------- one token --
// One CTA per (b, h).  The state comes into shared memory by asynchronous copies
// of 16 bytes, all issued before anything else; row group rg of a thread copies
// and uses rows rg, rg + RG, ... at four columns, so no thread waits for
// another's.  Bound by the state's traffic (8 bytes an element, 99 % of all bytes
// for N = 128, P = 64): 256 sequences of 32 heads, 0.54 GB, take 104 us, 5.2 TB/s.
// Five CTAs an SM.  The state in registers instead: 107 us with three or four
// CTAs, 132 with five, which leave too few registers for all loads at once; two
// CTAs that stay and ask for the next state before they work on the present one
// take 120 us.
__host__ __device__ constexpr int step_floats(int N, int P, int NPT) { return NPT * 1024 + 2 * N + P + 16 * P; }

template <typename T, int NPT>
__global__ void __launch_bounds__(256, NPT <= 8 ? 5 : 2) delta_step_kernel(DeltaParams q) {
    extern __shared__ __align__(16) float step_smem[];
    __shared__ float skq[8];
    const int N = q.dstate, P = q.headdim, tid = threadIdx.x;
    if (!M3_SPAN(29, 0, step_floats(N, P, NPT) * 4, dyn_smem_bytes())) return;
    float4* st = reinterpret_cast<float4*>(step_smem);         // [NPT][256]
    float* sk = step_smem + NPT * 1024;
    float* sq = sk + N;
    float* sv = sq + N;
    float* red = sv + P;                                       // [8][2][P]
    const int PC = P >> 2, RG = 256 / PC;
    const int pc = tid % PC, rg = tid / PC;
    const int bh = blockIdx.x, b = bh / q.nheads, h = bh % q.nheads, g = h / (q.nheads / q.ngroups);
    const long long ext_h = (long long)q.batch * q.nheads * N * P;
    const size_t hb = (size_t)bh * N * P;
    const float4* src = reinterpret_cast<const float4*>(q.init_h + hb);
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
        const int n = rg + RG * i;
        if (n < N && M3_SPAN(23, hb + (size_t)n * P + 4 * pc, 4, ext_h))
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                         ::"r"((uint32_t)__cvta_generic_to_shared(st + i * 256 + tid)), "l"(src + (size_t)n * PC + pc)
                         : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    const size_t ko = ((size_t)b * q.ngroups + g) * N;
    float kq = 0.f;
    if (tid < N && M3_IN(24, ko + tid, (long long)q.batch * q.ngroups * N)) {
        const float kv = ld_io(static_cast<const T*>(q.k) + ko + tid), qv = ld_io(static_cast<const T*>(q.q) + ko + tid);
        sk[tid] = kv;
        sq[tid] = qv;
        kq = kv * qv;
    }
    if (tid < P && M3_IN(25, (size_t)bh * P + tid, (long long)q.batch * q.nheads * P))
        sv[tid] = ld_io(static_cast<const T*>(q.v) + (size_t)bh * P + tid);
    kq = group_sum<32>(kq);
    if ((tid & 31) == 0) skq[tid >> 5] = kq;
    const bool okt = M3_IN(26, bh, (long long)q.batch * q.nheads);
    const float a = q.g && okt ? expf(clamp_g(q.g[bh])) : 1.f, beta = okt ? q.beta[bh] : 0.f;
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    float rk[4] = {0.f, 0.f, 0.f, 0.f}, rq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
        const int n = rg + RG * i;
        if (n >= N) continue;
        const float kv = sk[n], qv = sq[n];
        const float4 S = st[i * 256 + tid];
        rk[0] = fmaf(S.x, kv, rk[0]); rk[1] = fmaf(S.y, kv, rk[1]);
        rk[2] = fmaf(S.z, kv, rk[2]); rk[3] = fmaf(S.w, kv, rk[3]);
        rq[0] = fmaf(S.x, qv, rq[0]); rq[1] = fmaf(S.y, qv, rq[1]);
        rq[2] = fmaf(S.z, qv, rq[2]); rq[3] = fmaf(S.w, qv, rq[3]);
    }
    // over the row groups: lanes of a warp that share a column group (PC < 32),
    // then the warps; a column's value is the sum of the warps that hold it
    for (int o = PC; o < 32; o <<= 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            rk[j] += __shfl_xor_sync(kFull, rk[j], o);
            rq[j] += __shfl_xor_sync(kFull, rq[j], o);
        }
    }
    const int warp = tid >> 5, lane = tid & 31;
    // warps that hold column group pc: all of them if PC <= 32, else those with
    // the same part of the columns; slot = the warp's number among them
    const int parts = PC > 32 ? PC >> 5 : 1, slots = 8 / parts, slot = warp / parts;
    if (lane < PC) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            red[(2 * slot) * P + 4 * pc + j] = rk[j];
            red[(2 * slot + 1) * P + 4 * pc + j] = rq[j];
        }
    }
    __syncthreads();
    float u[4];
    kq = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) kq += skq[w];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float k2 = 0.f, q2 = 0.f;
        for (int w = 0; w < slots; ++w) {
            k2 += red[(2 * w) * P + 4 * pc + j];
            q2 += red[(2 * w + 1) * P + 4 * pc + j];
        }
        u[j] = beta * fmaf(-a, k2, sv[4 * pc + j]);
        if (rg == 0 && M3_IN(27, (size_t)bh * P + 4 * pc + j, (long long)q.batch * q.nheads * P))
            st_io(static_cast<T*>(q.y) + (size_t)bh * P + 4 * pc + j, q.scale * fmaf(kq, u[j], a * q2));
    }
    float4* dst = reinterpret_cast<float4*>(q.final_h + hb);
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
        const int n = rg + RG * i;
        if (n < N && M3_SPAN(28, hb + (size_t)n * P + 4 * pc, 4, ext_h)) {
            const float kv = sk[n];
            const float4 S = st[i * 256 + tid];
            __stcs(dst + (size_t)n * PC + pc,
                   make_float4(fmaf(kv, u[0], a * S.x), fmaf(kv, u[1], a * S.y), fmaf(kv, u[2], a * S.z),
                               fmaf(kv, u[3], a * S.w)));
        }
    }
}

template <typename K>
static cudaError_t launch(K* kernel, unsigned grid, int smem, cudaStream_t st, const DeltaParams& q) {
    if (smem > 40 * 1024) {              // (the kernels have a little static shared memory too)
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    kernel<<<grid, kThreads, smem, st>>>(q);
    return cudaGetLastError();
}

template <typename T>
static cudaError_t seq(const DeltaParams& q, unsigned grid, cudaStream_t st) {
    const int smem = stage_floats(q.dstate) * 4;
    if (q.dstate <= 32) return launch(delta_seq_kernel<T, 2>, grid, smem, st, q);
    if (q.dstate <= 64) return launch(delta_seq_kernel<T, 4>, grid, smem, st, q);
    if (q.dstate <= 128) return launch(delta_seq_kernel<T, 8>, grid, smem, st, q);
    return launch(delta_seq_kernel<T, 16>, grid, smem, st, q);
}

template <typename T>
static cudaError_t seq_bwd(const DeltaParams& q, unsigned grid, cudaStream_t st) {
    const int N = q.dstate;
    if (N <= 32) return launch(delta_seq_bwd_kernel<T, 2>, grid, grad_floats(N, 2, q.KB) * 4, st, q);
    if (N <= 64) return launch(delta_seq_bwd_kernel<T, 4>, grid, grad_floats(N, 4, q.KB) * 4, st, q);
    if (N <= 128) return launch(delta_seq_bwd_kernel<T, 8>, grid, grad_floats(N, 8, q.KB) * 4, st, q);
    return launch(delta_seq_bwd_kernel<T, 16>, grid, grad_floats(N, 16, q.KB) * 4, st, q);
}

template <typename T>
static cudaError_t step(const DeltaParams& q, unsigned grid, cudaStream_t st) {
    const int RG = 256 / (q.headdim / 4), npt = (q.dstate + RG - 1) / RG;
    if (npt <= 4) return launch(delta_step_kernel<T, 4>, grid, step_floats(q.dstate, q.headdim, 4) * 4, st, q);
    if (npt <= 8) return launch(delta_step_kernel<T, 8>, grid, step_floats(q.dstate, q.headdim, 8) * 4, st, q);
    return launch(delta_step_kernel<T, 16>, grid, step_floats(q.dstate, q.headdim, 16) * 4, st, q);
}

}  // namespace delta

// tokens a checkpoint: the block's states of 16 columns fit shared memory
int delta_block_tokens(const m3_dims& d) { return d.dstate <= 128 ? 16 : 8; }
int delta_tiles(const m3_dims& d) { return (d.headdim + delta::kCols - 1) / delta::kCols; }

cudaError_t launch_delta_seq(const m3_dims& d, const DeltaParams& q, cudaStream_t st) {
    const unsigned grid = (unsigned)((long long)d.batch * d.nheads * delta_tiles(d));
    return d.io_dtype == M3_BF16 ? delta::seq<__nv_bfloat16>(q, grid, st) : delta::seq<float>(q, grid, st);
}

static cudaError_t launch_delta_reduce(const m3_dims& d, const DeltaParams& q, int tiles, cudaStream_t st) {
    const unsigned rows = (unsigned)((long long)d.batch * d.seqlen * d.ngroups);
    if (d.io_dtype == M3_BF16) delta::delta_reduce_kernel<__nv_bfloat16><<<rows, delta::kThreads, 0, st>>>(q, tiles);
    else delta::delta_reduce_kernel<float><<<rows, delta::kThreads, 0, st>>>(q, tiles);
    return cudaGetLastError();
}

cudaError_t launch_delta_seq_bwd(const m3_dims& d, const DeltaParams& q, cudaStream_t st) {
    DeltaParams f = q;                       // checkpoints first
    f.y = nullptr;
    f.final_h = nullptr;
    cudaError_t e = launch_delta_seq(d, f, st);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((long long)d.batch * d.nheads * delta_tiles(d));
    e = d.io_dtype == M3_BF16 ? delta::seq_bwd<__nv_bfloat16>(q, grid, st) : delta::seq_bwd<float>(q, grid, st);
    return e == cudaSuccess ? launch_delta_reduce(d, q, delta_tiles(d), st) : e;
}

// The streaming kernel needs whole float4 columns that divide its 256 threads
// and at most 16 rows a thread; other shapes take the token kernel with one token.
cudaError_t launch_delta_step(const m3_dims& d, const DeltaParams& q, cudaStream_t st) {
    const int P = d.headdim;
    const bool stream = P >= 16 && P <= 256 && (P & (P - 1)) == 0 && d.dstate <= 16 * (1024 / P);
    if (!stream) return launch_delta_seq(d, q, st);
    const unsigned grid = (unsigned)((long long)d.batch * d.nheads);
    return d.io_dtype == M3_BF16 ? delta::step<__nv_bfloat16>(q, grid, st) : delta::step<float>(q, grid, st);
}

}  // namespace m3

M3_BOUNDS_EXPORT(delta)
