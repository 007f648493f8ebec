// k_delta_bwd_tc.cu -- chunked gradient of the gated delta rule (sm_100a):
// bfloat16 io, N = 128, P a multiple of 64.  The formulas of a chunk (notation
// of k_delta_tc.cu; ' marks the gradient of the state behind the chunk):
//   dU  = P^T dY + e^{G_C-G} o (K dS')              P = scale Gam o Q K^T
//   dR  = T^T dU                                     dV = beta o dR
//   dS  = e^{G_C} dS' + Q^T (scale e^G o dY) - K^T (beta e^G o dR)
//   dP  = dY U^T (j <= i)        dA = - dR U^T (j < i)
//   Z = dY S^T,  X = dR S^T,  Y = U dS'^T
//   dQ  = scale e^G o Z + (scale Gam o dP) K
//   dK  = (scale Gam o dP)^T Q + D K + D^T K + e^{G_C-G} o Y - beta e^G o X,   D = beta Gam o dA
//   dbeta_i = dR_i . v_i - e^{G_i} k_i . X_i + sum_j dA_ij Gam_ij k_i.k_j
//   dG_i = (rows - columns of E)_i + scale e^{G_i} q_i.Z_i - beta_i e^{G_i} k_i.X_i - e^{G_C-G_i} k_i.Y_i,
//          E = dP o P + dA o A
//   dG_C += e^{G_C} <S, dS'> + sum_j e^{G_C-G_j} k_j.Y_j;    dg_t = sum_{i >= t} dG_i
//
// Three passes.  The prefill runs once more and records T, P, the state before
// every chunk and U.  k_delta_rev.cu carries dS from the last chunk to the first
// and records dS' and dR.  delta_grad_kernel here then takes all chunks at once,
// one CTA each.  dq and dk of a group's heads
// are added by a further kernel in a fixed order.
//
// The chain and all that feeds sums keep float32 values as two bfloat16 parts
// (hi + lo); a product with two split operands drops lo x lo (2^-17 of the
// product).  Products are 16 x 8 x 16 warp-level mma with register
// accumulators: the matrices of a chunk (64 x 64 to 64 x 128) are masked,
// scaled and split between one product and the next, and register fragments
// take these steps without a way through tensor memory.
//
// Times on one B200 stand with the launcher.
#define M3_BOUNDS_FILE 13
#include "m3_bounds.cuh"
#include "delta_tc.cuh"

namespace m3 {
namespace dbw {

using namespace dtc;


// a matrix in shared memory: rows of 128 bytes (64 columns), 16-byte groups
// exchanged by row (sw128); columns 64.. go on `atom` bytes further
__device__ __forceinline__ uint32_t at(uint32_t base, int atom, int row, int col8) {
    return base + (col8 >> 3) * atom + row * 128 + (((col8 & 7) ^ (row & 7)) << 4);
}
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

struct Mat {
    uint32_t base;
    int atom;
};

// acc (16 rows from m0, 8 NT columns from n0) += A (B + B2), K steps of 16.
// AT: A is stored transposed ([k][m]); BT: B is stored as [n][k], else [k][n].
// B2 (same layout) is left out where its base is 0; n2 is its first column.
template <int NT, int K, bool AT, bool BT, bool TWO>
__device__ __forceinline__ void mm(float (*acc)[4], Mat A, int m0, Mat B, int n0, uint32_t base2, int n2) {
    const int lane = threadIdx.x & 31, mi = lane >> 3, l7 = lane & 7;
#pragma unroll 2
    for (int k0 = 0; k0 < K; k0 += 16) {
        uint32_t a[4];
        if (AT) ldsm4t(a, at(A.base, A.atom, k0 + (mi >> 1) * 8 + l7, (m0 >> 3) + (mi & 1)));
        else ldsm4(a, at(A.base, A.atom, m0 + (mi & 1) * 8 + l7, (k0 >> 3) + (mi >> 1)));
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
            uint32_t b[4];
            if (BT) ldsm4(b, at(B.base, B.atom, n0 + 8 * n + (mi >> 1) * 8 + l7, (k0 >> 3) + (mi & 1)));
            else ldsm4t(b, at(B.base, B.atom, k0 + (mi & 1) * 8 + l7, (n0 >> 3) + n + (mi >> 1)));
            mma16816(acc[n], a, b[0], b[1]);
            mma16816(acc[n + 1], a, b[2], b[3]);
            if (TWO) {
                if (BT) ldsm4(b, at(base2, B.atom, n2 + 8 * n + (mi >> 1) * 8 + l7, (k0 >> 3) + (mi & 1)));
                else ldsm4t(b, at(base2, B.atom, k0 + (mi & 1) * 8 + l7, (n2 >> 3) + n + (mi >> 1)));
                mma16816(acc[n], a, b[0], b[1]);
                mma16816(acc[n + 1], a, b[2], b[3]);
            }
        }
    }
}

template <int NT> __device__ __forceinline__ void zero(float (*acc)[4]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
    const int n = ok ? 16 : 0;               // 0: the destination gets zeros, the source is not read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) { asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory"); }
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ float2 unpack(uint32_t u) { return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)); }
__device__ __forceinline__ uint32_t elem(uint32_t base, int row, int col) { return at(base, 0, row, col >> 3) + (col & 7) * 2; }

__device__ __forceinline__ int length_of(const DeltaParams& q, int b) {
    if (!q.lengths) return q.seqlen;
    return M3_IN(1, b, q.batch) ? min(max(q.lengths[b], 0), q.seqlen) : 0;
}
__device__ __forceinline__ long long ext_rec(const DeltaParams& q) {
    return (long long)q.batch * q.nheads * q.nck * (long long)rec_elems(q.headdim, true);
}

// 64 token rows (chunk c) of q, k or one 64-column tile of v, dy into shared
// memory: `groups` 16-byte groups a row; rows behind the end are zeros
template <int NT>
__device__ __forceinline__ void load_tokens(uint32_t dst, int atom, const void* src, size_t row0, size_t pitch, size_t col,
                                            int groups, int nt, long long ext) {
    for (int e = threadIdx.x; e < 64 * groups; e += NT) {
        const int r = e / groups, g = e - r * groups;
        const size_t o = (row0 + r) * pitch + col + 8 * g;
        const bool ok = r < nt && M3_SPAN(2, o, 8, ext);
        cp16(at(dst, atom, r, g), static_cast<const __nv_bfloat16*>(src) + (ok ? o : 0), ok);
    }
}
// hi and lo part of a recorded matrix with R rows, lo R * 128 bytes behind hi
template <int NT, int R>
__device__ __forceinline__ void load_rec(const DeltaParams& q, uint32_t dst, size_t o) {
    for (int e = threadIdx.x; e < 2 * R * 8; e += NT) {
        const int part = e / (R * 8), f = e % (R * 8);
        const bool ok = M3_SPAN(3, o + (size_t)e * 8, 8, ext_rec(q));
        cp16(at(dst + part * R * 128, 0, f % R, f / R), q.rec + (ok ? o + (size_t)e * 8 : 0), ok);
    }
}

// ------------------------------------------------ the gradients of a chunk --
// 16 warps: warp w has 16 rows (w & 3) and a quarter of the columns (w >> 2).
// Loads arrive in three groups, in the order of their use, so that the products
// begin with the first.
constexpr int kGradThreads = 512;
constexpr uint32_t GR_K = 0, GR_Q = 16384, GR_DY = 32768, GR_V = 40960, GR_U = 49152, GR_DR = 65536, GR_S = 81920,
                   GR_DS = 114688, GR_GATES = 147456;
// where V, U and dR were, after the last slice: P's and A's gradients, rounded
// (they meet K and Q only in products that end in dq and dk, which are rounded
// too); the gradient of A with its transposed, one symmetric matrix
constexpr uint32_t GR_DQK = GR_U, GR_DKK = GR_U + 8192;
struct GradSums {
    float row[4][kC], beta[4][kC], tail[4][kC];      // by column quarter
    float col[4][kC];                                // by row tile
    float drv[kC], dot[16];
};
constexpr int GR_BYTES = GR_GATES + sizeof(Gates) + sizeof(GradSums) + 128;

__global__ void __launch_bounds__(kGradThreads, 1) delta_grad_kernel(DeltaParams q, int nchunks) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    const uint32_t sb = (su32(smem_raw) + 127u) & ~127u;
    uint8_t* smem = smem_raw + (sb - su32(smem_raw));
    Gates* gt = reinterpret_cast<Gates*>(smem + GR_GATES);
    GradSums* gs = reinterpret_cast<GradSums*>(smem + GR_GATES + sizeof(Gates));
    if (!M3_SPAN(11, sb - su32(smem_raw), GR_GATES + sizeof(Gates) + sizeof(GradSums), dyn_smem_bytes())) return;
    constexpr int NT = kGradThreads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, P = q.headdim, H = q.nheads;
    const int bh = blockIdx.x / nchunks, c = blockIdx.x % nchunks;
    const int b = bh / H, h = bh % H, hpg = H / q.ngroups, g = h / hpg;
    const int len = length_of(q, b), nt = min(kC, len - c * kC);
    const int mt = warp & 3, nq = warp >> 2, qr = lane >> 2, qc = (lane & 3) * 2;
    const long long ext_k = (long long)q.batch * q.seqlen * q.ngroups * kN, ext_v = (long long)q.batch * q.seqlen * H * P;
    [[maybe_unused]] const long long toks = (long long)q.batch * q.seqlen * H;
    const size_t row0 = (size_t)b * q.seqlen + c * kC;
    const int rows = min(kC, q.seqlen - c * kC);               // rows of the outputs in this chunk
    __nv_bfloat16* out_q = static_cast<__nv_bfloat16*>(q.dq);
    __nv_bfloat16* out_k = static_cast<__nv_bfloat16*>(q.dk);
    __nv_bfloat16* out_g = static_cast<__nv_bfloat16*>(q.dg);
    __nv_bfloat16* out_b = static_cast<__nv_bfloat16*>(q.dbeta);
    if (nt <= 0) {                                             // behind the end (a group's heads: the sum kernel's zeros)
        if (hpg == 1) {
            for (int e = tid; e < rows * 16; e += NT) {
                const size_t o = ((row0 + (e >> 4)) * q.ngroups + g) * kN + 8 * (e & 15);
                if (M3_SPAN(12, o, 8, ext_k)) {
                    *reinterpret_cast<uint4*>(out_q + o) = make_uint4(0u, 0u, 0u, 0u);
                    *reinterpret_cast<uint4*>(out_k + o) = make_uint4(0u, 0u, 0u, 0u);
                }
            }
            if (tid < rows && M3_IN(13, (row0 + tid) * H + h, toks)) {
                if (out_g) out_g[(row0 + tid) * H + h] = __float2bfloat16_rn(0.f);
                out_b[(row0 + tid) * H + h] = __float2bfloat16_rn(0.f);
            }
        }
        return;
    }
    const size_t rec0 = ((size_t)bh * q.nck + c) * rec_elems(P, true);
    const Mat K = {sb + GR_K, 8192}, Q = {sb + GR_Q, 8192}, dY = {sb + GR_DY, 0};
    const Mat Uh = {sb + GR_U, 0}, Ul = {sb + GR_U + 8192, 0}, dRh = {sb + GR_DR, 0}, dRl = {sb + GR_DR + 8192, 0};
    const Mat Sh = {sb + GR_S, 0}, Dh = {sb + GR_DS, 0};

    float kk[2][4], dP[2][4], dA[2][4], Z[4][4], X[4][4], Y[4][4];
    zero<2>(kk); zero<2>(dP); zero<2>(dA); zero<4>(Z); zero<4>(X); zero<4>(Y);
    float dot = 0.f, drv = 0.f;                                // <S, dS'>, dR . v of row tid / 8
    for (int sl = 0; sl < P / 64; ++sl) {
        if (sl > 0) __syncthreads();
        const size_t o = rec0 + kRecSlice + sl * kSliceElems;
        load_tokens<NT>(sb + GR_DY, 0, q.dy, row0, (size_t)H * P, (size_t)h * P + 64 * sl, 8, nt, ext_v);
        load_rec<NT, 64>(q, sb + GR_U, o + kSliceU);
        load_rec<NT, 64>(q, sb + GR_DR, o + kSliceDR);
        cp_commit();
        load_rec<NT, 128>(q, sb + GR_S, o + kSliceS);
        load_tokens<NT>(sb + GR_V, 0, q.v, row0, (size_t)H * P, (size_t)h * P + 64 * sl, 8, nt, ext_v);
        cp_commit();
        load_rec<NT, 128>(q, sb + GR_DS, o + kSliceDS);
        if (sl == 0) {
            load_tokens<NT>(sb + GR_K, 8192, q.k, row0, (size_t)q.ngroups * kN, (size_t)g * kN, 16, nt, ext_k);
            load_tokens<NT>(sb + GR_Q, 8192, q.q, row0, (size_t)q.ngroups * kN, (size_t)g * kN, 16, nt, ext_k);
        }
        cp_commit();
        if (sl == 0 && warp == 0) make_gates(load_raw(q, b, h, len, c), gt);
        asm volatile("cp.async.wait_group 2;" ::: "memory");
        __syncthreads();
        mm<2, 64, false, true, true>(dP, dY, 16 * mt, Uh, 16 * nq, Ul.base, 16 * nq);
        mm<2, 64, false, true, true>(dA, dRh, 16 * mt, Uh, 16 * nq, Ul.base, 16 * nq);
        mm<2, 64, false, true, false>(dA, dRl, 16 * mt, Uh, 16 * nq, 0, 0);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        mm<4, 64, false, true, true>(Z, dY, 16 * mt, Sh, 32 * nq, Sh.base + 16384, 32 * nq);
        mm<4, 64, false, true, true>(X, dRh, 16 * mt, Sh, 32 * nq, Sh.base + 16384, 32 * nq);
        mm<4, 64, false, true, false>(X, dRl, 16 * mt, Sh, 32 * nq, 0, 0);
        {
            const uint32_t p = at(0, 0, tid >> 3, tid & 7);
            const uint4 r0 = lds128(dRh.base + p), r1 = lds128(dRl.base + p), v0 = lds128(sb + GR_V + p);
            const uint32_t rh[4] = {r0.x, r0.y, r0.z, r0.w}, rl[4] = {r1.x, r1.y, r1.z, r1.w}, vv[4] = {v0.x, v0.y, v0.z, v0.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 d = __fadd2_rn(unpack(rh[j]), unpack(rl[j])), v = unpack(vv[j]);
                drv = fmaf(d.x, v.x, fmaf(d.y, v.y, drv));
            }
        }
        cp_wait();
        __syncthreads();
        mm<4, 64, false, true, true>(Y, Uh, 16 * mt, Dh, 32 * nq, Dh.base + 16384, 32 * nq);
        mm<4, 64, false, true, false>(Y, Ul, 16 * mt, Dh, 32 * nq, 0, 0);
#pragma unroll
        for (int e = tid; e < 128 * 8; e += NT) {
            const uint32_t p = at(0, 0, e >> 3, e & 7);
            const uint4 s0 = lds128(sb + GR_S + p), s1 = lds128(sb + GR_S + 16384 + p);
            const uint4 d0 = lds128(sb + GR_DS + p), d1 = lds128(sb + GR_DS + 16384 + p);
            const uint32_t sh[4] = {s0.x, s0.y, s0.z, s0.w}, s2[4] = {s1.x, s1.y, s1.z, s1.w};
            const uint32_t dh[4] = {d0.x, d0.y, d0.z, d0.w}, d2[4] = {d1.x, d1.y, d1.z, d1.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 a = __fadd2_rn(unpack(sh[j]), unpack(s2[j])), d = __fadd2_rn(unpack(dh[j]), unpack(d2[j]));
                dot = fmaf(a.x, d.x, fmaf(a.y, d.y, dot));
            }
        }
    }
    mm<2, 128, false, true, false>(kk, K, 16 * mt, K, 16 * nq, 0, 0);
    __syncthreads();                                           // U and dR have been read: their place takes dP and D
    drv += __shfl_xor_sync(kFull, drv, 1);
    drv += __shfl_xor_sync(kFull, drv, 2);
    drv += __shfl_xor_sync(kFull, drv, 4);
    if ((tid & 7) == 0) gs->drv[tid >> 3] = drv;
#pragma unroll
    for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
    if (lane == 0) gs->dot[warp] = dot;

    float rowG[2] = {0.f, 0.f}, rowB[2] = {0.f, 0.f}, tail[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const int j = 16 * nq + 8 * n + qc;
        float cs[2] = {0.f, 0.f};
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int i = 16 * mt + qr + 8 * r;
            const float2 Gi = gt->G[i];
            const float be = gt->beta[i];
            float fq[2];
            const size_t o = rec0 + (sw128(i, j >> 3) >> 1) + (j & 7);
            float2 pv = make_float2(0.f, 0.f);
            if (M3_SPAN(14, o + kRecPL, 2, ext_rec(q)))
                pv = __fadd2_rn(unpack(*reinterpret_cast<const uint32_t*>(q.rec + o + kRecX + kTok)),
                                unpack(*reinterpret_cast<const uint32_t*>(q.rec + o + kRecPL)));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float gam = i >= j + e ? ex2(diff_pair(Gi, gt->G[j + e])) : 0.f;
                const float dp = i >= j + e ? dP[n][2 * r + e] : 0.f;
                const float da = i > j + e ? -dA[n][2 * r + e] * gam : 0.f;
                const float t = da * kk[n][2 * r + e];
                const float E = fmaf(dp, e ? pv.y : pv.x, be * t);
                rowG[r] += E;
                cs[e] += E;
                rowB[r] += t;
                fq[e] = q.scale * gam * dp;
                // D at (i, j) and (j, i); the diagonal is zero
                const __nv_bfloat16 v = __float2bfloat16_rn(be * da);
                if (i >= j + e && M3_IN(19, i * 64 + j + e, 4096)) {
                    *reinterpret_cast<__nv_bfloat16*>(smem + elem(GR_DKK, i, j + e)) = v;
                    *reinterpret_cast<__nv_bfloat16*>(smem + elem(GR_DKK, j + e, i)) = v;
                }
            }
            sts32(elem(sb + GR_DQK, i, j), pack_bf16x2(fq[0], fq[1]));
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) cs[e] += __shfl_xor_sync(kFull, cs[e], o);
            if (qr == 0) gs->col[mt][j + e] = cs[e];
        }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int i = 16 * mt + qr + 8 * r;
        const float a = gt->a[i], tl = gt->at[i], be = gt->beta[i], sa = q.scale * a, ba = be * a;
        float zq = 0.f, xk = 0.f, yk = 0.f;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int col = 32 * nq + 8 * n + qc;
            const uint32_t p = at(0, 8192, i, col >> 3) + (col & 7) * 2;
            const float2 qv = unpack(lds32(sb + GR_Q + p)), kv = unpack(lds32(sb + GR_K + p));
            zq = fmaf(Z[n][2 * r], qv.x, fmaf(Z[n][2 * r + 1], qv.y, zq));
            xk = fmaf(X[n][2 * r], kv.x, fmaf(X[n][2 * r + 1], kv.y, xk));
            yk = fmaf(Y[n][2 * r], kv.x, fmaf(Y[n][2 * r + 1], kv.y, yk));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                Z[n][2 * r + e] *= sa;
                Y[n][2 * r + e] = fmaf(tl, Y[n][2 * r + e], -ba * X[n][2 * r + e]);
            }
        }
        rowG[r] += sa * zq - ba * xk - tl * yk;
        rowB[r] -= a * xk;
        tail[r] = tl * yk;
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            rowG[r] += __shfl_xor_sync(kFull, rowG[r], o);
            rowB[r] += __shfl_xor_sync(kFull, rowB[r], o);
            tail[r] += __shfl_xor_sync(kFull, tail[r], o);
        }
        if ((lane & 3) == 0) {
            gs->row[nq][i] = rowG[r];
            gs->beta[nq][i] = rowB[r];
            gs->tail[nq][i] = tail[r];
        }
    }
    __syncthreads();
    const Mat Pq = {sb + GR_DQK, 0}, Dk = {sb + GR_DKK, 0};
    mm<4, 64, false, false, false>(Z, Pq, 16 * mt, K, 32 * nq, 0, 0);
    mm<4, 64, true, false, false>(Y, Pq, 16 * mt, Q, 32 * nq, 0, 0);
    mm<4, 64, false, false, false>(Y, Dk, 16 * mt, K, 32 * nq, 0, 0);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int i = 16 * mt + qr + 8 * r;
        const float m = i < nt ? 1.f : 0.f;
        if (i >= rows) continue;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int col = 32 * nq + 8 * n + qc;
            const float2 vq = make_float2(m * Z[n][2 * r], m * Z[n][2 * r + 1]), vk = make_float2(m * Y[n][2 * r], m * Y[n][2 * r + 1]);
            if (hpg == 1) {
                const size_t o = ((row0 + i) * q.ngroups + g) * kN + col;
                if (M3_SPAN(15, o, 2, ext_k)) {
                    *reinterpret_cast<uint32_t*>(out_q + o) = pack_bf16x2(vq.x, vq.y);
                    *reinterpret_cast<uint32_t*>(out_k + o) = pack_bf16x2(vk.x, vk.y);
                }
            } else {
                const size_t o = ((row0 + i) * H + h) * 2 * kN + col;
                if (M3_SPAN(16, o + kN, 2, toks * 2 * kN)) {
                    *reinterpret_cast<float2*>(q.part_qk + o) = vq;
                    *reinterpret_cast<float2*>(q.part_qk + o + kN) = vk;
                }
            }
        }
    }
    if (warp == 0) {
        // lane l has tokens 2 l, 2 l + 1; dg is the sum from a token to the chunk's end
        float d[2], tl = 0.f, total = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = 2 * lane + e;
            d[e] = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                d[e] += gs->row[j][i] - gs->col[j][i];
                tl += gs->tail[j][i];
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) tl += __shfl_xor_sync(kFull, tl, o);
#pragma unroll
        for (int j = 0; j < 16; ++j) total += gs->dot[j];
        tl += gt->whole * total;
        float sum = d[0] + d[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float u = __shfl_down_sync(kFull, sum, o);
            if (lane + o < 32) sum += u;
        }
        const float dg[2] = {sum + tl, sum - d[0] + tl};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = 2 * lane + e;
            const size_t o = (row0 + i) * H + h;
            if (i >= rows || !M3_IN(17, o, toks)) continue;
            const float vg = i < nt ? dg[e] : 0.f;
            const float vb = i < nt ? gs->drv[i] + gs->beta[0][i] + gs->beta[1][i] + gs->beta[2][i] + gs->beta[3][i] : 0.f;
            if (hpg == 1) {
                if (out_g) out_g[o] = __float2bfloat16_rn(vg);
                out_b[o] = __float2bfloat16_rn(vb);
            } else {
                q.part_g[2 * o] = vg;
                q.part_g[2 * o + 1] = vb;
            }
        }
    }
}

}  // namespace dbw

cudaError_t launch_delta_bwd_tc(const m3_dims& d, const DeltaParams& q, int* status, cudaStream_t st) {
    using namespace dbw;
    DeltaParams f = q;                       // records of the prefill
    f.y = nullptr;
    f.final_h = nullptr;
    cudaError_t e = launch_delta_tc(d, f, true, status, st);
    if (e != cudaSuccess) return e;
    e = launch_delta_rev(d, q, status, st);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(delta_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, GR_BYTES);
    if (e != cudaSuccess) return e;
    delta_grad_kernel<<<(unsigned)((long long)d.batch * d.nheads * q.nck), kGradThreads, GR_BYTES, st>>>(q, q.nck);
    e = cudaGetLastError();
    if (e != cudaSuccess || d.nheads == d.ngroups) return e;
    return launch_delta_reduce(d, q, 1, st);
}

}  // namespace m3

M3_BOUNDS_EXPORT(delta_bwd_tc)
