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
//   warps 9-16   two groups, every other chunk each, up to two chunks ahead:
//                gates, K K^T and Q K^T (one product of the stacked rows
//                [K; Q] with K), T and the masked Q K^T
//   warp 17      one lane issues the TMA loads (three chunks of K, Q, two of V)
// Every product has M = 128 rows: [K; Q] against S gives K S and Q S at once,
// and the tile [T - I; P] (P = scale Gam o Q K^T) serves both T R (upper half
// of the accumulator) and P U (lower half); the unused half is never read.
// The parts of a split operand stand side by side as columns of one product
// (a 128 x 128 x 16 product takes 64 cycles, a 128 x 64 x 16 one 47) and the
// epilogue adds the columns.
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
// 2 x 8, scratch 2 x 12, gates 6: one CTA an SM.
//
// Every wait on an mbarrier is bounded (1 s); on expiry the kernel records
// M3_ERR_DEVICE_TIMEOUT in the workspace status word and runs out without
// further waiting.
#define M3_BOUNDS_FILE 12
#include "m3_bounds.cuh"
#include <stdlib.h>

#include "delta_tc.cuh"

namespace m3 {

bool make_tile_map(CUtensorMap* map, const void* base, int inner, int R, int grp, int L, int batch, int T);

namespace dtc {

constexpr int kP = 64;             // columns of a V tile; a CTA takes PC = 64, 32 or 16 of them
constexpr int kState = 256;        // threads of the chain
constexpr int kPrep = 128;         // threads of one of the two groups that make T
constexpr int kThreads = 32 + kState + 2 * kPrep + 32;

constexpr int OFF_KQ = 0;                       // 3 x 32 KB: two 64-column atoms, rows 0..63 K, 64..127 Q
constexpr int OFF_V = OFF_KQ + 3 * 32768;       // 2 x 8 KB
constexpr int OFF_S = OFF_V + 2 * 8192;         // S hi, S lo (16 KB each: rows n, 64 p)
constexpr int OFF_U = OFF_S;                    // R hi, lo; then e^{G_C-G} U in three parts (8 KB each: rows t, 64 p)
constexpr int OFF_UB = OFF_S + 24576;           // U rounded, for P U
constexpr int OFF_X = OFF_S + 32768;            // 2 x 16 KB: [T - I hi; P]
constexpr int OFF_TL = OFF_X + 2 * 16384;       // 2 x 8 KB: T - I lo (its operand reads 64 more rows, unused)
constexpr int OFF_SCR = OFF_TL + 2 * 8192;      // of each group:
constexpr int SCR_D = 0;                        //   4 KB: A's 16 x 16 diagonal blocks, float32, by columns
constexpr int SCR_21 = 4096;                    //   4 KB: A's lower left 32 x 32 block, hi and lo side by side
constexpr int SCR_10 = 8192;                    //   2 KB: its two 16 x 16 blocks under the diagonal, hi, lo, hi, lo
constexpr int SCR_BYTES = 10240;
constexpr int OFF_MISC = OFF_SCR + 2 * SCR_BYTES;

// TMEM columns: K S, Q S against [S hi | S lo] and, once they are read, the
// state's update in three parts; T R against [R hi | R lo] and, once read, P U;
// one Gram product a group
constexpr uint32_t D_KS = 0, D_S = 0, D_TR = 192, D_G = 320;

struct Misc {
    uint64_t kq_full[3], kq_free[3], v_full[2], v_free[2], t_full[2], x_free[2], g[2];
    uint64_t s_ready, ks, r, tr, u, s, o, drain[3];
    uint32_t tmem_base;
    int abort_flag, drain_flag, pad;
    Gates gates[5];
};
constexpr int SMEM_BYTES = OFF_MISC + (int)sizeof(Misc) + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory of the delta kernel");

__device__ __forceinline__ bool wait(uint64_t* b, int phase, Misc* m, int* status, int where) {
    return mbar_wait_flag(b, (uint32_t)(phase & 1), &m->abort_flag, status, where);
}
__device__ __forceinline__ void group_sync(int group) { asm volatile("bar.sync %0, %1;" ::"r"(2 + group), "n"(kPrep) : "memory"); }
// Products and commits by one elected lane of a converged warp: the warp runs
// the loop as one, so that descriptors stay in uniform registers (measured:
// 47 cycles a 128 x 64 x 16 product instead of 97 from a divergent lane).
__device__ __forceinline__ void umma_one(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void commit_one(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(su32(bar))
        : "memory");
}

// 16 bytes at `off` of the tile that starts at `tile` and has `limit` bytes
__device__ __forceinline__ void put16(uint8_t* smem, int tile, uint32_t off, int limit, uint4 v) {
    if (M3_SPAN(1, off, 16, limit)) *reinterpret_cast<uint4*>(smem + tile + off) = v;
}

struct Where {
    int b, h, g, p0, len, nch;     // p0: first column of the CTA
};

template <int PC>
__device__ __forceinline__ Where where_am_i(const DeltaParams& q) {
    Where w;
    const int slices = q.headdim / PC;
    const int bh = blockIdx.x / slices;
    w.p0 = (blockIdx.x % slices) * PC;
    w.b = bh / q.nheads;
    w.h = bh % q.nheads;
    w.g = w.h / (q.nheads / q.ngroups);
    int len = q.seqlen;
    if (q.lengths && M3_IN(3, w.b, q.batch)) len = min(max(q.lengths[w.b], 0), q.seqlen);
    w.len = len;
    w.nch = (len + kC - 1) / kC;
    return w;
}

// column `lane` (< 16) of the inverse of a unit lower triangular 16 x 16 matrix
// whose strict lower part is at[col * 16 + row] (zeros elsewhere): x starts as
// the unit vector, and a finished x_i takes A_ri x_i off every later x_r
__device__ __forceinline__ void invert16(const float* at, float2* x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = make_float2(2 * i == lane ? 1.f : 0.f, 2 * i + 1 == lane ? 1.f : 0.f);
#pragma unroll
    for (int i = 0; i < 15; ++i) {
        const float xi = (i & 1) ? -x[i >> 1].y : -x[i >> 1].x;
        const float2 x2 = make_float2(xi, xi);
#pragma unroll
        for (int r4 = (i + 1) / 4; r4 < 4; ++r4) {
            const float4 v = *reinterpret_cast<const float4*>(at + i * 16 + 4 * r4);
            if (4 * r4 + 1 > i) x[2 * r4] = __ffma2_rn(make_float2(v.x, v.y), x2, x[2 * r4]);
            x[2 * r4 + 1] = __ffma2_rn(make_float2(v.z, v.w), x2, x[2 * r4 + 1]);
        }
    }
}

__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void stsm4(uint32_t addr, const uint32_t* r) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) { asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory"); }
__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// accumulators of two 8-column tiles as the left operand of the next product, hi and lo
__device__ __forceinline__ void split_acc(const float (*c)[4], uint32_t* hi, uint32_t* lo) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 f = make_float2(c[i >> 1][2 * (i & 1)], c[i >> 1][2 * (i & 1) + 1]);
        hi[i] = take2(f);
        lo[i] = pack_bf16x2(f.x, f.y);
    }
}

// The inverse of a chunk's unit lower triangular matrix from its 16 x 16
// diagonal blocks' inverses, as T^T (upper triangular, hi at `hi`, lo at `lo`,
// rows of 128 bytes).  With M^T = T_a^T A_ba^T the block below T_a, left of
// T_b, is T_ba^T = - M^T T_b^T: the accumulators of the first product are the
// left operand of the second as they stand.  Level 1: 16 x 16 blocks (A_ba in
// `a10`), warps 2 p and 2 p + 1 do the 32 x 32 block p.
__device__ __forceinline__ void join16(uint32_t hi, uint32_t lo, uint32_t a10, int wq) {
    const int lane = threadIdx.x & 31, mi = lane >> 3, l7 = lane & 7, p = wq >> 1, nh = wq & 1;
    uint32_t ah[4], al[4], bh[4], bl[4];
    const uint32_t oa = sw128(32 * p + (mi & 1) * 8 + l7, 4 * p + (mi >> 1));
    ldsm4(ah, hi + oa);
    ldsm4(al, lo + oa);
    const int rb = (mi >> 1) * 8 + l7;
    ldsm4(bh, a10 + sw128(rb, 4 * p + (mi & 1)));
    ldsm4(bl, a10 + sw128(rb, 4 * p + 2 + (mi & 1)));
    float c[2][4] = {};
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        mma16816(c[n], al, bh[2 * n], bh[2 * n + 1]);
        mma16816(c[n], ah, bl[2 * n], bl[2 * n + 1]);
        mma16816(c[n], ah, bh[2 * n], bh[2 * n + 1]);
    }
    split_acc(c, ah, al);
    // T_b^T: k rows 32 p + 16 .., 8 columns; hi and lo in one load
    ldsm4t(bh, ((mi >> 1) ? lo : hi) + sw128(32 * p + 16 + (mi & 1) * 8 + l7, 4 * p + 2 + nh));
    float d[4] = {};
    mma16816(d, al, bh[0], bh[1]);
    mma16816(d, ah, bh[2], bh[3]);
    mma16816(d, ah, bh[0], bh[1]);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float2 f = make_float2(-d[2 * r], -d[2 * r + 1]);
        const uint32_t o = sw128(32 * p + (lane >> 2) + 8 * r, 4 * p + 2 + nh) + (lane & 3) * 4;
        sts32(hi + o, take2(f));
        sts32(lo + o, pack_bf16x2(f.x, f.y));
    }
    if (lane < 16) {               // below T_a^T stands zero
        const uint32_t o = sw128(32 * p + 16 + lane, 4 * p + nh);
        sts128(hi + o, make_uint4(0u, 0u, 0u, 0u));
        sts128(lo + o, make_uint4(0u, 0u, 0u, 0u));
    }
}
// Level 2: the 32 x 32 block (A_ba in `a21`); a warp has 16 of its columns and rows
__device__ __forceinline__ void join32(uint32_t hi, uint32_t lo, uint32_t a21, int wq) {
    const int lane = threadIdx.x & 31, mi = lane >> 3, l7 = lane & 7, mt = wq & 1, nh = wq >> 1;
    float c[4][4] = {};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t ah[4], al[4];
        const uint32_t oa = sw128(16 * mt + (mi & 1) * 8 + l7, 2 * k + (mi >> 1));
        ldsm4(ah, hi + oa);
        ldsm4(al, lo + oa);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            uint32_t bh[4], bl[4];
            const int rb = 16 * n + (mi >> 1) * 8 + l7;
            ldsm4(bh, a21 + sw128(rb, 2 * k + (mi & 1)));
            ldsm4(bl, a21 + sw128(rb, 4 + 2 * k + (mi & 1)));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mma16816(c[2 * n + e], al, bh[2 * e], bh[2 * e + 1]);
                mma16816(c[2 * n + e], ah, bl[2 * e], bl[2 * e + 1]);
                mma16816(c[2 * n + e], ah, bh[2 * e], bh[2 * e + 1]);
            }
        }
    }
    float d[2][4] = {};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t ah[4], al[4], bh[4], bl[4];
        split_acc(c + 2 * k, ah, al);
        const uint32_t ob = sw128(32 + 16 * k + (mi & 1) * 8 + l7, 4 + 2 * nh + (mi >> 1));
        ldsm4t(bh, hi + ob);
        ldsm4t(bl, lo + ob);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            mma16816(d[e], al, bh[2 * e], bh[2 * e + 1]);
            mma16816(d[e], ah, bl[2 * e], bl[2 * e + 1]);
            mma16816(d[e], ah, bh[2 * e], bh[2 * e + 1]);
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float2 f = make_float2(-d[e][2 * r], -d[e][2 * r + 1]);
            const uint32_t o = sw128(16 * mt + (lane >> 2) + 8 * r, 4 + 2 * nh + e) + (lane & 3) * 4;
            sts32(hi + o, take2(f));
            sts32(lo + o, pack_bf16x2(f.x, f.y));
        }
}

// NP loads of W consecutive columns (32 lanes, thread = lane), `step` columns
// apart, issued back to back with one wait; their sum
template <int W, int NP> __device__ __forceinline__ void tmem_sum(uint32_t t, uint32_t step, float2* f);
template <> __device__ __forceinline__ void tmem_sum<8, 1>(uint32_t t, uint32_t step, float2* f) {
    uint32_t r[8];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(t + 0)
        : "memory");
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[j] = make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
    }
}
template <> __device__ __forceinline__ void tmem_sum<8, 2>(uint32_t t, uint32_t step, float2* f) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%16];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%17];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t + 0), "r"(t + 1 * step)
        : "memory");
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[j] = make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
        f[j] = __fadd2_rn(f[j], make_float2(__uint_as_float(r[8 + 2 * j]), __uint_as_float(r[9 + 2 * j])));
    }
}
template <> __device__ __forceinline__ void tmem_sum<8, 3>(uint32_t t, uint32_t step, float2* f) {
    uint32_t r[24];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%24];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%25];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16,%17,%18,%19,%20,%21,%22,%23}, [%26];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23])
        : "r"(t + 0), "r"(t + 1 * step), "r"(t + 2 * step)
        : "memory");
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[j] = make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
        f[j] = __fadd2_rn(f[j], __fadd2_rn(make_float2(__uint_as_float(r[8 + 2 * j]), __uint_as_float(r[9 + 2 * j])),
                                           make_float2(__uint_as_float(r[16 + 2 * j]), __uint_as_float(r[17 + 2 * j]))));
    }
}
template <> __device__ __forceinline__ void tmem_sum<16, 1>(uint32_t t, uint32_t step, float2* f) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t + 0)
        : "memory");
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        f[j] = make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
    }
}
template <> __device__ __forceinline__ void tmem_sum<16, 2>(uint32_t t, uint32_t step, float2* f) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(t + 0), "r"(t + 1 * step)
        : "memory");
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        f[j] = make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
        f[j] = __fadd2_rn(f[j], make_float2(__uint_as_float(r[16 + 2 * j]), __uint_as_float(r[17 + 2 * j])));
    }
}
template <> __device__ __forceinline__ void tmem_sum<16, 3>(uint32_t t, uint32_t step, float2* f) {
    uint32_t r[48];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%48];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%49];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47}, [%50];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47])
        : "r"(t + 0), "r"(t + 1 * step), "r"(t + 2 * step)
        : "memory");
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        f[j] = make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
        f[j] = __fadd2_rn(f[j], __fadd2_rn(make_float2(__uint_as_float(r[16 + 2 * j]), __uint_as_float(r[17 + 2 * j])),
                                           make_float2(__uint_as_float(r[32 + 2 * j]), __uint_as_float(r[33 + 2 * j]))));
    }
}

// Split operands.  A row of a tile has 128 bytes, 64 bfloat16 columns; the parts
// of an operand stand side by side, PC columns each, and go on in further tiles
// (16 KB for 128 rows, 8 KB for 64).  Byte offset of part `part`, 16-byte
// column group `ch` (PC / 8 a part) of row `row`:
template <int PC>
__device__ __forceinline__ uint32_t part_at(int row, int part, int ch, int tile_bytes) {
    const int col = part * (PC / 8) + ch;
    return (uint32_t)((col >> 3) * tile_bytes) + sw128(row, col & 7);
}

// DUMP: also write the records that the gradient's passes read
template <int PC, bool DUMP>
__global__ void __launch_bounds__(kThreads, 1)
    delta_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ,
                    const __grid_constant__ CUtensorMap tmV, DeltaParams q, int* status) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (su32(smem_raw) & 1023u)) & 1023u);
    Misc* m = reinterpret_cast<Misc*>(smem + OFF_MISC);
    const uint32_t sbase = su32(smem);
    if (!M3_SPAN(5, smem - smem_raw, OFF_MISC + (int)sizeof(Misc), dyn_smem_bytes())) return;
    const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
    const Where w = where_am_i<PC>(q);
    constexpr int kCols = PC / 2;                  // state columns a thread
    constexpr int W = kCols < 16 ? kCols : 16;     // columns of a TMEM load
    constexpr int NH = kCols / W, NG = kCols / 8;  // loads; 16-byte groups
    const int P = q.headdim;
    const size_t bh = (size_t)w.b * q.nheads + w.h;

    if (tid == 0) {
        for (int i = 0; i < 3; ++i) { mbar_init(&m->kq_full[i], 1); mbar_init(&m->kq_free[i], 1); mbar_init(&m->drain[i], 1); }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m->v_full[i], 1);
            mbar_init(&m->v_free[i], kState / 2);
            mbar_init(&m->t_full[i], kPrep);
            mbar_init(&m->x_free[i], 1);
            mbar_init(&m->g[i], 1);
        }
        mbar_init(&m->s_ready, kState);
        mbar_init(&m->ks, 1);
        mbar_init(&m->r, kState);
        mbar_init(&m->tr, 1);
        mbar_init(&m->u, kState);
        mbar_init(&m->s, 1);
        mbar_init(&m->o, 1);
        m->abort_flag = 0;
        m->drain_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
    }
    if (warp == 0) {
        tmem_alloc(&m->tmem_base, 512);
        tmem_relinquish();
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = m->tmem_base;

    if (warp == 0) {
        // ------------------------------------------------ the chain's products
        // (descriptor starts count 16 bytes)
        constexpr uint32_t idKS = idesc_bf16(128, 2 * PC, 0, 1);   // A K-major, B MN-major
        constexpr uint32_t idTl = idesc_bf16(128, PC, 0, 1);
        constexpr uint32_t idS = idesc_bf16(128, 3 * PC, 1, 1);    // A MN-major (K^T)
        const uint64_t bS = sdesc(sbase + OFF_S, 16384, 1024), bU = sdesc(sbase + OFF_U, 8192, 1024);
        const uint64_t bUB = sdesc(sbase + OFF_UB, 8192, 1024);
        for (int c = 0; c < w.nch; ++c) {
            const uint32_t kq = sbase + OFF_KQ + (c % 3) * 32768;
            const uint64_t aKQ = sdesc(kq, 16, 1024), aKT = sdesc(kq, 16384, 1024);
            const uint64_t aX = sdesc(sbase + OFF_X + (c & 1) * 16384, 16, 1024);
            const uint64_t aTL = sdesc(sbase + OFF_TL + (c & 1) * 8192, 16, 1024);
            wait(&m->kq_full[c % 3], c / 3, m, status, 1);
            // a chunk that ends behind the sequence: its K rows are cleaned by
            // the group that hands over T
            if ((c + 1) * kC > w.len) wait(&m->t_full[c & 1], c >> 1, m, status, 2);
            wait(&m->s_ready, c, m, status, 3);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                umma_one(tmem + D_KS, aKQ + (kk >> 2) * 1024 + (kk & 3) * 2, bS + kk * 128, idKS, kk > 0);
            commit_one(&m->ks);
            wait(&m->t_full[c & 1], c >> 1, m, status, 4);
            wait(&m->r, c, m, status, 5);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) umma_one(tmem + D_TR, aX + kk * 2, bU + kk * 128, idKS, kk > 0);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) umma_one(tmem + D_TR, aTL + kk * 2, bU + kk * 128, idTl, 1);
            commit_one(&m->tr);
            wait(&m->u, c, m, status, 6);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) umma_one(tmem + D_S, aKT + kk * 128, bU + kk * 128, idS, kk > 0);
            commit_one(&m->s);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) umma_one(tmem + D_TR + PC, aX + kk * 2, bUB + kk * 128, idTl, kk > 0);
            commit_one(&m->o);
            commit_one(&m->kq_free[c % 3]);
            commit_one(&m->x_free[c & 1]);
        }
        commit_one(&m->drain[2]);
        mbar_wait_flag(&m->drain[2], 0, &m->drain_flag, nullptr, 0);
        __syncwarp();
    } else if (warp <= 8) {
        // ---------------------------------------------- the chain's arithmetic
        const int wk = tid - 32, wg = wk >> 7, quarter = warp & 3, row = quarter * 32 + lane, c0 = wg * kCols;
        const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16) + c0;
        const bool top = quarter < 2;              // holds a token's K S and U; else its Q S and y
        const int tok = row & 63, ch0 = c0 / 8, vch = (w.p0 & 63) / 8 + ch0;
        [[maybe_unused]] const long long ext_h = (long long)q.batch * q.nheads * kN * P;
        const size_t ho = (bh * kN + row) * P + w.p0 + c0;
        float2 S[kCols / 2];
#pragma unroll
        for (int c4 = 0; c4 < kCols / 4; ++c4) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (q.init_h && M3_SPAN(6, ho + 4 * c4, 4, ext_h)) v = *reinterpret_cast<const float4*>(q.init_h + ho + 4 * c4);
            S[2 * c4] = make_float2(v.x, v.y);
            S[2 * c4 + 1] = make_float2(v.z, v.w);
        }
        // this CTA's columns in a record, and this thread's first one
        auto slice_of = [&](int c) {
            return q.rec + (bh * q.nck + c) * rec_elems(P) + kRecSlice + (size_t)(w.p0 >> 6) * kSliceElems + (w.p0 & 63) + c0;
        };
        auto keep = [&](__nv_bfloat16* dst, int ch, uint4 v) {
            if (M3_SPAN(10, dst + 8 * ch - q.rec, 8, (long long)q.batch * q.nheads * q.nck * rec_elems(P)))
                *reinterpret_cast<uint4*>(dst + 8 * ch) = v;
        };
        auto store_state = [&](int c) {            // S hi, S lo before chunk c
#pragma unroll
            for (int ch = 0; ch < NG; ++ch) {
                float2 f[4] = {S[4 * ch], S[4 * ch + 1], S[4 * ch + 2], S[4 * ch + 3]};
                const uint4 hi = take8(f), lo = round8(f);
                put16(smem, OFF_S, part_at<PC>(row, 0, ch0 + ch, 16384), 32768, hi);
                put16(smem, OFF_S, part_at<PC>(row, 1, ch0 + ch, 16384), 32768, lo);
                if (DUMP) {
                    keep(slice_of(c) + kSliceS + row * 64, ch, hi);
                    keep(slice_of(c) + kSliceS + kSt + row * 64, ch, lo);
                }
            }
            fence_async_smem();
            tc_fence_before();
            mbar_arrive(&m->s_ready);
        };
        if (w.nch > 0) store_state(0);
#pragma unroll 1
        for (int c = 0; c < w.nch; ++c) {
            const Gates* gt = &m->gates[c % 5];
            float2 buf[kCols / 2];                 // top: beta V, R, then U; else Q S
            if (top) {
                wait(&m->v_full[c & 1], c >> 1, m, status, 10);
                wait(&m->t_full[c & 1], c >> 1, m, status, 11);
                const float be = gt->beta[tok], ba = -be * gt->a[tok], at = gt->at[tok];
                const bool in = c * kC + tok < w.len;
                const float2 be2 = make_float2(be, be), ba2 = make_float2(ba, ba), at2 = make_float2(at, at);
                // beta V; rows behind the end (other data, possibly not numbers) count as zero
#pragma unroll
                for (int ch = 0; ch < NG; ++ch) {
                    const uint32_t o = sw128(tok, vch + ch);
                    uint4 vv = make_uint4(0u, 0u, 0u, 0u);
                    if (in && M3_SPAN(7, o, 16, 8192)) vv = *reinterpret_cast<const uint4*>(smem + OFF_V + (c & 1) * 8192 + o);
                    const uint32_t u[4] = {vv.x, vv.y, vv.z, vv.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        buf[4 * ch + j] = __fmul2_rn(be2, make_float2(__uint_as_float(u[j] << 16),
                                                                      __uint_as_float(u[j] & 0xffff0000u)));
                }
                wait(&m->ks, c, m, status, 12);
                __syncwarp();
                tc_fence_after();
#pragma unroll
                for (int hh = 0; hh < NH; ++hh) {
                    float2 d[W / 2];
                    tmem_sum<W, 2>(tl + D_KS + W * hh, PC, d);
#pragma unroll
                    for (int j = 0; j < W / 2; ++j) d[j] = buf[W / 2 * hh + j] = __ffma2_rn(ba2, d[j], buf[W / 2 * hh + j]);
#pragma unroll
                    for (int ch = 0; ch < W / 8; ++ch) {
                        put16(smem, OFF_U, part_at<PC>(tok, 0, ch0 + W / 8 * hh + ch, 8192), 24576, take8(d + 4 * ch));
                        put16(smem, OFF_U, part_at<PC>(tok, 1, ch0 + W / 8 * hh + ch, 8192), 24576, round8(d + 4 * ch));
                    }
                }
                fence_async_smem();
                tc_fence_before();
                mbar_arrive(&m->r);
                // V is free only now: R, which is stored, shows that it has been read
                // (an arrival right behind the loads let the next V overtake them)
                mbar_arrive(&m->v_free[c & 1]);
                wait(&m->tr, c, m, status, 13);
                __syncwarp();
                tc_fence_after();
#pragma unroll
                for (int hh = 0; hh < NH; ++hh) {
                    float2 f[W / 2];
                    tmem_sum<W, 2>(tl + D_TR + W * hh, PC, f);
#pragma unroll
                    for (int j = 0; j < W / 2; ++j) f[j] = __fadd2_rn(f[j], buf[W / 2 * hh + j]);
#pragma unroll
                    for (int ch = 0; ch < W / 8; ++ch) {
                        const int cc = ch0 + W / 8 * hh + ch;
                        put16(smem, OFF_UB, sw128(tok, cc), 8192, round8(f + 4 * ch));
                        if (DUMP) {
                            float2 e[4] = {f[4 * ch], f[4 * ch + 1], f[4 * ch + 2], f[4 * ch + 3]};
                            keep(slice_of(c) + kSliceU + tok * 64, W / 8 * hh + ch, take8(e));
                            keep(slice_of(c) + kSliceU + kTok + tok * 64, W / 8 * hh + ch, round8(e));
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) f[4 * ch + j] = __fmul2_rn(at2, f[4 * ch + j]);
                        put16(smem, OFF_U, part_at<PC>(tok, 0, cc, 8192), 24576, take8(f + 4 * ch));
                        put16(smem, OFF_U, part_at<PC>(tok, 1, cc, 8192), 24576, take8(f + 4 * ch));
                        put16(smem, OFF_U, part_at<PC>(tok, 2, cc, 8192), 24576, round8(f + 4 * ch));
                    }
                }
                fence_async_smem();
                tc_fence_before();
                mbar_arrive(&m->u);
            } else {
                tc_fence_before();
                mbar_arrive(&m->r);                // the previous chunk's P U has been read
                wait(&m->t_full[c & 1], c >> 1, m, status, 14);
                const float sa = q.scale * gt->a[tok];
                const float2 sa2 = make_float2(sa, sa);
                wait(&m->ks, c, m, status, 15);
                __syncwarp();
                tc_fence_after();
#pragma unroll
                for (int hh = 0; hh < NH; ++hh) {
                    tmem_sum<W, 2>(tl + D_KS + W * hh, PC, buf + W / 2 * hh);
#pragma unroll
                    for (int j = 0; j < W / 2; ++j) buf[W / 2 * hh + j] = __fmul2_rn(sa2, buf[W / 2 * hh + j]);
                }
                tc_fence_before();
                mbar_arrive(&m->u);
            }
            const float whole = gt->whole;
            const float2 w2 = make_float2(whole, whole);
            wait(&m->s, c, m, status, 16);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int hh = 0; hh < NH; ++hh) {
                float2 d[W / 2];
                tmem_sum<W, 3>(tl + D_S + W * hh, PC, d);
#pragma unroll
                for (int j = 0; j < W / 2; ++j) S[W / 2 * hh + j] = __ffma2_rn(w2, S[W / 2 * hh + j], d[j]);
            }
            // S takes the place of the U that P U reads
            wait(&m->o, c, m, status, 17);
            __syncwarp();
            if (c + 1 < w.nch) store_state(c + 1);
            if (!top) {
                tc_fence_after();
                const size_t o = (((size_t)w.b * q.seqlen + c * kC + tok) * q.nheads + w.h) * P + w.p0 + c0;
                const bool in = c * kC + tok < w.len && M3_SPAN(8, o, kCols, (long long)q.batch * q.seqlen * q.nheads * P);
                uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(q.y) + o);
#pragma unroll
                for (int hh = 0; hh < NH; ++hh) {
                    float2 f[W / 2];
                    tmem_sum<W, 1>(tl + D_TR + PC + W * hh, PC, f);
#pragma unroll
                    for (int j = 0; j < W / 2; ++j) f[j] = __fadd2_rn(buf[W / 2 * hh + j], f[j]);
                    if (!DUMP && in) {
#pragma unroll
                        for (int ch = 0; ch < W / 8; ++ch) dst[W / 8 * hh + ch] = round8(f + 4 * ch);
                    }
                }
            }
        }
        if (q.final_h && M3_SPAN(9, ho, kCols, ext_h)) {
#pragma unroll
            for (int c4 = 0; c4 < kCols / 4; ++c4)
                *reinterpret_cast<float4*>(q.final_h + ho + 4 * c4) =
                    make_float4(S[2 * c4].x, S[2 * c4].y, S[2 * c4 + 1].x, S[2 * c4 + 1].y);
        }
    } else if (warp <= 16) {
        // ------------------- T and the masked Q K^T of every other chunk
        const int group = (warp - 9) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const int pt = tid - 32 - kState - group * kPrep;
        const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16) + D_G + 64 * group;
        const int scr = OFF_SCR + group * SCR_BYTES;
        float* diag = reinterpret_cast<float*>(smem + scr + SCR_D);
        const int xo = OFF_X + group * 16384, lo = OFF_TL + group * 8192;
        const int tok = row & 63, blk = quarter & 1;       // the row's token; its 32-token block
        constexpr uint32_t idG = idesc_bf16(128, 64, 0, 0);
        // T and P of the records (one CTA of a head writes them)
        auto keep = [&](size_t at, int c, int r, int ch, uint4 v) {
            const size_t o = (bh * q.nck + c) * rec_elems(P) + at + r * 64 + ch * 8;
            if (w.p0 == 0 && M3_SPAN(11, o, 8, (long long)q.batch * q.nheads * q.nck * rec_elems(P)))
                *reinterpret_cast<uint4*>(q.rec + o) = v;
        };
        // P rows of tokens behind the end (other data, possibly not numbers) are recorded as zeros
        auto keep_p = [&](int c, int ch, const float2* e, bool live) {
            float2 f[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = live ? e[j] : make_float2(0.f, 0.f);
            keep(kRecP, c, tok, ch, take8(f));
            keep(kRecP + kTok, c, tok, ch, round8(f));
        };
        Raw raw = {};
        if (quarter == 2) raw = load_raw(q, w.b, w.h, w.len, group);
#pragma unroll 1
        for (int c = group; c < w.nch; c += 2) {
            const int kqo = OFF_KQ + (c % 3) * 32768;
            const int nt = min(kC, w.len - c * kC);
            Gates* gt = &m->gates[c % 5];
            // The gates take the place of chunk c - 5's.  This group has seen the
            // products of chunk c - 4 end (x_free below), so every chain thread
            // has begun that chunk and left the one before.
            if (quarter == 2) {
                make_gates(raw, gt);
                raw = load_raw(q, w.b, w.h, w.len, c + 2);       // the group's next
            }
            wait(&m->kq_full[c % 3], c / 3, m, status, 20);
            // K rows behind the sequence's end (other data, possibly not numbers)
            // must be zeros: K^T U sums over all rows of the tile
            if (nt < kC) {
                for (int e = pt; e < (kC - nt) * 16; e += kPrep) {
                    const int r = nt + (e >> 4), ch = e & 15;
                    put16(smem, kqo + (ch >> 3) * 16384, sw128(r, ch & 7), 16384, make_uint4(0u, 0u, 0u, 0u));
                }
                fence_async_smem();
            }
            tc_fence_before();
            group_sync(group);
            if (quarter == 1) {
                tc_fence_after();
                const uint64_t aKQ = sdesc(sbase + kqo, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const uint64_t o = aKQ + (kk >> 2) * 1024 + (kk & 3) * 2;
                    umma_one(tmem + D_G + 64 * group, o, o, idG, kk > 0);
                }
                commit_one(&m->g[group]);
            }
            const float2 G = gt->G[tok];
            const float f = row < 64 ? gt->beta[tok] : q.scale;
            const float fm = f * gt->mid[tok];             // (only rows of the second block use it)
            wait(&m->g[group], c >> 1, m, status, 22);
            __syncwarp();
            tc_fence_after();
            uint4 pk[8];                                   // P's row, rounded (rows 64..)
#pragma unroll
            for (int ch = 0; ch < 8; ++ch) pk[ch] = make_uint4(0u, 0u, 0u, 0u);
            if (blk == 1) {                                // the block left of the diagonal
                float d[32];
                tmem_ld32(tl, d);
                const float2 f2 = make_float2(fm, fm);
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    float2 e[4];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float4 u = *reinterpret_cast<const float4*>(&gt->mid[8 * ch + 4 * j]);
                        e[2 * j] = __fmul2_rn(__fmul2_rn(make_float2(u.x, u.y), f2), make_float2(d[8 * ch + 4 * j], d[8 * ch + 4 * j + 1]));
                        e[2 * j + 1] = __fmul2_rn(__fmul2_rn(make_float2(u.z, u.w), f2), make_float2(d[8 * ch + 4 * j + 2], d[8 * ch + 4 * j + 3]));
                    }
                    if (row < 64) {
                        put16(smem, scr + SCR_21, sw128(lane, ch), 4096, take8(e));
                        put16(smem, scr + SCR_21, sw128(lane, 4 + ch), 4096, round8(e));
                    } else {
                        pk[ch] = round8(e);
                        if (DUMP) keep_p(c, ch, e, tok < nt);
                    }
                }
            } else if (DUMP && row >= 64) {
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    keep(kRecP, c, tok, 4 + ch, make_uint4(0u, 0u, 0u, 0u));
                    keep(kRecP + kTok, c, tok, 4 + ch, make_uint4(0u, 0u, 0u, 0u));
                }
            }
            {                                              // the diagonal block
                float d[32];
                tmem_ld32(tl + 32 * blk, d);
                const int last = row < 64 ? lane - 1 : lane;
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    float2 e[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int k = 8 * ch + 2 * j;
                        const float4 u = *reinterpret_cast<const float4*>(&gt->G[32 * blk + k]);
                        const float x0 = ex2((G.x - u.x) + (G.y - u.y)), x1 = ex2((G.x - u.z) + (G.y - u.w));
                        e[j] = make_float2(k <= last ? f * x0 * d[k] : 0.f, k + 1 <= last ? f * x1 * d[k + 1] : 0.f);
                    }
                    if (row < 64) {
                        // rows 0..15: diagonal block 2 blk, columns 0..15; rows 16..31: block
                        // 2 blk + 1, columns 16..31, and the block left of it
                        const bool low = lane >= 16;
                        if (low == (ch >= 2)) {
                            float* dst = diag + (2 * blk + (ch >> 1)) * 256 + (8 * (ch & 1)) * 16 + (lane & 15);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                dst[2 * j * 16] = e[j].x;
                                dst[(2 * j + 1) * 16] = e[j].y;
                            }
                        } else if (low) {
                            put16(smem, scr + SCR_10, sw128(lane & 15, 4 * blk + ch), 2048, take8(e));
                            put16(smem, scr + SCR_10, sw128(lane & 15, 4 * blk + 2 + ch), 2048, round8(e));
                        }
                    } else {
                        if (blk) pk[4 + ch] = round8(e);
                        else pk[ch] = round8(e);
                        if (DUMP) keep_p(c, 4 * blk + ch, e, tok < nt);
                    }
                }
            }
            tc_fence_before();
            group_sync(group);
            float2 x[8];
            invert16(diag + 256 * quarter, x);             // (lanes 16.. repeat zeros)
            // T and P take the places of chunk c - 2's
            if (c >= 2) wait(&m->x_free[group], (c >> 1) - 1, m, status, 23);
            __syncwarp();
            const uint32_t th = sbase + xo, tlo = sbase + lo;
            if (lane < 16) {                               // row `lane` of the block's T^T
#pragma unroll
                for (int ch = 0; ch < 2; ++ch) {
                    const uint32_t o = sw128(16 * quarter + lane, 2 * quarter + ch);
                    sts128(th + o, take8(x + 4 * ch));
                    sts128(tlo + o, round8(x + 4 * ch));
                }
            }
            if (row >= 64) {
#pragma unroll
                for (int ch = 0; ch < 8; ++ch) put16(smem, xo, sw128(row, ch), 16384, pk[ch]);
            }
            group_sync(group);
            join16(th, tlo, sbase + scr + SCR_10, quarter);
            group_sync(group);
            join32(th, tlo, sbase + scr + SCR_21, quarter);
            group_sync(group);
            {
                // T - I from T^T, in place: rows 16 quarter .. of T, 8 x 8 blocks
                // exchanged; blocks right of the diagonal are zeros
                const int mi = lane >> 3, l7 = lane & 7;
                uint32_t rh[4][4], rl[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int ib = 2 * quarter + (i >> 1), jb = 4 * (i & 1) + mi;
                    if (4 * (i & 1) <= ib) {
                        const uint32_t o = sw128(8 * jb + l7, ib);
                        ldsm4t(rh[i], th + o);
                        ldsm4t(rl[i], tlo + o);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = 4 * (i & 1) + e;
                        if (j > ib) rh[i][e] = rl[i][e] = 0u;
                        if (j == ib && (lane >> 3) == (lane & 3)) rh[i][e] &= (lane & 4) ? 0x0000ffffu : 0xffff0000u;
                    }
                }
                group_sync(group);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int ib = 2 * quarter + (i >> 1), jb = 4 * (i & 1) + mi;
                    const uint32_t o = sw128(8 * ib + l7, jb);
                    stsm4(th + o, rh[i]);
                    stsm4(tlo + o, rl[i]);
                    if (DUMP && w.p0 == 0) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const size_t at = (bh * q.nck + c) * rec_elems(P) + kRecT + (8 * ib + (lane >> 2)) * 64 +
                                              8 * (4 * (i & 1) + e) + 2 * (lane & 3);
                            if (M3_SPAN(12, at + kTok, 2, (long long)q.batch * q.nheads * q.nck * rec_elems(P))) {
                                *reinterpret_cast<uint32_t*>(q.rec + at) = rh[i][e];
                                *reinterpret_cast<uint32_t*>(q.rec + at + kTok) = rl[i][e];
                            }
                        }
                    }
                }
            }
            fence_async_smem();
            mbar_arrive(&m->t_full[group]);
        }
        if (quarter == 1) {
            __syncwarp();
            commit_one(&m->drain[group]);
            mbar_wait_flag(&m->drain[group], 0, &m->drain_flag, nullptr, 0);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------- loads
        if (lane == 0) {
            for (int c = 0; c < w.nch; ++c) {
                const uint32_t kq = sbase + OFF_KQ + (c % 3) * 32768;
                if (c >= 3) wait(&m->kq_free[c % 3], c / 3 - 1, m, status, 30);
                // chunk c + 3 into L2: its load waits for a stage, and then finds it there
                if (c + 3 < w.nch) {
                    const int t = (c + 3) * kC;
                    tma_prefetch_5d(&tmK, 0, 0, w.g, t, w.b);
                    tma_prefetch_5d(&tmK, 64, 0, w.g, t, w.b);
                    tma_prefetch_5d(&tmQ, 0, 0, w.g, t, w.b);
                    tma_prefetch_5d(&tmQ, 64, 0, w.g, t, w.b);
                    tma_prefetch_5d(&tmV, w.p0 & ~63, 0, w.h, t, w.b);
                }
                uint64_t* bar = &m->kq_full[c % 3];
                mbar_expect_tx(bar, 32768);
                tma_load_5d(kq, &tmK, bar, 0, 0, w.g, c * kC, w.b);
                tma_load_5d(kq + 16384, &tmK, bar, 64, 0, w.g, c * kC, w.b);
                tma_load_5d(kq + 8192, &tmQ, bar, 0, 0, w.g, c * kC, w.b);
                tma_load_5d(kq + 24576, &tmQ, bar, 64, 0, w.g, c * kC, w.b);
                if (c >= 2) wait(&m->v_free[c & 1], (c >> 1) - 1, m, status, 31);
                bar = &m->v_full[c & 1];
                mbar_expect_tx(bar, 8192);
                tma_load_5d(sbase + OFF_V + (c & 1) * 8192, &tmV, bar, w.p0 & ~63, 0, w.h, c * kC, w.b);
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

template <int PC, bool DUMP>
static cudaError_t launch_pc(const CUtensorMap& mK, const CUtensorMap& mQ, const CUtensorMap& mV, const m3_dims& d,
                             const DeltaParams& q, int* status, cudaStream_t st) {
    using namespace dtc;
    const cudaError_t e = cudaFuncSetAttribute(delta_tc_kernel<PC, DUMP>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((long long)d.batch * d.nheads * (d.headdim / PC));
    delta_tc_kernel<PC, DUMP><<<grid, kThreads, SMEM_BYTES, st>>>(mK, mQ, mV, q, status);
    return cudaGetLastError();
}

cudaError_t launch_delta_tc(const m3_dims& d, const DeltaParams& q, int* status, cudaStream_t st) {
    using namespace dtc;
    CUtensorMap mK, mQ, mV;
    if (!make_tile_map(&mK, q.k, kN, 1, d.ngroups, d.seqlen, d.batch, kC) ||
        !make_tile_map(&mQ, q.q, kN, 1, d.ngroups, d.seqlen, d.batch, kC) ||
        !make_tile_map(&mV, q.v, d.headdim, 1, d.nheads, d.seqlen, d.batch, kC))
        return cudaErrorInvalidValue;
    const char* env = getenv("M3_DTC_PC");
    const int pc = env ? atoi(env) : q.rec ? 32 : 64;
    if (q.rec) {
        if (pc == 64) return launch_pc<64, true>(mK, mQ, mV, d, q, status, st);
        return launch_pc<32, true>(mK, mQ, mV, d, q, status, st);
    }
    if (pc == 64) return launch_pc<64, false>(mK, mQ, mV, d, q, status, st);
    if (pc == 32) return launch_pc<32, false>(mK, mQ, mV, d, q, status, st);
    return launch_pc<16, false>(mK, mQ, mV, d, q, status, st);
}

}  // namespace m3

M3_BOUNDS_EXPORT(delta_tc)
