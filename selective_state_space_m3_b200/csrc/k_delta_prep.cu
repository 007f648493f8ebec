// k_delta_prep.cu -- what the chunked gated delta rule needs of a chunk that
// does not depend on the state (sm_100a; bfloat16 io, N = 128), all chunks at
// once: gates, T = (I + A)^{-1} and P = scale Gam o Q K^T (notation of
// k_delta_tc.cu), as the images of shared memory that the chain loads.
//
// One CTA of four warps a chunk of a (batch, head).  One tcgen05 product of the
// stacked rows [K; Q] with K gives both Gram matrices; a thread has one row of
// them.  T: the four 16 x 16 diagonal blocks by substitution in float32 (a lane
// per column), the blocks below them by warp-level products whose accumulators
// are the next product's operand as they stand (hi and lo bfloat16 parts, three
// products for one); kept transposed until the end.  K and Q are dead after the
// Gram product, and their place takes the images: 37 KB a CTA, five an SM, whose
// loads, products and substitutions overlap.
//
// Bound by memory: 32 KB in and 25 KB out a chunk; 4096 chunks take 51 us
// (4.7 TB/s), 16384 chunks 186 us (5.1 TB/s).  In the chain itself this work
// took half of every chunk's time (32768 tokens 1.45 ms instead of 0.85).
//
// Every wait on an mbarrier is bounded (1 s); on expiry the kernel records
// M3_ERR_DEVICE_TIMEOUT in the workspace status word and runs out without
// further waiting.
#define M3_BOUNDS_FILE 14
#include "m3_bounds.cuh"
#include "delta_tc.cuh"

namespace m3 {

bool make_tile_map(CUtensorMap* map, const void* base, int inner, int R, int grp, int L, int batch, int T);

namespace dprep {

using namespace dtc;

constexpr int kThreads = 128;
// K, Q (two 64-column atoms, rows 0..63 K, 64..127 Q); then X, TL and scratch
constexpr int OFF_X = 0, OFF_TL = 16384;
constexpr int OFF_D = 24576;                    // A's 16 x 16 diagonal blocks, float32, by columns (4 KB)
constexpr int OFF_21 = OFF_D + 4096;            // A's lower left 32 x 32 block, hi and lo side by side (4 KB)
constexpr int OFF_10 = 32768;                   // its two 16 x 16 blocks under the diagonal, hi, lo, hi, lo (2 KB)
constexpr int OFF_MISC = OFF_10 + 2048;

struct Misc {
    Gates gates;
    uint64_t full, g;
    uint32_t tmem_base;
    int abort_flag, drain_flag, pad;
};
constexpr int SMEM_BYTES = OFF_MISC + (int)sizeof(Misc) + 1024;

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


__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}

template <bool GRAD>
__global__ void __launch_bounds__(kThreads, 5)
    delta_prep_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ, DeltaParams q,
                      int* status) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (su32(smem_raw) & 1023u)) & 1023u);
    Misc* m = reinterpret_cast<Misc*>(smem + OFF_MISC);
    const uint32_t sbase = su32(smem);
    if (!M3_SPAN(1, smem - smem_raw, OFF_MISC + (int)sizeof(Misc), dyn_smem_bytes())) return;
    const int tid = threadIdx.x, quarter = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31, row = tid;
    const int bh = blockIdx.x / q.nck, c = blockIdx.x % q.nck;
    const int b = bh / q.nheads, h = bh % q.nheads, g = h / (q.nheads / q.ngroups);
    if (q.flags && blockIdx.x == 0)                // no state has been handed over yet (the chain is the next kernel)
        for (int e = tid; e < kDeltaSlots; e += kThreads) q.flags[e] = 0;
    int len = q.seqlen;
    if (q.lengths && M3_IN(3, b, q.batch)) len = min(max(q.lengths[b], 0), q.seqlen);
    const int nt = min(kC, len - c * kC);
    if (nt <= 0) return;                           // behind the end
    if (tid == 0) {
        mbar_init(&m->full, 1);
        mbar_init(&m->g, 1);
        m->abort_flag = 0;
        m->drain_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
        mbar_expect_tx(&m->full, 32768);
        tma_load_5d(sbase, &tmK, &m->full, 0, 0, g, c * kC, b);
        tma_load_5d(sbase + 16384, &tmK, &m->full, 64, 0, g, c * kC, b);
        tma_load_5d(sbase + 8192, &tmQ, &m->full, 0, 0, g, c * kC, b);
        tma_load_5d(sbase + 24576, &tmQ, &m->full, 64, 0, g, c * kC, b);
    }
    __syncwarp();
    if (quarter == 0) {
        tmem_alloc(&m->tmem_base, 64);
        tmem_relinquish();
    }
    if (quarter == 2) make_gates(load_raw(q, b, h, len, c), &m->gates);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = m->tmem_base, tl = tmem + ((uint32_t)(quarter * 32) << 16);
    const Gates* gt = &m->gates;
    const int tok = row & 63, blk = quarter & 1;       // the row's token; its 32-token block
    mbar_wait_flag(&m->full, 0, &m->abort_flag, status, 1);
    if (quarter == 1) {
        __syncwarp();
        constexpr uint32_t idG = idesc_bf16(128, 64, 0, 0);
        const uint64_t aKQ = sdesc(sbase, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
            const uint64_t o = aKQ + (kk >> 2) * 1024 + (kk & 3) * 2;
            umma_one(tmem, o, o, idG, kk > 0);
        }
        commit_one(&m->g);
    }
    const float2 G = gt->G[tok];
    const float f = row < 64 ? gt->beta[tok] : q.scale;
    const float fm = f * gt->mid[tok];             // (only rows of the second block use it)
    // nothing may write over K and Q before the product has read them
    if (!mbar_wait_flag(&m->g, 0, &m->abort_flag, status, 2)) mbar_wait_flag(&m->g, 0, &m->drain_flag, nullptr, 0);
    __syncwarp();
    tc_fence_after();
    __nv_bfloat16* rec = q.rec + (size_t)blockIdx.x * rec_elems(q.headdim, GRAD);
    const long long ext_rec = (long long)q.batch * q.nheads * q.nck * (long long)rec_elems(q.headdim, GRAD);
    // what the rounding left of P, 16 bytes of this row
    auto keep_low = [&](int ch, uint4 v) {
        const size_t o = kRecPL + sw128(tok, ch) / 2;
        if (M3_SPAN(11, rec - q.rec + o, 8, ext_rec)) *reinterpret_cast<uint4*>(rec + o) = v;
    };
    // columns and rows behind the end count as zero (their K and Q are other data, possibly not numbers)
    const bool live = tok < nt;
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
#pragma unroll
            for (int j = 0; j < 4; ++j) e[j] = live ? e[j] : make_float2(0.f, 0.f);    // (a live row's columns here are live)
            if (row < 64) {
                put16(smem, OFF_21, sw128(lane, ch), 4096, take8(e));
                put16(smem, OFF_21, sw128(lane, 4 + ch), 4096, round8(e));
            } else {
                pk[ch] = take8(e);
                if (GRAD) keep_low(ch, round8(e));
            }
        }
    } else if (GRAD && row >= 64) {
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) keep_low(4 + ch, make_uint4(0u, 0u, 0u, 0u));
    }
    {                                              // the diagonal block
        float d[32];
        tmem_ld32(tl + 32 * blk, d);
        const int last = !live ? -1 : row < 64 ? lane - 1 : lane;
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
                    float* dst = reinterpret_cast<float*>(smem + OFF_D) + (2 * blk + (ch >> 1)) * 256 + (8 * (ch & 1)) * 16 + (lane & 15);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        dst[2 * j * 16] = e[j].x;
                        dst[(2 * j + 1) * 16] = e[j].y;
                    }
                } else if (low) {
                    put16(smem, OFF_10, sw128(lane & 15, 4 * blk + ch), 2048, take8(e));
                    put16(smem, OFF_10, sw128(lane & 15, 4 * blk + 2 + ch), 2048, round8(e));
                }
            } else {
                const uint4 v = take8(e);
                if (blk) pk[4 + ch] = v;
                else pk[ch] = v;
                if (GRAD) keep_low(4 * blk + ch, round8(e));
            }
        }
    }
    if (row >= 64) {
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) put16(smem, OFF_X, sw128(row, ch), 16384, pk[ch]);
    }
    __syncthreads();
    float2 x[8];
    invert16(reinterpret_cast<float*>(smem + OFF_D) + 256 * quarter, x);     // (lanes 16.. repeat zeros)
    const uint32_t th = sbase + OFF_X, tlo = sbase + OFF_TL;
    if (lane < 16) {                               // row `lane` of the block's T^T
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
            const uint32_t o = sw128(16 * quarter + lane, 2 * quarter + ch);
            sts128(th + o, take8(x + 4 * ch));
            sts128(tlo + o, round8(x + 4 * ch));
        }
    }
    __syncthreads();
    join16(th, tlo, sbase + OFF_10, quarter);
    __syncthreads();
    join32(th, tlo, sbase + OFF_21, quarter);
    __syncthreads();
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
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t o = sw128(8 * (2 * quarter + (i >> 1)) + l7, 4 * (i & 1) + mi);
            stsm4(th + o, rh[i]);
            stsm4(tlo + o, rl[i]);
        }
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && M3_SPAN(12, rec - q.rec, kRecPL, ext_rec)) {
        bulk_store(rec + kRecX, sbase, 24576);
        bulk_store(rec + kRecGates, su32(static_cast<ChainGates*>(&m->gates)), sizeof(ChainGates));
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    if (quarter == 0) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 64);
    }
}

}  // namespace dprep

cudaError_t launch_delta_prep(const m3_dims& d, const DeltaParams& q, bool grad, int* status, cudaStream_t st) {
    using namespace dprep;
    CUtensorMap mK, mQ;
    if (!make_tile_map(&mK, q.k, kN, 1, d.ngroups, d.seqlen, d.batch, kC) ||
        !make_tile_map(&mQ, q.q, kN, 1, d.ngroups, d.seqlen, d.batch, kC))
        return cudaErrorInvalidValue;
    const void* kernel = grad ? (const void*)delta_prep_kernel<true> : (const void*)delta_prep_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((long long)d.batch * d.nheads * q.nck);
    if (grad) delta_prep_kernel<true><<<grid, kThreads, SMEM_BYTES, st>>>(mK, mQ, q, status);
    else delta_prep_kernel<false><<<grid, kThreads, SMEM_BYTES, st>>>(mK, mQ, q, status);
    return cudaGetLastError();
}

}  // namespace m3

M3_BOUNDS_EXPORT(delta_prep)
