// k_delta_rev.cu -- the chain of the gated delta rule's gradient, from the last
// chunk to the first (sm_100a tensor cores; bfloat16 io, N = 128).  Notation and
// formulas: k_delta_bwd_tc.cu.  A chunk (dS' the gradient of the state behind it):
//   dU = P^T dY + e^{G_C-G} o (K dS')
//   dR = dU + (T - I)^T dU               dV = beta o dR
//   dS = e^{G_C} dS' + Q^T (scale e^G o dY) - K^T (beta e^G o dR)
// P^T dY and Q^T (..) do not depend on dS' and are issued ahead; the chain of a
// chunk is K dS', T^T dU and K^T (..), as in the prefill, whose layout this
// kernel shares (k_delta_tc.cu): one CTA per (batch, head, PC columns), products
// with M = 128 rows, split operands side by side as columns, dS in registers.
//   warp 0     products (one elected lane)
//   warps 1..  the arithmetic: rows 0..63 of the accumulators (tokens) make dU and
//              dR, rows 64..127 have no tokens: their warps bring dY in, scaled and
//              split, a chunk ahead; dS is everybody's
//   last warp  loads, two chunks ahead
// Recorded for k_delta_bwd_tc.cu: dR and the gradient of the state behind every
// chunk.  The transposed products read the images of T and P that the prefill
// uses, as MN-major operands (64 of the 128 rows are other data and unused).
// Bound by the chain's latency: 2.1 us a chunk with 32 columns a CTA, 1.7 with 16
// (tensor pipe 22 and 14 % active).
//
// Every wait on an mbarrier is bounded (1 s); on expiry the kernel records
// M3_ERR_DEVICE_TIMEOUT in the workspace status word and runs out without
// further waiting.
#define M3_BOUNDS_FILE 15
#include "m3_bounds.cuh"
#include "delta_tc.cuh"

namespace m3 {

bool make_tile_map(CUtensorMap* map, const void* base, int inner, int R, int grp, int L, int batch, int T);

namespace drev {

using namespace dtc;

// Column groups of the arithmetic, four warps each: 8 columns a thread
template <int PC> constexpr int kState = 128 * (PC / 8);           // threads of the chain
template <int PC> constexpr int kThreads = 32 + kState<PC> + 32;

// a stage: K, Q (two 64-column atoms, rows 0..63 K, 64..127 Q), then a record's
// X, TL, gates and PL as they stand there
constexpr int ST_X = 32768, ST_TL = ST_X + 16384, ST_GATES = ST_TL + 8192, ST_PL = ST_GATES + 1024;
constexpr int kRecBytes = 33792, kStage = ST_PL + 8192;
static_assert(kStage == ST_X + kRecBytes && kRecBytes == 2 * (int)kRecSlice, "a record's head");
constexpr int OFF_DY = 2 * kStage;              // 2 x 8 KB: dY as loaded
constexpr int OFF_DS = OFF_DY + 2 * 8192;       // dS hi, lo (16 KB: rows n)
constexpr int OFF_DU = OFF_DS + 16384;          // hi, lo (8 KB each: rows t): dU,
constexpr int OFF_DR = OFF_DU + 8192;           //   - beta e^G dR,
constexpr int OFF_DYS = OFF_DR + 8192;          //   scale e^G dY;
constexpr int OFF_DYR = OFF_DYS + 8192;         //   and the CTA's columns of dY
constexpr int OFF_MISC = OFF_DYR + 8192;
// TMEM columns: K dS' in two parts, P^T dY, T^T dU in two parts, dS's update in two parts
constexpr uint32_t D_K = 0, D_U0 = 64, D_T = 96, D_S = 160;

struct Misc {
    uint64_t full[2], freed[2], dy_full[2], dy_free[2];
    uint64_t s_ready, ks, r, tr, u, s, dy, a, drain;
    uint32_t tmem_base;
    int abort_flag, drain_flag, pad;
};
constexpr int SMEM_BYTES = OFF_MISC + (int)sizeof(Misc) + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory of the reverse chain");

__device__ __forceinline__ bool wait(uint64_t* b, int phase, Misc* m, int* status, int where) {
    return mbar_wait_flag(b, (uint32_t)(phase & 1), &m->abort_flag, status, where);
}

template <int PC>
__global__ void __launch_bounds__(kThreads<PC>, 1)
    delta_rev_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmY, DeltaParams q, int* status) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (su32(smem_raw) & 1023u)) & 1023u);
    Misc* m = reinterpret_cast<Misc*>(smem + OFF_MISC);
    const uint32_t sbase = su32(smem);
    if (!M3_SPAN(1, smem - smem_raw, OFF_MISC + (int)sizeof(Misc), dyn_smem_bytes())) return;
    const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
    const Where w = where_is<PC>(q, blockIdx.x);
    const int P = q.headdim;
    const size_t bh = (size_t)w.b * q.nheads + w.h, rec = rec_elems(P, true);
    [[maybe_unused]] const long long ext_rec = (long long)q.batch * q.nheads * q.nck * (long long)rec;
    const int nch = w.nch;                         // iteration i takes chunk nch - 1 - i

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m->full[i], 1);
            mbar_init(&m->freed[i], 1);
            mbar_init(&m->dy_full[i], 1);
            mbar_init(&m->dy_free[i], kState<PC> / 2);
        }
        mbar_init(&m->s_ready, kState<PC>);
        mbar_init(&m->ks, 1);
        mbar_init(&m->r, kState<PC> / 2);
        mbar_init(&m->tr, 1);
        mbar_init(&m->u, kState<PC>);
        mbar_init(&m->s, 1);
        mbar_init(&m->dy, kState<PC> / 2);
        mbar_init(&m->a, 1);
        mbar_init(&m->drain, 1);
        m->abort_flag = 0;
        m->drain_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
    }
    if (warp == 0) {
        tmem_alloc(&m->tmem_base, 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = m->tmem_base;

    if (warp == 0) {
        // ------------------------------------------------------- products
        // (descriptor starts count 16 bytes)
        constexpr uint32_t idK = idesc_bf16(128, 2 * PC, 0, 1);    // A K-major, B MN-major
        constexpr uint32_t idM = idesc_bf16(128, 2 * PC, 1, 1);    // A MN-major
        constexpr uint32_t idM1 = idesc_bf16(128, PC, 1, 1);
        const uint64_t bDS = sdesc(sbase + OFF_DS, 16384, 1024), bDU = sdesc(sbase + OFF_DU, 8192, 1024);
        const uint64_t bDR = sdesc(sbase + OFF_DR, 8192, 1024), bDYS = sdesc(sbase + OFF_DYS, 8192, 1024);
        const uint64_t bDYR = sdesc(sbase + OFF_DYR, 8192, 1024);
        // P^T dY of iteration i
        auto head = [&](int i) {
            const uint32_t st = sbase + (i & 1) * kStage;
            const uint64_t aP = sdesc(st + ST_X + 8192, 8192, 1024), aPL = sdesc(st + ST_PL, 8192, 1024);
            wait(&m->full[i & 1], i >> 1, m, status, 1);
            wait(&m->dy, i, m, status, 2);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) umma_one(tmem + D_U0, aP + kk * 128, bDYR + kk * 128, idM1, kk > 0);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) umma_one(tmem + D_U0, aPL + kk * 128, bDYR + kk * 128, idM1, 1);
            commit_one(&m->a);
        };
        if (nch > 0) head(0);
        for (int i = 0; i < nch; ++i) {
            const uint32_t st = sbase + (i & 1) * kStage;
            const uint64_t aKQ = sdesc(st, 16, 1024), aKT = sdesc(st, 16384, 1024), aQT = sdesc(st + 8192, 16384, 1024);
            const uint64_t aT = sdesc(st + ST_X, 8192, 1024), aTL = sdesc(st + ST_TL, 8192, 1024);
            wait(&m->s_ready, i, m, status, 3);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                umma_one(tmem + D_K, aKQ + (kk >> 2) * 1024 + (kk & 3) * 2, bDS + kk * 128, idK, kk > 0);
            commit_one(&m->ks);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) umma_one(tmem + D_S, aQT + kk * 128, bDYS + kk * 128, idM, kk > 0);
            wait(&m->r, i, m, status, 4);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) umma_one(tmem + D_T, aT + kk * 128, bDU + kk * 128, idM, kk > 0);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) umma_one(tmem + D_T, aTL + kk * 128, bDU + kk * 128, idM1, 1);
            commit_one(&m->tr);
            wait(&m->u, i, m, status, 5);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) umma_one(tmem + D_S, aKT + kk * 128, bDR + kk * 128, idM, 1);
            commit_one(&m->s);
            commit_one(&m->freed[i & 1]);
            if (i + 1 < nch) head(i + 1);
        }
        commit_one(&m->drain);
        mbar_wait_flag(&m->drain, 0, &m->drain_flag, nullptr, 0);
        __syncwarp();
    } else if (warp <= kState<PC> / 32) {
        // ------------------------------------------------- the arithmetic
        const int wk = tid - 32, wg = wk >> 7, quarter = warp & 3, row = quarter * 32 + lane, c0 = wg * 8;
        const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16) + c0;
        const bool top = quarter < 2;
        const int tok = row & 63, H = q.nheads;
        [[maybe_unused]] const long long ext_h = (long long)q.batch * H * kN * P, ext_v = (long long)q.batch * q.seqlen * H * P;
        const size_t ho = (bh * kN + row) * P + w.p0 + c0;
        float2 dS[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (q.d_final_h && M3_SPAN(2, ho + 4 * j, 4, ext_h)) v = *reinterpret_cast<const float4*>(q.d_final_h + ho + 4 * j);
            dS[2 * j] = make_float2(v.x, v.y);
            dS[2 * j + 1] = make_float2(v.z, v.w);
        }
        // this thread's 8 columns of row r of a recorded part of chunk c with `rows` rows
        auto keep = [&](int c, size_t at, int rows, int r, uint4 v) {
            const size_t o = (bh * q.nck + c) * rec + kRecSlice + (size_t)(w.p0 >> 6) * kSliceElems + at +
                             rec_at(rows, r, (w.p0 & 63) + c0);
            if (M3_SPAN(3, o, 8, ext_rec)) *reinterpret_cast<uint4*>(q.rec + o) = v;
        };
        // dS into shared memory and, as the gradient of the state behind chunk c, into the record
        auto store_ds = [&](int c) {
            float2 f[4] = {dS[0], dS[1], dS[2], dS[3]};
            const uint4 hi = take8(f), lo = round8(f);
            put16(smem, OFF_DS, part_at<PC>(row, 0, c0 / 8, 16384), 16384, hi);
            put16(smem, OFF_DS, part_at<PC>(row, 1, c0 / 8, 16384), 16384, lo);
            fence_async_smem();
            tc_fence_before();
            mbar_arrive(&m->s_ready);
            keep(c, kSliceDS, 128, row, hi);
            keep(c, kSliceDS + kSt, 128, row, lo);
        };
        // dY of iteration i: as it is and scaled by scale e^G; rows behind the end
        // (other data, possibly not numbers) count as zero
        auto bring_dy = [&](int i) {
            const int c = nch - 1 - i, st = (i & 1) * kStage;
            wait(&m->full[i & 1], i >> 1, m, status, 10);
            wait(&m->dy_full[i & 1], i >> 1, m, status, 11);
            const bool in = c * kC + tok < w.len;
            const uint32_t o = sw128(tok, (w.p0 & 63) / 8 + c0 / 8);
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (in && M3_SPAN(4, o, 16, 8192)) v = *reinterpret_cast<const uint4*>(smem + OFF_DY + (i & 1) * 8192 + o);
            put16(smem, OFF_DYR, sw128(tok, c0 / 8), 8192, v);
            const float sa = q.scale * reinterpret_cast<const ChainGates*>(smem + st + ST_GATES)->a[tok];
            const float2 sa2 = make_float2(sa, sa);
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
            float2 f[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                f[j] = __fmul2_rn(sa2, make_float2(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xffff0000u)));
            put16(smem, OFF_DYS, part_at<PC>(tok, 0, c0 / 8, 8192), 8192, take8(f));
            put16(smem, OFF_DYS, part_at<PC>(tok, 1, c0 / 8, 8192), 8192, round8(f));
            const int nt = w.len - c * kC;
            if (nt < kC) {
                // K and Q rows behind the end must be zeros: K^T (..) and Q^T (..) sum over all rows of the tile
                for (int e = wg * 64 + tok; e < (kC - nt) * 32; e += kState<PC> / 2) {
                    const int r = nt + (e >> 5), ch = e & 31;      // 16 groups of K, 16 of Q
                    put16(smem, st + ((ch >> 3) & 1) * 16384, sw128(r + (ch >> 4) * 64, ch & 7), 16384, make_uint4(0u, 0u, 0u, 0u));
                }
            }
            fence_async_smem();
            tc_fence_before();
            mbar_arrive(&m->dy);
            mbar_arrive(&m->dy_free[i & 1]);
        };
        if (nch > 0) {
            if (!top) bring_dy(0);
            store_ds(nch - 1);
        }
#pragma unroll 1
        for (int i = 0; i < nch; ++i) {
            const int c = nch - 1 - i;
            const ChainGates* gt = reinterpret_cast<const ChainGates*>(smem + (i & 1) * kStage + ST_GATES);
            wait(&m->full[i & 1], i >> 1, m, status, 12);
            const float whole = gt->whole;
            if (top) {
                const bool in = c * kC + tok < w.len;
                const float be = gt->beta[tok], at = gt->at[tok], ra = -be * gt->a[tok];
                const float2 at2 = make_float2(at, at), be2 = make_float2(be, be), ra2 = make_float2(ra, ra);
                wait(&m->a, i, m, status, 13);
                wait(&m->ks, i, m, status, 14);
                __syncwarp();
                tc_fence_after();
                float2 dU[4], f[4], d[4];
                tmem_sum<8, 2>(tl + D_K, PC, f);
                tmem_sum<8, 1>(tl + D_U0, PC, d);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    dU[j] = in ? __ffma2_rn(at2, f[j], d[j]) : make_float2(0.f, 0.f);
                    f[j] = dU[j];
                }
                put16(smem, OFF_DU, part_at<PC>(tok, 0, c0 / 8, 8192), 8192, take8(f));
                put16(smem, OFF_DU, part_at<PC>(tok, 1, c0 / 8, 8192), 8192, round8(f));
                fence_async_smem();
                tc_fence_before();
                mbar_arrive(&m->r);
                wait(&m->tr, i, m, status, 15);
                __syncwarp();
                tc_fence_after();
                tmem_sum<8, 2>(tl + D_T, PC, f);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    d[j] = __fadd2_rn(f[j], dU[j]);
                    f[j] = __fmul2_rn(ra2, d[j]);
                }
                put16(smem, OFF_DR, part_at<PC>(tok, 0, c0 / 8, 8192), 8192, take8(f));
                put16(smem, OFF_DR, part_at<PC>(tok, 1, c0 / 8, 8192), 8192, round8(f));
                fence_async_smem();
                tc_fence_before();
                arrive_after(&m->u, __float_as_uint(whole));
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = __fmul2_rn(be2, d[j]);
                const size_t vo = (((size_t)w.b * q.seqlen + c * kC + tok) * H + w.h) * P + w.p0 + c0;
                if (in && M3_SPAN(5, vo, 8, ext_v)) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(q.dv) + vo) = round8(f);
                keep(c, kSliceDR, 64, tok, take8(d));
                keep(c, kSliceDR + kTok, 64, tok, round8(d));
            } else {
                arrive_after(&m->u, __float_as_uint(whole));       // (the stage is free once everybody has its gates)
                if (i + 1 < nch) {
                    // dY's places are free once this chunk's products with it are done
                    wait(&m->tr, i, m, status, 16);
                    bring_dy(i + 1);
                }
            }
            wait(&m->s, i, m, status, 17);
            __syncwarp();
            tc_fence_after();
            {
                float2 d[4];
                tmem_sum<8, 2>(tl + D_S, PC, d);
                const float2 w2 = make_float2(whole, whole);
#pragma unroll
                for (int j = 0; j < 4; ++j) dS[j] = __ffma2_rn(w2, dS[j], d[j]);
            }
            if (c > 0) store_ds(c - 1);
        }
        if (q.d_init_h && M3_SPAN(6, ho, 8, ext_h)) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                *reinterpret_cast<float4*>(q.d_init_h + ho + 4 * j) =
                    make_float4(dS[2 * j].x, dS[2 * j].y, dS[2 * j + 1].x, dS[2 * j + 1].y);
        }
        // tokens behind the end of the sequence have no gradient
        for (size_t e = (size_t)w.len * (PC / 8) + wk; e < (size_t)q.seqlen * (PC / 8); e += kState<PC>) {
            const size_t vo = (((size_t)w.b * q.seqlen + e / (PC / 8)) * H + w.h) * P + w.p0 + 8 * (e % (PC / 8));
            if (M3_SPAN(7, vo, 8, ext_v))
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(q.dv) + vo) = make_uint4(0u, 0u, 0u, 0u);
        }
    } else {
        // ------------------------------------------------------------- loads
        if (lane == 0) {
            int asked = 0, asked_y = 0;            // (fewer than the chunks after a wait that ran out)
            for (int i = 0; i < nch; ++i) {
                const int c = nch - 1 - i;
                const uint32_t st = sbase + (i & 1) * kStage;
                if (i >= 2 && !wait(&m->freed[i & 1], (i >> 1) - 1, m, status, 30)) break;
                // the chunk after next into L2: its load waits for a stage, and then finds it there
                if (c >= 2) {
                    const int t = (c - 2) * kC;
                    tma_prefetch_5d(&tmK, 0, 0, w.g, t, w.b);
                    tma_prefetch_5d(&tmK, 64, 0, w.g, t, w.b);
                    tma_prefetch_5d(&tmQ, 0, 0, w.g, t, w.b);
                    tma_prefetch_5d(&tmQ, 64, 0, w.g, t, w.b);
                    tma_prefetch_5d(&tmY, w.p0 & ~63, 0, w.h, t, w.b);
                    bulk_prefetch(q.rec + (bh * q.nck + c - 2) * rec, kRecBytes);
                }
                uint64_t* bar = &m->full[i & 1];
                M3_NOTE(8, (bh * q.nck + c) * rec + kRecSlice - 1, ext_rec);
                ++asked;
                mbar_expect_tx(bar, 32768 + kRecBytes);
                tma_load_5d(st, &tmK, bar, 0, 0, w.g, c * kC, w.b);
                tma_load_5d(st + 16384, &tmK, bar, 64, 0, w.g, c * kC, w.b);
                tma_load_5d(st + 8192, &tmQ, bar, 0, 0, w.g, c * kC, w.b);
                tma_load_5d(st + 24576, &tmQ, bar, 64, 0, w.g, c * kC, w.b);
                bulk_load(st + ST_X, q.rec + (bh * q.nck + c) * rec, kRecBytes, bar);
                if (i >= 2 && !wait(&m->dy_free[i & 1], (i >> 1) - 1, m, status, 31)) break;
                ++asked_y;
                bar = &m->dy_full[i & 1];
                mbar_expect_tx(bar, 8192);
                tma_load_5d(sbase + OFF_DY + (i & 1) * 8192, &tmY, bar, w.p0 & ~63, 0, w.h, c * kC, w.b);
            }
            // nothing may still be on its way into shared memory when the CTA ends
            for (int i = max(0, asked - 2); i < asked; ++i) mbar_wait_flag(&m->full[i & 1], (i >> 1) & 1, &m->drain_flag, nullptr, 0);
            for (int i = max(0, asked_y - 2); i < asked_y; ++i)
                mbar_wait_flag(&m->dy_full[i & 1], (i >> 1) & 1, &m->drain_flag, nullptr, 0);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 256);
}

template <int PC>
static cudaError_t launch(const CUtensorMap& mK, const CUtensorMap& mQ, const CUtensorMap& mY, const m3_dims& d,
                          const DeltaParams& q, int* status, cudaStream_t st) {
    const cudaError_t e = cudaFuncSetAttribute(delta_rev_kernel<PC>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((long long)d.batch * d.nheads * (d.headdim / PC));
    delta_rev_kernel<PC><<<grid, kThreads<PC>, SMEM_BYTES, st>>>(mK, mQ, mY, q, status);
    return cudaGetLastError();
}

}  // namespace drev

cudaError_t launch_delta_rev(const m3_dims& d, const DeltaParams& q, int columns, int* status, cudaStream_t st) {
    using namespace drev;
    CUtensorMap mK, mQ, mY;
    if (!make_tile_map(&mK, q.k, kN, 1, d.ngroups, d.seqlen, d.batch, kC) ||
        !make_tile_map(&mQ, q.q, kN, 1, d.ngroups, d.seqlen, d.batch, kC) ||
        !make_tile_map(&mY, q.dy, d.headdim, 1, d.nheads, d.seqlen, d.batch, kC))
        return cudaErrorInvalidValue;
    // columns a CTA: the least time over the rounds that the CTAs make, as for the
    // prefill's chain (2.1 us a chunk with 32, 1.7 with 16)
    const long long tiles = (long long)d.batch * d.nheads * (d.headdim / 64), sms = device_sm_count();
    const long long t32 = 210 * ((2 * tiles + sms - 1) / sms), t16 = 170 * ((4 * tiles + sms - 1) / sms);
    return columns == 32 || (!columns && t32 <= t16) ? launch<32>(mK, mQ, mY, d, q, status, st)
                                                     : launch<16>(mK, mQ, mY, d, q, status, st);
}

}  // namespace m3

M3_BOUNDS_EXPORT(delta_rev)
