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
//   dg_t = sum_{i >= t > j} W_ij + sum_{i >= t} z_i + sum_{j < t} e^{G_C-G_j} k_j.Y_j + e^{G_C} <S, dS'>,
//     W = dP o P + dA o A (j < i),   z_i = scale e^{G_i} q_i.Z_i - beta_i e^{G_i} k_i.X_i
// (dg_t is the sum of all that crosses from the tokens before t to t and those behind
// it, and every term of it has the factor e^{g_t}: nothing is taken off again, so a
// strongly decaying gate's small gradient keeps its relative accuracy, and that of a
// gate that resets the state is zero.  As suffix sums of dG_i = q_i.dQ_i - k_i.dK_i
// + .. it is a small remainder of large numbers: an absolute error of 1e-8 to 1e-6,
// all of dg from mean gates of -16 on.)
//
// Three passes.  The prefill runs once more and records T, P, the state before
// every chunk and U.  k_delta_rev.cu carries dS from the last chunk to the first
// and records dS' and dR.  delta_grad_kernel here then takes all chunks in any
// order, one CTA an SM, the next chunk's records on their way while the present
// one is finished.  dq and dk of a group's heads are added by a further kernel in a
// fixed order.
//
// Products (tcgen05, M = 128 rows, accumulators in TMEM; rows 0..63 and 64..127
// of the left operand are two matrices, so that a thread finds all that belongs
// to a token in its row):
//   [Q; K] K^T,  [dY; dR] U^T,  [dY; dR] S^T,  [.; U] dS'^T
//   [scale Gam o dP; D] K,  [.; (scale Gam o dP)^T] Q + [.; D^T] K
// Float32 values enter as two bfloat16 parts (hi + lo; a product of two split
// operands drops lo x lo): dg and dbeta are sums with cancellation.  The records
// are stored in the layout that the products read (8 columns a piece), so no
// matrix is rearranged.
//
// A chunk takes 9.6 us on its SM (4096 chunks 0.265 ms): of some 14,000 cycles the
// 68 products take 4,000, the instructions 6,000 a scheduler, and the phases wait
// for one another and share the bandwidth of shared memory.  155 KB come in and
// 32 KB go out a chunk (2.9 TB/s), so memory does not bound it.
//
// Every wait on an mbarrier is bounded (1 s); on expiry the kernel records
// M3_ERR_DEVICE_TIMEOUT in the workspace status word and runs out without
// further waiting.
#define M3_BOUNDS_FILE 13
#include "m3_bounds.cuh"
#include "delta_tc.cuh"
#include "side_stream.h"

namespace m3 {

bool make_tile_map(CUtensorMap* map, const void* base, int inner, int R, int grp, int L, int batch, int T);

namespace dbw {

using namespace dtc;

constexpr int kThreads = 512;        // 4 row quarters x 4 column groups of warps

constexpr int OFF_QK = 0;                        // Q rows 0..63, K rows 64..127 (two 64-column atoms, sw128)
constexpr int OFF_A2 = 32768;                    // [0; dR lo] (16 KB; pieces of 8 columns, 128 rows each)
constexpr int OFF_U = OFF_A2 + 16384;            // U hi, lo (8 KB each; pieces of 64 rows)
constexpr int OFF_A = OFF_U + 16384;             // [dY; dR hi] (16 KB)
constexpr int OFF_S = OFF_A + 16384;             // S hi, lo (16 KB each; pieces of 128 rows)
constexpr int OFF_DS = OFF_S + 32768;            // dS' hi, lo
constexpr int OFF_D = OFF_DS + 32768;            // [scale Gam o dP; D] hi, lo (16 KB each, sw128)
constexpr int OFF_OUT = OFF_D + 32768;           // dQ, dK on their way out (as Q, K)
constexpr int OFF_MISC = OFF_OUT + 32768;
// TMEM columns; the last product takes the place of the first two
constexpr uint32_t D_PA = 0, D_QK = 64, D_ZX = 128, D_Y = 256, D_LAST = 384, D_T = 0;

struct Misc {
    Gates gates[2];
    float row[4][2 * kC], beta[4][kC], tail[4][kC];    // by column group (row: z, from dq's and dk's rows)
    float left[3][2 * kC], cross[4][kC];               // W: sums of rows by column group, of what crosses by row quarter
    float drv[4][kC], dot[16];
    uint64_t full[4], done[3], drain;
    uint32_t tmem_base;
    int abort_flag, drain_flag, pad;
};
constexpr int SMEM_BYTES = OFF_MISC + (int)sizeof(Misc) + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory of the chunk gradients");

// matrix descriptor without exchange of 16-byte groups: 8 rows x 16 bytes lie
// together, `lbo` bytes to the next 8 columns, `sbo` to the next 8 rows
__device__ __forceinline__ uint64_t sdesc0(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((saddr >> 4) & 0x3FFF) | ((uint64_t)((lbo >> 4) & 0x3FFF) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3FFF) << 32) | (1ull << 46);
}

__device__ __forceinline__ float2 unpack(uint32_t u) { return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)); }
__device__ __forceinline__ void unpack8(uint4 v, float* f) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 t = unpack(u[j]);
        f[2 * j] = t.x;
        f[2 * j + 1] = t.y;
    }
}

// part of a row's inner product: 8 columns
__device__ __forceinline__ float dot8(const float* x, const float* y, float t) {
#pragma unroll
    for (int j = 0; j < 8; ++j) t = fmaf(x[j], y[j], t);
    return t;
}
// a tile of shared memory into the tensor, rows behind its end left out
__device__ __forceinline__ void tma_store_5d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2, int c3, int c4) {
    asm volatile("cp.async.bulk.tensor.5d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5, %6}], [%1];"
                 ::"l"((uint64_t)map), "r"(src), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
                 : "memory");
}

// The CTAs (one an SM) walk the chunks; the records of a CTA's next chunk are on
// their way while it finishes the present one.
__global__ void __launch_bounds__(kThreads, 1)
    delta_grad_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmDK, const __grid_constant__ CUtensorMap tmDQ, DeltaParams q,
                      int total_chunks, int* status) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (su32(smem_raw) & 1023u)) & 1023u);
    Misc* m = reinterpret_cast<Misc*>(smem + OFF_MISC);
    const uint32_t sb = su32(smem);
    if (!M3_SPAN(1, smem - smem_raw, OFF_MISC + (int)sizeof(Misc), dyn_smem_bytes())) return;
    const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31, P = q.headdim, H = q.nheads;
    const int hpg = H / q.ngroups, slices = P / 64;
    [[maybe_unused]] const long long ext_k = (long long)q.batch * q.seqlen * q.ngroups * kN;
    [[maybe_unused]] const long long ext_v = (long long)q.batch * q.seqlen * H * P;
    [[maybe_unused]] const long long toks = (long long)q.batch * q.seqlen * H;
    [[maybe_unused]] const long long ext_rec = (long long)q.batch * H * q.nck * (long long)rec_elems(P, true);
    __nv_bfloat16* out_q = static_cast<__nv_bfloat16*>(q.dq);
    __nv_bfloat16* out_k = static_cast<__nv_bfloat16*>(q.dk);
    __nv_bfloat16* out_g = static_cast<__nv_bfloat16*>(q.dg);
    __nv_bfloat16* out_b = static_cast<__nv_bfloat16*>(q.dbeta);
    struct At {
        int b, h, g, c, len, nt;                   // nt <= 0: behind the sequence's end
    };
    auto locate = [&](int n) {
        At t;
        const int bh = n / q.nck;
        t.c = n % q.nck;
        t.b = bh / H;
        t.h = bh % H;
        t.g = t.h / hpg;
        t.len = q.seqlen;
        if (q.lengths && M3_IN(2, t.b, q.batch)) t.len = min(max(q.lengths[t.b], 0), q.seqlen);
        t.nt = min(kC, t.len - t.c * kC);
        return t;
    };
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) mbar_init(&m->full[i], 1);
        for (int i = 0; i < 3; ++i) mbar_init(&m->done[i], 1);
        mbar_init(&m->drain, 1);
        m->abort_flag = 0;
        m->drain_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
    }
    __syncwarp();
    if (warp == 0) {
        tmem_alloc(&m->tmem_base, 512);
        tmem_relinquish();
    }
    put16(smem, OFF_A2, (tid & 7) * 2048 + (tid >> 3) * 16, 16384, make_uint4(0u, 0u, 0u, 0u));    // (rows 0..63 stay zero)
    __syncthreads();
    int asked = 0;                                 // sets of records asked for (thread 0)
    // the recorded matrices of a slice, by the copy engine, in three groups
    auto load_records = [&](int n, int sl) {
        const size_t o = (size_t)n * rec_elems(P, true) + kRecSlice + sl * kSliceElems;
        const __nv_bfloat16* src = q.rec + o;
        M3_NOTE(5, o + kSliceElems - 1, ext_rec);
        mbar_expect_tx(&m->full[0], 16384 + 8192);
        bulk_load(sb + OFF_U, src + kSliceU, 16384, &m->full[0]);
        for (int p = 0; p < 8; ++p) bulk_load(sb + OFF_A + p * 2048 + 1024, src + kSliceDR + p * 512, 1024, &m->full[0]);
        mbar_expect_tx(&m->full[1], 8192 + 32768);
        for (int p = 0; p < 8; ++p) bulk_load(sb + OFF_A2 + p * 2048 + 1024, src + kSliceDR + kTok + p * 512, 1024, &m->full[1]);
        bulk_load(sb + OFF_S, src + kSliceS, 32768, &m->full[1]);
        mbar_expect_tx(&m->full[2], 32768);
        ++asked;
        bulk_load(sb + OFF_DS, src + kSliceDS, 32768, &m->full[2]);
    };
    // 16 bytes a thread of the slice's dY; rows behind the end (other data, possibly not numbers) are zeros
    auto fetch_dy = [&](const At& t, int sl) {
        const int r = tid >> 3;
        const size_t vo = (((size_t)t.b * q.seqlen + t.c * kC + r) * H + t.h) * P + 64 * sl + 8 * (tid & 7);
        if (r >= t.nt || !M3_SPAN(7, vo, 8, ext_v)) return make_uint4(0u, 0u, 0u, 0u);
        return __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(q.dy) + vo));
    };
    int fph = 0, done_y = 0, done_c = 0, par = 0;  // phases: records, Y, a chunk's other products; gates
    bool loaded = false;
    uint4 dy = make_uint4(0u, 0u, 0u, 0u);
    int stop = 0;
    for (int n = blockIdx.x; n < total_chunks && !stop; n += gridDim.x) {
        const At me = locate(n);
        const int b = me.b, h = me.h, g = me.g, c = me.c, len = me.len, nt = me.nt;
        const size_t row0 = (size_t)b * q.seqlen + c * kC;
        const int rows = min(kC, q.seqlen - c * kC);               // rows of the outputs in this chunk
        if (nt <= 0) {                                             // behind the end (a group's heads: the sum kernel's zeros)
            if (hpg == 1) {
                for (int e = tid; e < rows * 16; e += kThreads) {
                    const size_t o = ((row0 + (e >> 4)) * q.ngroups + g) * kN + 8 * (e & 15);
                    if (M3_SPAN(3, o, 8, ext_k)) {
                        *reinterpret_cast<uint4*>(out_q + o) = make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4*>(out_k + o) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
            }
            if (tid < rows && M3_IN(4, (row0 + tid) * H + h, toks)) {
                if (out_g) out_g[(row0 + tid) * H + h] = __float2bfloat16_rn(0.f);
                out_b[(row0 + tid) * H + h] = __float2bfloat16_rn(0.f);
            }
            continue;
        }
        if (tid == 0) {
            mbar_expect_tx(&m->full[3], 32768);
            tma_load_5d(sb + OFF_QK, &tmQ, &m->full[3], 0, 0, g, c * kC, b);
            tma_load_5d(sb + OFF_QK + 16384, &tmQ, &m->full[3], 64, 0, g, c * kC, b);
            tma_load_5d(sb + OFF_QK + 8192, &tmK, &m->full[3], 0, 0, g, c * kC, b);
            tma_load_5d(sb + OFF_QK + 24576, &tmK, &m->full[3], 64, 0, g, c * kC, b);
            if (!loaded) load_records(n, 0);
        }
        __syncwarp();
        if (!loaded) dy = fetch_dy(me, 0);
        if (warp == 4) make_gates(load_raw(q, b, h, len, c), &m->gates[par]);
        // the chunk after next into L2
        if ((long long)n + 2LL * gridDim.x < total_chunks) {
            const int n2 = n + 2 * gridDim.x;
            const At t = locate(n2);
            if (tid < slices)
                bulk_prefetch(q.rec + (size_t)n2 * rec_elems(P, true) + kRecSlice + tid * kSliceElems, (uint32_t)(kSliceElems * 2));
            if (tid >= 64 && tid < 128 && t.c * kC + tid - 64 < q.seqlen) {
                const size_t r = (size_t)t.b * q.seqlen + t.c * kC + tid - 64;
                const size_t ko = (r * q.ngroups + t.g) * kN, vo = (r * H + t.h) * P;
                if (M3_SPAN(13, ko, kN, ext_k) && M3_SPAN(14, vo, P, ext_v)) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        prefetch_l2(static_cast<const __nv_bfloat16*>(q.k) + ko + 64 * j);
                        prefetch_l2(static_cast<const __nv_bfloat16*>(q.q) + ko + 64 * j);
                    }
                    for (int j = 0; j < slices; ++j) {
                        prefetch_l2(static_cast<const __nv_bfloat16*>(q.dy) + vo + 64 * j);
                        prefetch_l2(static_cast<const __nv_bfloat16*>(q.v) + vo + 64 * j);
                    }
                }
            }
        }

        // all threads' copies of a group are in place and visible to the products
        auto arrived = [&]() {
            fence_async_smem();
            tc_fence_before();
            __syncthreads();
            tc_fence_after();
        };
        const uint64_t aQK = sdesc(sb + OFF_QK, 16, 1024), bK = sdesc(sb + OFF_QK + 8192, 16, 1024);
        const uint64_t aA = sdesc0(sb + OFF_A, 2048, 128), aA2 = sdesc0(sb + OFF_A2, 2048, 128);
        const uint64_t bU = sdesc0(sb + OFF_U, 1024, 128), bUl = sdesc0(sb + OFF_U + 8192, 1024, 128);
        const uint64_t aU = sdesc0(sb + OFF_U - 1024, 1024, 128), aUl = sdesc0(sb + OFF_U + 8192 - 1024, 1024, 128);   // rows 64..127
        const uint64_t bS = sdesc0(sb + OFF_S, 2048, 128), bSl = sdesc0(sb + OFF_S + 16384, 2048, 128);
        const uint64_t bDS = sdesc0(sb + OFF_DS, 2048, 128), bDSl = sdesc0(sb + OFF_DS + 16384, 2048, 128);
        constexpr uint32_t id64 = idesc_bf16(128, 64, 0, 0), id128 = idesc_bf16(128, 128, 0, 0);
        const int quarter = warp & 3, cg = warp >> 2, row = quarter * 32 + lane, tok = row & 63;
        const bool up = quarter < 2;                   // rows 0..63: dq's side; 64..127: dk's
        const uint32_t tmem = m->tmem_base;
        float2 dot2 = make_float2(0.f, 0.f);           // <S, dS'>
        float drv = 0.f;                               // dR . v
        for (int sl = 0; sl < slices; ++sl) {
            if (sl > 0) {
                mbar_wait_flag(&m->done[2], (done_y - 1) & 1, &m->abort_flag, status, 1);
                // (a barrier that waits for the sums, so that all they read has been read)
                __syncthreads_or(drv != drv && dot2.x != dot2.x);
                if (tid == 0 && !m->abort_flag) load_records(n, sl);
                __syncwarp();
                dy = fetch_dy(me, sl);
            }
            put16(smem, OFF_A, (tid & 7) * 2048 + (tid >> 3) * 16, 16384, dy);
            // V for dR . v: 16 of the slice's columns
            uint4 vv[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const size_t vo = ((row0 + tok) * H + h) * P + 64 * sl + 8 * (2 * cg + j);
                vv[j] = make_uint4(0u, 0u, 0u, 0u);
                if (!up && tok < nt && M3_SPAN(8, vo, 8, ext_v))
                    vv[j] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(q.v) + vo));
            }
            if (sl == 0) {
                mbar_wait_flag(&m->full[3], done_c & 1, &m->abort_flag, status, 8);
                if (nt < kC)
                    // Q and K rows behind the end must be zeros: the last products sum over all rows of the tiles
                    for (int e = tid; e < (kC - nt) * 32; e += kThreads) {
                        const int r = nt + (e >> 5), ch = e & 31;
                        put16(smem, OFF_QK + ((ch >> 3) & 1) * 16384, sw128(r + (ch >> 4) * 64, ch & 7), 16384,
                              make_uint4(0u, 0u, 0u, 0u));
                    }
            }
            mbar_wait_flag(&m->full[0], fph & 1, &m->abort_flag, status, 5);
            arrived();
            if (warp == 0) {
                if (sl == 0)
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        umma_one(tmem + D_QK, aQK + (kk >> 2) * 1024 + (kk & 3) * 2, bK + (kk >> 2) * 1024 + (kk & 3) * 2, id64,
                                 kk > 0);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) umma_one(tmem + D_PA, aA + kk * 256, bU + kk * 128, id64, sl + kk > 0);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) umma_one(tmem + D_PA, aA + kk * 256, bUl + kk * 128, id64, 1);
            }
            mbar_wait_flag(&m->full[1], fph & 1, &m->abort_flag, status, 6);
            if (warp == 0) {
                __syncwarp();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) umma_one(tmem + D_PA, aA2 + kk * 256, bU + kk * 128, id64, 1);
                if (sl == slices - 1) commit_one(&m->done[0]);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) umma_one(tmem + D_ZX, aA + kk * 256, bS + kk * 256, id128, sl + kk > 0);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) umma_one(tmem + D_ZX, aA + kk * 256, bSl + kk * 256, id128, 1);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) umma_one(tmem + D_ZX, aA2 + kk * 256, bS + kk * 256, id128, 1);
            }
            if (!up) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int p = 2 * cg + j;
                    float v[8], r[8], l[8];
                    unpack8(vv[j], v);
                    unpack8(*reinterpret_cast<const uint4*>(smem + OFF_A + p * 2048 + row * 16), r);
                    unpack8(*reinterpret_cast<const uint4*>(smem + OFF_A2 + p * 2048 + row * 16), l);
#pragma unroll
                    for (int e = 0; e < 8; ++e) drv = fmaf(r[e] + l[e], v[e], drv);
                }
            }
            mbar_wait_flag(&m->full[2], fph & 1, &m->abort_flag, status, 7);
            if (warp == 0) {
                __syncwarp();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) umma_one(tmem + D_Y, aU + kk * 128, bDS + kk * 256, id128, sl + kk > 0);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) umma_one(tmem + D_Y, aU + kk * 128, bDSl + kk * 256, id128, 1);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) umma_one(tmem + D_Y, aUl + kk * 128, bDS + kk * 256, id128, 1);
                commit_one(&m->done[2]);
            }
#pragma unroll
            for (int e = tid; e < 1024; e += kThreads) {
                const uint4 s0 = *reinterpret_cast<const uint4*>(smem + OFF_S + e * 16);
                const uint4 s1 = *reinterpret_cast<const uint4*>(smem + OFF_S + 16384 + e * 16);
                const uint4 d0 = *reinterpret_cast<const uint4*>(smem + OFF_DS + e * 16);
                const uint4 d1 = *reinterpret_cast<const uint4*>(smem + OFF_DS + 16384 + e * 16);
                const uint32_t a0[4] = {s0.x, s0.y, s0.z, s0.w}, a1[4] = {s1.x, s1.y, s1.z, s1.w};
                const uint32_t b0[4] = {d0.x, d0.y, d0.z, d0.w}, b1[4] = {d1.x, d1.y, d1.z, d1.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    dot2 = __ffma2_rn(__fadd2_rn(unpack(a0[j]), unpack(a1[j])), __fadd2_rn(unpack(b0[j]), unpack(b1[j])), dot2);
            }
            ++fph;
            ++done_y;
        }
        float dot = dot2.x + dot2.y;
#pragma unroll
        for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
        if (lane == 0) m->dot[warp] = dot;
        if (!up) m->drv[cg][tok] = drv;

        const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
        const Gates* gt = &m->gates[par];
        const float2 Gi = gt->G[tok];
        const float a = gt->a[tok], at = gt->at[tok], be = gt->beta[tok], sa = q.scale * a, ba = be * a;
        const bool live = tok < nt;
        float rowB = 0.f, tail = 0.f;
        mbar_wait_flag(&m->done[0], done_c & 1, &m->abort_flag, status, 2);
        __syncwarp();
        tc_fence_after();
        // 16 columns: up, scale Gam o dP; down, D, and the rows' sums of dA o Gam o K K^T
        if (16 * cg > (tok | 31)) {                    // right of the diagonal for all of the warp
#pragma unroll
            for (int j = 0; j < 4; ++j)
                put16(smem, OFF_D + (j & 1) * 16384, sw128(row, 2 * cg + (j >> 1)), 16384, make_uint4(0u, 0u, 0u, 0u));
            if (lane < 16) m->cross[quarter][16 * cg + lane] = 0.f;
            if (cg < 3) m->left[cg][row] = 0.f;
        } else {
            float d[16], s[16];
            tmem_ld16x2(tl + D_PA + 16 * cg, tl + D_QK + 16 * cg, d, s);
            float2 f[8];
            const float f0 = up ? q.scale : -be;
            float w = 0.f;                             // sum of W's row up to here
#pragma unroll
            for (int k2 = 0; k2 < 8; ++k2) {
                const int j = 16 * cg + 2 * k2;
                const float4 Gj = *reinterpret_cast<const float4*>(&gt->G[j]);
                float v[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int k = 2 * k2 + x;
                    const float2 gj = x ? make_float2(Gj.z, Gj.w) : make_float2(Gj.x, Gj.y);
                    const bool in = live && (up ? j + x <= tok : j + x < tok);
                    const float t = in ? d[k] * ex2(diff_pair(Gi, gj)) : 0.f;      // Gam o dP, or - Gam o dA
                    const float ts = in ? t * s[k] : 0.f;
                    if (!up) rowB -= ts;
                    v[x] = f0 * t;
                    if (j + x < tok) w = fmaf(f0, ts, w);
                    s[k] = j + x < tok ? w : 0.f;      // what crosses from the group's columns up to this one to this row
                }
                f[k2] = make_float2(v[0], v[1]);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                put16(smem, OFF_D, sw128(row, 2 * cg + j), 16384, take8(f + 4 * j));
                put16(smem, OFF_D + 16384, sw128(row, 2 * cg + j), 16384, round8(f + 4 * j));
            }
            if (cg < 3) m->left[cg][row] = w;
            // sums over the warp's rows, half of the columns going to the other half of the lanes at each step:
            // lanes 2 j and 2 j + 1 end with column j
#pragma unroll
            for (int o = 16; o > 1; o >>= 1) {
                const bool high = lane & o;
#pragma unroll
                for (int j = 0; j < o / 2; ++j) {
                    const float keep = high ? s[j + o / 2] : s[j], give = high ? s[j] : s[j + o / 2];
                    s[j] = keep + __shfl_xor_sync(kFull, give, o);
                }
            }
            s[0] += __shfl_xor_sync(kFull, s[0], 1);
            if (!(lane & 1)) m->cross[quarter][16 * cg + (lane >> 1)] = s[0];
        }
        // the last chunk's gradients have left their place in shared memory
        if (tid == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
        arrived();
        if (warp == 0) {
            const uint64_t aD = sdesc(sb + OFF_D, 16, 1024), aDT = sdesc(sb + OFF_D - 8192, 8192, 1024);   // second atom: rows 64..127
            const uint64_t mK = sdesc(sb + OFF_QK + 8192, 16384, 1024), mQ = sdesc(sb + OFF_QK, 16384, 1024);
            constexpr uint32_t idL = idesc_bf16(128, 128, 0, 1), idT = idesc_bf16(128, 128, 1, 1);
#pragma unroll
            for (int x = 0; x < 2; ++x) {              // hi, lo
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) umma_one(tmem + D_LAST, aD + x * 1024 + kk * 2, mK + kk * 128, idL, x + kk > 0);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) umma_one(tmem + D_T, aDT + x * 1024 + kk * 128, mQ + kk * 128, idT, x + kk > 0);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) umma_one(tmem + D_T, aDT + x * 1024 + 512 + kk * 128, mK + kk * 128, idT, 1);
            }
            commit_one(&m->done[1]);
        }
        // 32 columns of Z (up) or X and Y (down)
        mbar_wait_flag(&m->done[2], (done_y - 1) & 1, &m->abort_flag, status, 3);
        __syncwarp();
        tc_fence_after();
        // the next chunk's matrices: the products and (before the barrier above) the
        // sums that read their places are done
        loaded = false;
        if ((long long)n + gridDim.x < total_chunks) {
            const At t = locate(n + gridDim.x);
            if (t.nt > 0) {
                if (tid == 0 && !m->abort_flag) load_records(n + gridDim.x, 0);
                __syncwarp();
                dy = fetch_dy(t, 0);
                loaded = true;
            }
        }
        auto own8 = [&](int ch, float* k) {            // 8 columns of q (up) or k (down)
            const int col8 = 4 * cg + ch;
            unpack8(*reinterpret_cast<const uint4*>(smem + OFF_QK + (col8 >> 3) * 16384 + sw128(row, col8 & 7)), k);
        };
        float r[32];
        tmem_ld32(tl + D_ZX + 32 * cg, r);
        if (up) {
            float t0 = 0.f;
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {
                float k[8];
                own8(ch, k);
#pragma unroll
                for (int j = 8 * ch; j < 8 * ch + 8; ++j) r[j] *= sa;
                t0 = dot8(r + 8 * ch, k, t0);
            }
            m->row[cg][row] = t0;
        } else {
            float y[32], t0 = 0.f, t1 = 0.f;
            tmem_ld32(tl + D_Y + 32 * cg, y);
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {
                float k[8];
                own8(ch, k);
                t0 = dot8(r + 8 * ch, k, t0);
                t1 = dot8(y + 8 * ch, k, t1);
#pragma unroll
                for (int j = 8 * ch; j < 8 * ch + 8; ++j) r[j] = fmaf(at, y[j], -ba * r[j]);
            }
            rowB -= a * t0;
            m->row[cg][row] = -ba * t0;
            tail = at * t1;
            m->beta[cg][tok] = rowB;
            m->tail[cg][tok] = tail;
        }
        mbar_wait_flag(&m->done[1], done_c & 1, &m->abort_flag, status, 4);
        __syncwarp();
        tc_fence_after();
        {
            float l[32];
            tmem_ld32(tl + D_LAST + 32 * cg, l);
#pragma unroll
            for (int j = 0; j < 32; ++j) r[j] += l[j];
            if (!up) {
                tmem_ld32(tl + D_T + 32 * cg, l);
#pragma unroll
                for (int j = 0; j < 32; ++j) r[j] += l[j];
            }
            if (!live)
#pragma unroll
                for (int j = 0; j < 32; ++j) r[j] = 0.f;
            if (hpg == 1) {
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    const int col8 = 4 * cg + ch;
                    put16(smem, OFF_OUT, (col8 >> 3) * 16384 + sw128(row, col8 & 7), 32768, pack_chunk(r + 8 * ch));
                }
                fence_async_smem();
            } else {
                // pieces of 4 columns, so that a warp writes 512 bytes together
                const size_t o = ((size_t)n * 2 + (up ? 0 : 1)) * kC * kN + (8 * cg * kC + tok) * 4;
                if (M3_SPAN(11, o, 7 * kC * 4 + 4, (long long)total_chunks * 2 * kC * kN)) {
                    float4* dst = reinterpret_cast<float4*>(q.part_qk + o);
#pragma unroll
                    for (int j = 0; j < 8; ++j) dst[j * kC] = make_float4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
                }
            }
        }
        tc_fence_before();
        stop = __syncthreads_or(m->abort_flag);
        tc_fence_after();
        ++done_c;
        par ^= 1;
        if (hpg == 1 && tid == 0) {                    // rows behind the tensor's end are left out
            tma_store_5d(&tmDQ, sb + OFF_OUT, 0, 0, g, c * kC, b);
            tma_store_5d(&tmDQ, sb + OFF_OUT + 16384, 64, 0, g, c * kC, b);
            tma_store_5d(&tmDK, sb + OFF_OUT + 8192, 0, 0, g, c * kC, b);
            tma_store_5d(&tmDK, sb + OFF_OUT + 24576, 64, 0, g, c * kC, b);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
        __syncwarp();
        if (warp == 0) {
            // lane l has tokens 2 l, 2 l + 1.  suf[0]: sums of z from a token to the end; suf[x]:
            // of W's rows in the column groups before x; before: sums of Y's terms before a token
            float own[4][2], suf[4], tl2[2], before, total = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * lane + e;
                own[0][e] = tl2[e] = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    own[0][e] += m->row[j][i] + m->row[j][64 + i];
                    tl2[e] += m->tail[j][i];
                }
#pragma unroll
                for (int x = 1; x < 4; ++x)
                    own[x][e] = (x > 1 ? own[x - 1][e] : 0.f) + (m->left[x - 1][i] + m->left[x - 1][64 + i]);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) suf[x] = own[x][0] + own[x][1];
            before = tl2[0] + tl2[1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float u = __shfl_down_sync(kFull, suf[x], o);
                    if (lane + o < 32) suf[x] += u;
                }
                const float u = __shfl_up_sync(kFull, before, o);
                if (lane >= o) before += u;
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {              // the tokens behind this lane's
                suf[x] = __shfl_down_sync(kFull, suf[x], 1);
                if (lane == 31) suf[x] = 0.f;
            }
            before = __shfl_up_sync(kFull, before, 1);
            if (lane == 0) before = 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) total += m->dot[j];
            total *= gt->whole;
            float dg[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * lane + e, grp = i > 0 ? (i - 1) >> 4 : 0;
                float s[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) s[x] = suf[x] + own[x][1] + (e ? 0.f : own[x][0]);
                float v = s[0] + (grp == 1 ? s[1] : grp == 2 ? s[2] : grp == 3 ? s[3] : 0.f);
                if (i > 0)
#pragma unroll
                    for (int j = 0; j < 4; ++j) v += m->cross[j][i - 1];
                dg[e] = v + (e ? before + tl2[0] : before) + total;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * lane + e;
                const size_t o = (row0 + i) * H + h;
                if (i >= rows || !M3_IN(12, o, toks)) continue;
                float vb = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) vb += m->drv[j][i] + m->beta[j][i];
                const float vg = i < nt ? dg[e] : 0.f;
                vb = i < nt ? vb : 0.f;
                if (out_g) out_g[o] = __float2bfloat16_rn(vg);
                out_b[o] = __float2bfloat16_rn(vb);
            }
        }
    }
    if (tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (stop && warp == 0) {                       // a wait ran out: what is still on its way has a second to end
        commit_one(&m->drain);
        mbar_wait_flag(&m->drain, 0, &m->drain_flag, nullptr, 0);
        if (tid == 0) {
            for (int i = 0; i < 3; ++i) mbar_wait_flag(&m->full[i], (asked - 1) & 1, &m->drain_flag, nullptr, 0);
            mbar_wait_flag(&m->full[3], (done_c - 1) & 1, &m->drain_flag, nullptr, 0);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(m->tmem_base, 512);
}

// dq, dk: the sum of a group's heads, in their order.  One CTA per chunk of a
// group and half the columns of dq or dk; a thread adds 8 columns of a token, a
// warp 8 tokens x 32 columns, so that what it reads and writes are whole sectors.
__global__ void __launch_bounds__(256) delta_group_sum_kernel(DeltaParams q) {
    const int H = q.nheads, hpg = H / q.ngroups;
    const int c = blockIdx.x % q.nck, bg = blockIdx.x / q.nck, b = bg / q.ngroups, g = bg % q.ngroups;
    const int side = blockIdx.y >> 1;
    int len = q.seqlen;
    if (q.lengths && M3_IN(15, b, q.batch)) len = min(max(q.lengths[b], 0), q.seqlen);
    [[maybe_unused]] const long long ext = (long long)q.batch * H * q.nck * 2 * kC * kN;
    for (int e = threadIdx.x; e < 8 * kC; e += 256) {
        const int l = e & 31, tok = 8 * ((e >> 5) & 7) + (l & 7), col8 = (blockIdx.y & 1) * 8 + (e >> 8) * 4 + (l >> 3);
        const int t = c * kC + tok;
        if (t >= q.seqlen) continue;
        float s[8] = {};
        if (t < len)
#pragma unroll 4
            for (int hh = 0; hh < hpg; ++hh) {
                const size_t o = ((((size_t)b * H + g * hpg + hh) * q.nck + c) * 2 + side) * kC * kN + (2 * col8 * kC + tok) * 4;
                if (!M3_SPAN(16, o, 4 * kC + 4, ext)) continue;
                const float4 x = *reinterpret_cast<const float4*>(q.part_qk + o);
                const float4 y = *reinterpret_cast<const float4*>(q.part_qk + o + 4 * kC);
                s[0] += x.x;
                s[1] += x.y;
                s[2] += x.z;
                s[3] += x.w;
                s[4] += y.x;
                s[5] += y.y;
                s[6] += y.z;
                s[7] += y.w;
            }
        const size_t o = (((size_t)b * q.seqlen + t) * q.ngroups + g) * kN + 8 * col8;
        if (M3_SPAN(17, o, 8, (long long)q.batch * q.seqlen * q.ngroups * kN))
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(side ? q.dk : q.dq) + o) = pack_chunk(s);
    }
}

}  // namespace dbw

static SideStreams side_streams;

// Both chains: the prefill's and the reverse one need the chunk matrices, not each
// other.  Where both fit the SMs they run side by side (32 chains with 32
// columns: 2.1 us a chunk instead of 1.45 + 1.7 one after the other with 16), else
// one after the other.
static cudaError_t launch_chains(const m3_dims& d, const DeltaParams& f, const DeltaParams& q, int* status, cudaStream_t st) {
    const long long tiles = (long long)d.batch * d.nheads * (d.headdim / 64), sms = device_sm_count();
    int fwd = 0, rev = 0;
    if (tiles * (4 + 4) <= sms) fwd = 16, rev = 16;
    else if (tiles * (2 + 2) <= sms) fwd = 32, rev = 32;
    else if (tiles * (1 + 2) <= sms) fwd = 64, rev = 32;
    std::unique_lock<std::mutex> use;
    SideStream* side = fwd ? side_streams.take(st, &use) : nullptr;
    if (side && (cudaEventRecord(side->fork, st) != cudaSuccess ||
                 cudaStreamWaitEvent(side->stream, side->fork, 0) != cudaSuccess))
        side = nullptr;
    if (!side) {
        cudaGetLastError();                  // (a second stream that could not be had is no error)
        const cudaError_t e = launch_delta_chain(d, f, true, 0, status, st);
        return e == cudaSuccess ? launch_delta_rev(d, q, 0, status, st) : e;
    }
    const cudaError_t e1 = launch_delta_rev(d, q, rev, status, side->stream);
    const cudaError_t e2 = launch_delta_chain(d, f, true, fwd, status, st);
    // joined in any case, so that nothing of this call is left behind
    const cudaError_t e3 = cudaEventRecord(side->join, side->stream), e4 = cudaStreamWaitEvent(st, side->join, 0);
    return e1 != cudaSuccess ? e1 : e2 != cudaSuccess ? e2 : e3 != cudaSuccess ? e3 : e4;
}

cudaError_t launch_delta_bwd_tc(const m3_dims& d, const DeltaParams& q, int* status, cudaStream_t st) {
    using namespace dbw;
    DeltaParams f = q;                       // records of the prefill
    f.y = nullptr;
    f.final_h = nullptr;
    cudaError_t e = launch_delta_prep(d, f, true, status, st);
    if (e != cudaSuccess) return e;
    e = launch_chains(d, f, q, status, st);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(delta_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e != cudaSuccess) return e;
    CUtensorMap mK, mQ, mDK, mDQ;
    if (!make_tile_map(&mK, q.k, kN, 1, d.ngroups, d.seqlen, d.batch, kC) ||
        !make_tile_map(&mQ, q.q, kN, 1, d.ngroups, d.seqlen, d.batch, kC) ||
        !make_tile_map(&mDK, q.dk, kN, 1, d.ngroups, d.seqlen, d.batch, kC) ||
        !make_tile_map(&mDQ, q.dq, kN, 1, d.ngroups, d.seqlen, d.batch, kC))
        return cudaErrorInvalidValue;
    const long long total = (long long)d.batch * d.nheads * q.nck, sms = device_sm_count();
    delta_grad_kernel<<<(unsigned)(total < sms ? total : sms), kThreads, SMEM_BYTES, st>>>(mK, mQ, mDK, mDQ, q, (int)total,
                                                                                         status);
    e = cudaGetLastError();
    if (e != cudaSuccess || d.nheads == d.ngroups) return e;
    const dim3 grid((unsigned)((long long)d.batch * d.ngroups * q.nck), 4);
    delta_group_sum_kernel<<<grid, 256, 0, st>>>(q);
    return cudaGetLastError();
}

}  // namespace m3

M3_BOUNDS_EXPORT(delta_bwd_tc)
