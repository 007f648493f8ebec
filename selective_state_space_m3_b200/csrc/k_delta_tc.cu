// k_delta_tc.cu -- chunked prefill of the gated delta rule on the sm_100a
// tensor cores (tcgen05 + TMEM + TMA): bfloat16 io, N = 128, P a multiple of 64.
//
// A chunk is C = 64 tokens.  With G the inclusive sum of g in the chunk,
// Gam_ij = e^{G_i - G_j} (j <= i) and S the state before the chunk:
//   A_ij = beta_i Gam_ij k_i.k_j (j < i)      T = (I + A)^{-1}
//   R = beta o (V - e^G o K S)                U = T R
//   Y = scale (e^G o Q S + (Gam o Q K^T) U)
//   S' = e^{G_C} S + K^T (e^{G_C - G} o U)
// T and P = scale Gam o Q K^T do not depend on S: a kernel before this one makes
// them for all chunks at once (k_delta_prep.cu).  The chain of a chunk is the
// three products K S, T R and K^T U.
//
// A CTA walks the chunks of a chain, a (batch, head) and PC of its columns:
//   warp 0       one elected lane issues the tcgen05.mma
//   warps 1..    the arithmetic between them: S lives in registers in float32 (a
//                thread has one state row and 8 or 16 columns)
//   last warp    one lane issues the loads (three chunks ahead: K, Q by TMA, the
//                images of T and P; two of V)
// Every product has M = 128 rows: [K; Q] against S gives K S and Q S at once,
// and the tile [T - I; P] serves both T R (upper half of the accumulator) and
// P U (lower half); the unused half is never read.  The parts of a split
// operand stand side by side as columns of one product (a 128 x 128 x 16 product
// takes 64 cycles, a 128 x 64 x 16 one 47) and the epilogue adds the columns.
//
// Chains that outnumber the SMs are laid end to end and cut into equal shares, one
// a CTA.  Where a cut goes through a chain, its first chunks belong to the CTA
// behind the cut, which starts with them and hands the state over through the
// workspace, and the rest to the CTA before the cut, which ends with them: a
// share is at least a chain long, so the state is there when it is wanted.  CTAs
// are numbered from the end of the line, so that one waits only for one that
// the GPU has started before it.  256 chains of 64 chunks on 148 SMs: 110 chunks a
// CTA instead of 128 in two rounds, 0.60 ms instead of 0.625 (chunk matrices and all).
//
// Precision.  K, Q, V are bfloat16 and enter the products as they are.  The
// chain keeps float32: S, R, U and T are split into bfloat16 parts (hi + lo, 16
// to 17 bits; the state's update of S takes three parts), the products of the
// parts add up in the float32 accumulators, and the identity of T is left out
// of the product and added in registers.  P alone is rounded to bfloat16 (half a
// step of 2^-8 relative, as y itself is); the U that it meets has two parts.  Where
// P U is a small difference of large terms, that rounding shows: the error of y is
// 2.3e-3 with keys as good as independent (1.7e-3 is y's own rounding), 4e-3 with
// cosines of 0.9 between keys, 1e-2 with 0.99.  P's low part, as the gradient's
// records have it, would be 8 KB more a chunk to write, to read and to hold.
//
// Shared memory (KB): K, Q 3 x 32, [T - I; P] 3 x 16, T lo 3 x 8, V 2 x 8, S hi/lo
// 32 (R and U take its place between the first product's end and the new state):
// one CTA an SM.
//
// Bound by latency: the three products and the conversions between them follow one
// another, 3.2 us a chunk with 64 columns a CTA, 1.95 with 32, 1.45 with 16 (tensor
// pipe 25, 23 and 15 % active).  U lo in P U costs 2 % of the time.
//
// Every wait on an mbarrier is bounded (1 s); on expiry the kernel records
// M3_ERR_DEVICE_TIMEOUT in the workspace status word and runs out without
// further waiting.
#define M3_BOUNDS_FILE 12
#include "m3_bounds.cuh"
#include "delta_tc.cuh"

#include <type_traits>

namespace m3 {

bool make_tile_map(CUtensorMap* map, const void* base, int inner, int R, int grp, int L, int batch, int T);

namespace dtc {

constexpr int kP = 64;             // columns of a V tile; a CTA takes PC = 64, 32 or 16 of them
// Column groups of the arithmetic, four warps each: 16 or 8 columns a thread
template <int PC> constexpr int kGroups = PC == 16 ? 2 : 4;
template <int PC> constexpr int kState = 128 * kGroups<PC>;        // threads of the chain
template <int PC> constexpr int kThreads = 32 + kState<PC> + 32;

constexpr int OFF_KQ = 0;                       // 3 x 32 KB: two 64-column atoms, rows 0..63 K, 64..127 Q
constexpr int OFF_X = OFF_KQ + 3 * 32768;       // 3 x 24 KB: [T - I hi; P], T - I lo (whose operand reads 64 more rows, unused)
constexpr int kXBytes = 24576;
constexpr int OFF_S = OFF_X + 3 * kXBytes;      // S hi, S lo (16 KB each: rows n, 64 p)
constexpr int OFF_U = OFF_S;                    // R hi, lo; then e^{G_C-G} U in three parts (8 KB each: rows t, 64 p)
constexpr int OFF_V = OFF_S + 32768;            // 2 x 8 KB; U hi (and lo beside it, for PC = 64 in T lo's place) for P U takes V's place
constexpr int OFF_GATES = OFF_V + 2 * 8192;     // 3 x 1 KB
constexpr int OFF_MISC = OFF_GATES + 3 * (int)sizeof(ChainGates);

// TMEM columns: K S, Q S against [S hi | S lo] and, once they are read, the
// state's update in three parts; T R against [R hi | R lo]; P U against [U hi | U lo]
constexpr uint32_t D_KS = 0, D_S = 0, D_TR = 192, D_O = 320;

struct Misc {
    uint64_t full[3], freed[3], v_full[2], v_free[2];
    uint64_t s_ready, ks, r, tr, u, ub, s, o, drain;
    uint32_t tmem_base;
    int abort_flag, drain_flag, pad;
};
constexpr int SMEM_BYTES = OFF_MISC + (int)sizeof(Misc) + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory of the delta kernel");

// The k-th piece of this CTA's share: chunks from .. to of a chain
struct Piece {
    Where w;
    int from, to;
    int take, give;                    // slot of the state that it starts from, that it leaves (-1: none)
    bool rest;                         // not the chain's first chunks
};
template <int PC, bool CUT>
__device__ __forceinline__ bool piece_at(const DeltaParams& q, int k, Piece* p) {
    if constexpr (!CUT) {                          // a CTA each
        if (k > 0) return false;
        p->w = where_is<PC>(q, blockIdx.x);
        p->from = 0;
        p->to = p->w.nch;
        p->take = p->give = -1;
        p->rest = false;
        return true;
    }
    const int cta = gridDim.x - 1 - blockIdx.x;
    const long long nck = q.nck, all = (long long)q.batch * q.nheads * (q.headdim / PC) * nck;
    const long long share = (all + gridDim.x - 1) / gridDim.x, lo = cta * share, hi = min(all, lo + share);
    const long long tile = lo / nck + k;
    if (tile * nck >= hi) return false;
    const int a = (int)max(lo - tile * nck, 0ll), b = (int)min(hi - tile * nck, nck);
    p->w = where_is<PC>(q, (int)tile);
    const int c0 = (int)nck - b, c1 = (int)nck - a;    // (one of them is an end of the chain)
    p->rest = c0 > 0;
    p->from = min(c0, p->w.nch);
    p->to = min(c1, p->w.nch);
    p->take = c0 > 0 ? cta + 1 : -1;
    p->give = p->w.nch > c1 ? cta : -1;
    return true;
}

__device__ __forceinline__ bool wait(uint64_t* b, int phase, Misc* m, int* status, int where) {
    return mbar_wait_flag(b, (uint32_t)(phase & 1), &m->abort_flag, status, where);
}
// a state that another CTA leaves (one thread; the others wait at a barrier)
__device__ __forceinline__ void wait_hand(const int* flag, Misc* m, int* status) {
    const uint64_t t0 = globaltimer_ns();
    int there = 0;
    while (!*(volatile int*)&m->abort_flag) {
        asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(there) : "l"(flag) : "memory");
        if (there) return;
        if (globaltimer_ns() - t0 > kWaitNs) {
            *(volatile int*)&m->abort_flag = 1;
            if (atomicCAS(status, 0, (int)M3_ERR_DEVICE_TIMEOUT) == 0) status[1] = 20;
        }
        __nanosleep(100);
    }
}
// DUMP: write the records that the gradient's passes read, and no y.
// CUT: chains may be cut between CTAs (the code for it costs 3 % where none is)
template <int PC, bool DUMP, bool CUT>
__global__ void __launch_bounds__(kThreads<PC>, 1)
    delta_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ,
                    const __grid_constant__ CUtensorMap tmV, DeltaParams q, int* status) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (su32(smem_raw) & 1023u)) & 1023u);
    Misc* m = reinterpret_cast<Misc*>(smem + OFF_MISC);
    const uint32_t sbase = su32(smem);
    if (!M3_SPAN(5, smem - smem_raw, OFF_MISC + (int)sizeof(Misc), dyn_smem_bytes())) return;
    const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
    constexpr int kCols = PC / kGroups<PC>;        // state columns a thread
    constexpr int W = kCols < 16 ? kCols : 16;     // columns of a TMEM load
    constexpr int NH = kCols / W, NG = kCols / 8;  // loads; 16-byte groups
    const int P = q.headdim;
    Piece pc;

    if (tid == 0) {
        for (int i = 0; i < 3; ++i) { mbar_init(&m->full[i], 1); mbar_init(&m->freed[i], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&m->v_full[i], 1); mbar_init(&m->v_free[i], 1); }
        mbar_init(&m->drain, 1);
        mbar_init(&m->s_ready, kState<PC>);
        mbar_init(&m->ks, 1);
        mbar_init(&m->r, kState<PC> / 2);
        mbar_init(&m->tr, 1);
        mbar_init(&m->u, kState<PC>);
        mbar_init(&m->ub, kState<PC> / 2);
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
        int total = 0;
        for (int k = 0; piece_at<PC, CUT>(q, k, &pc); ++k) total += pc.to - pc.from;
        for (int c = 0; c < total; ++c) {
            const uint32_t kq = sbase + OFF_KQ + (c % 3) * 32768;
            const uint64_t aKQ = sdesc(kq, 16, 1024), aKT = sdesc(kq, 16384, 1024);
            // (PC = 64: the lo part first, the hi part that many bytes behind it)
            const uint32_t hi = OFF_V + (c & 1) * 8192, lo = OFF_X + (c % 3) * kXBytes + 16384;
            const uint64_t bUB = PC == 64 ? sdesc(sbase + lo, hi - lo, 1024) : sdesc(sbase + hi, 8192, 1024);
            const uint64_t aX = sdesc(sbase + OFF_X + (c % 3) * kXBytes, 16, 1024);
            const uint64_t aTL = sdesc(sbase + OFF_X + (c % 3) * kXBytes + 16384, 16, 1024);
            wait(&m->full[c % 3], c / 3, m, status, 1);
            wait(&m->s_ready, c, m, status, 3);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                umma_one(tmem + D_KS, aKQ + (kk >> 2) * 1024 + (kk & 3) * 2, bS + kk * 128, idKS, kk > 0);
            commit_one(&m->ks);
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
            if (!DUMP) {
                wait(&m->ub, c, m, status, 7);
                __syncwarp();
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) umma_one(tmem + D_O, aX + kk * 2, bUB + kk * 128, idKS, kk > 0);
                commit_one(&m->o);
            }
            commit_one(&m->v_free[c & 1]);
            commit_one(&m->freed[c % 3]);
        }
        commit_one(&m->drain);
        mbar_wait_flag(&m->drain, 0, &m->drain_flag, nullptr, 0);
        __syncwarp();
    } else if (warp <= kState<PC> / 32) {
        // ---------------------------------------------- the chain's arithmetic
        const int wk = tid - 32, wg = wk >> 7, quarter = warp & 3, row = quarter * 32 + lane, c0 = wg * kCols;
        const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16) + c0;
        const bool top = quarter < 2;              // holds a token's K S and U; else its Q S and y
        const int tok = row & 63, ch0 = c0 / 8;
        [[maybe_unused]] const long long ext_h = (long long)q.batch * q.nheads * kN * P;
        const Where& w = pc.w;
        int done = 0;                              // chunks of the pieces before
        float2 S[kCols / 2];
        // 8 columns (group ch of this thread's) of row r of a recorded part with `rows` rows
        auto keep = [&](int c, size_t at, int rows, int r, int ch, uint4 v) {
            const size_t o = (((size_t)w.b * q.nheads + w.h) * q.nck + c) * rec_elems(P, true) + kRecSlice +
                             (size_t)(w.p0 >> 6) * kSliceElems + at + rec_at(rows, r, (w.p0 & 63) + c0 + 8 * ch);
            if (M3_SPAN(10, o, 8, (long long)q.batch * q.nheads * q.nck * rec_elems(P, true)))
                *reinterpret_cast<uint4*>(q.rec + o) = v;
        };
        auto store_state = [&](int c) {            // S hi, S lo before chunk c
            uint4 hi[NG], lo[NG];
#pragma unroll
            for (int ch = 0; ch < NG; ++ch) {
                float2 f[4] = {S[4 * ch], S[4 * ch + 1], S[4 * ch + 2], S[4 * ch + 3]};
                hi[ch] = take8(f);
                lo[ch] = round8(f);
                put16(smem, OFF_S, part_at<PC>(row, 0, ch0 + ch, 16384), 32768, hi[ch]);
                put16(smem, OFF_S, part_at<PC>(row, 1, ch0 + ch, 16384), 32768, lo[ch]);
            }
            fence_async_smem();
            tc_fence_before();
            mbar_arrive(&m->s_ready);
            if (DUMP) {
#pragma unroll
                for (int ch = 0; ch < NG; ++ch) {
                    keep(c, kSliceS, 128, row, ch, hi[ch]);
                    keep(c, kSliceS + kSt, 128, row, ch, lo[ch]);
                }
            }
        };
        // beta V of chunk c; rows behind the end (other data, possibly not numbers) count as zero
        float2 buf[kCols / 2];                     // top: beta V, R, then U; else Q S
        auto load_v = [&](int c, int i) {
            wait(&m->v_full[i & 1], i >> 1, m, status, 10);
            wait(&m->full[i % 3], i / 3, m, status, 11);
            const float be = reinterpret_cast<const ChainGates*>(smem + OFF_GATES)[i % 3].beta[tok];
            const float2 be2 = make_float2(be, be);
            const int vch = (w.p0 & 63) / 8 + ch0;
#pragma unroll
            for (int ch = 0; ch < NG; ++ch) {
                const uint32_t o = sw128(tok, vch + ch);
                uint4 vv = make_uint4(0u, 0u, 0u, 0u);
                if (c * kC + tok < w.len && M3_SPAN(7, o, 16, 8192))
                    vv = *reinterpret_cast<const uint4*>(smem + OFF_V + (i & 1) * 8192 + o);
                const uint32_t u[4] = {vv.x, vv.y, vv.z, vv.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    buf[4 * ch + j] = __fmul2_rn(be2, make_float2(__uint_as_float(u[j] << 16),
                                                                  __uint_as_float(u[j] & 0xffff0000u)));
            }
        };
#pragma unroll 1
        for (int k = 0; piece_at<PC, CUT>(q, k, &pc); ++k) {
            if (pc.rest && pc.from == pc.to) continue;         // (the sequence ends before this piece)
            const size_t ho = (((size_t)w.b * q.nheads + w.h) * kN + row) * P + w.p0 + c0;
            const float* src = q.init_h ? q.init_h + ho : nullptr;
            if (pc.take >= 0) {
                if (tid == 32) wait_hand(q.flags + pc.take, m, status);
                __syncwarp();
                asm volatile("bar.sync 1, %0;" ::"n"(kState<PC>) : "memory");
                src = q.hand + ((size_t)pc.take * kN + row) * 64 + c0;
            }
            [[maybe_unused]] const long long off_s = pc.take >= 0 ? src - q.hand : (long long)ho;
            [[maybe_unused]] const long long ext_s = pc.take >= 0 ? (long long)kDeltaSlots * kN * 64 : ext_h;
#pragma unroll
            for (int c4 = 0; c4 < kCols / 4; ++c4) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (src && M3_SPAN(6, off_s + 4 * c4, 4, ext_s)) v = __ldcg(reinterpret_cast<const float4*>(src + 4 * c4));
                S[2 * c4] = make_float2(v.x, v.y);
                S[2 * c4 + 1] = make_float2(v.z, v.w);
            }
            const int base = CUT ? done - pc.from : 0;
            done += pc.to - pc.from;
            if (pc.from < pc.to) {
                store_state(pc.from);
                if (top) load_v(pc.from, base + pc.from);
            }
#pragma unroll 1
            for (int c = pc.from; c < pc.to; ++c) {
                const int i = base + c;            // stages and phases count over all pieces
                const ChainGates* gt = reinterpret_cast<const ChainGates*>(smem + OFF_GATES) + i % 3;
                const bool tail = (c + 1) * kC > w.len;
                float whole;
                if (top) {
                    const float ba = -gt->beta[tok] * gt->a[tok], at = gt->at[tok];
                    whole = gt->whole;
                    const bool in = c * kC + tok < w.len;
                    const float2 ba2 = make_float2(ba, ba), at2 = make_float2(at, at);
                    wait(&m->ks, i, m, status, 12);
                    __syncwarp();
                    tc_fence_after();
#pragma unroll
                    for (int hh = 0; hh < NH; ++hh) {
                        float2 d[W / 2];
                        tmem_sum<W, 2>(tl + D_KS + W * hh, PC, d);
#pragma unroll
                        for (int j = 0; j < W / 2; ++j) d[j] = buf[W / 2 * hh + j] = __ffma2_rn(ba2, d[j], buf[W / 2 * hh + j]);
                        if (tail) {                    // K S of tokens behind the end may be anything
#pragma unroll
                            for (int j = 0; j < W / 2; ++j)
                                if (!in) d[j] = buf[W / 2 * hh + j] = make_float2(0.f, 0.f);
                        }
#pragma unroll
                        for (int ch = 0; ch < W / 8; ++ch) {
                            put16(smem, OFF_U, part_at<PC>(tok, 0, ch0 + W / 8 * hh + ch, 8192), 24576, take8(d + 4 * ch));
                            put16(smem, OFF_U, part_at<PC>(tok, 1, ch0 + W / 8 * hh + ch, 8192), 24576, round8(d + 4 * ch));
                        }
                    }
                    fence_async_smem();
                    tc_fence_before();
                    mbar_arrive(&m->r);
                    wait(&m->tr, i, m, status, 13);
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
#pragma unroll
                            for (int j = 0; j < 4; ++j) buf[W / 2 * hh + 4 * ch + j] = f[4 * ch + j];
#pragma unroll
                            for (int j = 0; j < 4; ++j) f[4 * ch + j] = __fmul2_rn(at2, f[4 * ch + j]);
                            put16(smem, OFF_U, part_at<PC>(tok, 0, cc, 8192), 24576, take8(f + 4 * ch));
                            put16(smem, OFF_U, part_at<PC>(tok, 1, cc, 8192), 24576, take8(f + 4 * ch));
                            put16(smem, OFF_U, part_at<PC>(tok, 2, cc, 8192), 24576, round8(f + 4 * ch));
                        }
                    }
                    fence_async_smem();
                    tc_fence_before();
                    arrive_after(&m->u, __float_as_uint(whole));
                    // U's parts for P U, while the state's update is made
#pragma unroll
                    for (int ch = 0; ch < NG; ++ch) {
                        const uint4 hi = take8(buf + 4 * ch), lo = round8(buf + 4 * ch);
                        if (DUMP) {
                            keep(c, kSliceU, 64, tok, ch, hi);
                            keep(c, kSliceU + kTok, 64, tok, ch, lo);
                        } else {
                            put16(smem, OFF_V + (i & 1) * 8192, sw128(tok, ch0 + ch), 8192, hi);
                            if (PC == 64) put16(smem, OFF_X + (i % 3) * kXBytes + 16384, sw128(tok, ch0 + ch), 8192, lo);
                            else put16(smem, OFF_V + (i & 1) * 8192, part_at<PC>(tok, 1, ch0 + ch, 8192), 8192, lo);
                        }
                    }
                    if (!DUMP) {
                        fence_async_smem();
                        mbar_arrive(&m->ub);
                    }
                    if (c + 1 < pc.to) load_v(c + 1, i + 1);  // while the state's update is made
                } else {
                    wait(&m->full[i % 3], i / 3, m, status, 14);
                    const float a = gt->a[tok];
                    whole = gt->whole;
                    const float sa = q.scale * a;
                    const float2 sa2 = make_float2(sa, sa);
                    wait(&m->ks, i, m, status, 15);
                    __syncwarp();
                    tc_fence_after();
#pragma unroll
                    for (int hh = 0; hh < NH; ++hh) {
                        tmem_sum<W, 2>(tl + D_KS + W * hh, PC, buf + W / 2 * hh);
#pragma unroll
                        for (int j = 0; j < W / 2; ++j) buf[W / 2 * hh + j] = __fmul2_rn(sa2, buf[W / 2 * hh + j]);
                    }
                    if (tail) {
                        // K rows behind the sequence's end (other data, possibly not numbers)
                        // must be zeros: K^T U sums over all rows of the tile
                        const int nt = w.len - c * kC;
                        for (int e = wg * 64 + tok; e < (kC - nt) * 16; e += kState<PC> / 2) {
                            const int r = nt + (e >> 4), ch = e & 15;
                            put16(smem, OFF_KQ + (i % 3) * 32768 + (ch >> 3) * 16384, sw128(r, ch & 7), 16384, make_uint4(0u, 0u, 0u, 0u));
                        }
                        fence_async_smem();
                    }
                    tc_fence_before();
                    arrive_after(&m->u, __float_as_uint(whole) | __float_as_uint(a));
                }
                const float2 w2 = make_float2(whole, whole);
                wait(&m->s, i, m, status, 16);
                __syncwarp();
                tc_fence_after();
#pragma unroll
                for (int hh = 0; hh < NH; ++hh) {
                    float2 d[W / 2];
                    tmem_sum<W, 3>(tl + D_S + W * hh, PC, d);
#pragma unroll
                    for (int j = 0; j < W / 2; ++j) S[W / 2 * hh + j] = __ffma2_rn(w2, S[W / 2 * hh + j], d[j]);
                }
                if (c + 1 < pc.to) store_state(c + 1);
                if (!DUMP && !top) {
                    wait(&m->o, i, m, status, 17);
                    __syncwarp();
                    tc_fence_after();
                    const size_t o = (((size_t)w.b * q.seqlen + c * kC + tok) * q.nheads + w.h) * P + w.p0 + c0;
                    const bool in = c * kC + tok < w.len && M3_SPAN(8, o, kCols, (long long)q.batch * q.seqlen * q.nheads * P);
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(q.y) + o);
#pragma unroll
                    for (int hh = 0; hh < NH; ++hh) {
                        float2 f[W / 2];
                        tmem_sum<W, 2>(tl + D_O + W * hh, PC, f);
#pragma unroll
                        for (int j = 0; j < W / 2; ++j) f[j] = __fadd2_rn(buf[W / 2 * hh + j], f[j]);
                        if (in) {
#pragma unroll
                            for (int ch = 0; ch < W / 8; ++ch) dst[W / 8 * hh + ch] = round8(f + 4 * ch);
                        }
                    }
                }
            }
            float* dst = pc.give >= 0 ? q.hand + ((size_t)pc.give * kN + row) * 64 + c0 : q.final_h ? q.final_h + ho : nullptr;
            [[maybe_unused]] const long long off_d = pc.give >= 0 ? dst - q.hand : (long long)ho;
            [[maybe_unused]] const long long ext_d = pc.give >= 0 ? (long long)kDeltaSlots * kN * 64 : ext_h;
            if (dst && M3_SPAN(9, off_d, kCols, ext_d)) {
#pragma unroll
                for (int c4 = 0; c4 < kCols / 4; ++c4)
                    *reinterpret_cast<float4*>(dst + 4 * c4) =
                        make_float4(S[2 * c4].x, S[2 * c4].y, S[2 * c4 + 1].x, S[2 * c4 + 1].y);
            }
            if (pc.give >= 0) {
                __threadfence();
                asm volatile("bar.sync 1, %0;" ::"n"(kState<PC>) : "memory");
                if (tid == 32) asm volatile("st.release.gpu.global.b32 [%0], 1;" ::"l"(q.flags + pc.give) : "memory");
            }
        }
    } else {
        // ------------------------------------------------------------- loads
        if (lane == 0) {
            const size_t rec = rec_elems(P, DUMP);
            int asked = 0, asked_v = 0;            // (fewer than the chunks after a wait that ran out)
            const Where& w = pc.w;
            bool go = true;
            for (int k = 0, done = 0; go && piece_at<PC, CUT>(q, k, &pc); ++k) {
                const size_t bh = (size_t)w.b * q.nheads + w.h;
                const int base = CUT ? done - pc.from : 0;
                done += pc.to - pc.from;
                for (int c = pc.from; c < pc.to; ++c) {
                    const int i = base + c;
                    const uint32_t kq = sbase + OFF_KQ + (i % 3) * 32768, x = sbase + OFF_X + (i % 3) * kXBytes;
                    go = i < 3 || wait(&m->freed[i % 3], i / 3 - 1, m, status, 30);
                    if (!go) break;
                    // chunk c + 3 into L2: its load waits for a stage, and then finds it there
                    if (c + 3 < pc.to) {
                        const int t = (c + 3) * kC;
                        tma_prefetch_5d(&tmK, 0, 0, w.g, t, w.b);
                        tma_prefetch_5d(&tmK, 64, 0, w.g, t, w.b);
                        tma_prefetch_5d(&tmQ, 0, 0, w.g, t, w.b);
                        tma_prefetch_5d(&tmQ, 64, 0, w.g, t, w.b);
                        tma_prefetch_5d(&tmV, w.p0 & ~63, 0, w.h, t, w.b);
                        bulk_prefetch(q.rec + (bh * q.nck + c + 3) * rec, kXBytes + sizeof(ChainGates));
                    }
                    uint64_t* bar = &m->full[i % 3];
                    const __nv_bfloat16* src = q.rec + (bh * q.nck + c) * rec;
                    M3_NOTE(13, (bh * q.nck + c) * rec + kRecPL - 1, (long long)q.batch * q.nheads * q.nck * (long long)rec);
                    mbar_expect_tx(bar, 32768 + kXBytes + sizeof(ChainGates));
                    tma_load_5d(kq, &tmK, bar, 0, 0, w.g, c * kC, w.b);
                    tma_load_5d(kq + 16384, &tmK, bar, 64, 0, w.g, c * kC, w.b);
                    tma_load_5d(kq + 8192, &tmQ, bar, 0, 0, w.g, c * kC, w.b);
                    tma_load_5d(kq + 24576, &tmQ, bar, 64, 0, w.g, c * kC, w.b);
                    ++asked;
                    bulk_load(x, src + kRecX, kXBytes, bar);
                    bulk_load(sbase + OFF_GATES + (i % 3) * (int)sizeof(ChainGates), src + kRecGates, sizeof(ChainGates), bar);
                    go = i < 2 || wait(&m->v_free[i & 1], (i >> 1) - 1, m, status, 31);
                    if (!go) break;
                    ++asked_v;
                    bar = &m->v_full[i & 1];
                    mbar_expect_tx(bar, 8192);
                    tma_load_5d(sbase + OFF_V + (i & 1) * 8192, &tmV, bar, w.p0 & ~63, 0, w.h, c * kC, w.b);
                }
            }
            // nothing may still be on its way into shared memory when the CTA ends
            for (int c = max(0, asked - 3); c < asked; ++c)
                mbar_wait_flag(&m->full[c % 3], (c / 3) & 1, &m->drain_flag, nullptr, 0);
            for (int c = max(0, asked_v - 2); c < asked_v; ++c)
                mbar_wait_flag(&m->v_full[c & 1], (c >> 1) & 1, &m->drain_flag, nullptr, 0);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

}  // namespace dtc

static long long chain_ctas() {
    const int sms = device_sm_count();
    return sms < kDeltaSlots ? sms : kDeltaSlots;
}
// (0 where even chains of 16 columns have a CTA each)
size_t delta_hand_bytes(const m3_dims& d) {
    if ((long long)d.batch * d.nheads * (d.headdim / 16) <= chain_ctas()) return 0;
    return kDeltaFlagBytes + sizeof(float) * kDeltaSlots * dtc::kN * dtc::kP;
}

size_t delta_record_bytes(const m3_dims& d, bool grad) { return dtc::rec_elems(d.headdim, grad) * 2; }

bool delta_tc_eligible(const m3_dims& d) {
    return d.io_dtype == M3_BF16 && d.dstate == dtc::kN && d.headdim % dtc::kP == 0;
}

template <int PC, bool DUMP, bool CUT>
static cudaError_t launch_pc(const CUtensorMap& mK, const CUtensorMap& mQ, const CUtensorMap& mV, const m3_dims& d,
                             const DeltaParams& q, int* status, cudaStream_t st) {
    using namespace dtc;
    const cudaError_t e = cudaFuncSetAttribute(delta_tc_kernel<PC, DUMP, CUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e != cudaSuccess) return e;
    const long long chains = (long long)d.batch * d.nheads * (d.headdim / PC), most = chain_ctas();
    const unsigned grid = (unsigned)(chains < most ? chains : most);
    delta_tc_kernel<PC, DUMP, CUT><<<grid, kThreads<PC>, SMEM_BYTES, st>>>(mK, mQ, mV, q, status);
    return cudaGetLastError();
}

// Columns a CTA.  A chunk of a chain takes 3.2 us with 64 columns, 1.95 with 32
// and 1.45 with 16 (measured; the products' latency stays, the arithmetic
// shrinks): the choice is the least time of a CTA's share, a chain or more, so
// that few sequences are spread over the SMs.
static int chain_columns(long long tiles) {
    const long long most = chain_ctas();
    auto share = [&](int split) { return tiles * split > most ? tiles * split : most; };
    const long long t64 = 320 * share(1), t32 = 195 * share(2), t16 = 145 * share(4);
    return t64 <= t32 && t64 <= t16 ? 64 : t32 <= t16 ? 32 : 16;
}

cudaError_t launch_delta_chain(const m3_dims& d, const DeltaParams& q, bool grad, int columns, int* status, cudaStream_t st) {
    using namespace dtc;
    CUtensorMap mK, mQ, mV;
    if (!make_tile_map(&mK, q.k, kN, 1, d.ngroups, d.seqlen, d.batch, kC) ||
        !make_tile_map(&mQ, q.q, kN, 1, d.ngroups, d.seqlen, d.batch, kC) ||
        !make_tile_map(&mV, q.v, d.headdim, 1, d.nheads, d.seqlen, d.batch, kC))
        return cudaErrorInvalidValue;
    const long long tiles = (long long)d.batch * d.nheads * (d.headdim / kP), most = chain_ctas();
    const int pc = columns ? columns : chain_columns(tiles);
    const bool cut = tiles * (kP / pc) > most;
    auto go = [&](auto dump, auto cuts) {
        constexpr bool D = decltype(dump)::value, C = decltype(cuts)::value;
        return pc == 64 ? launch_pc<64, D, C>(mK, mQ, mV, d, q, status, st)
             : pc == 32 ? launch_pc<32, D, C>(mK, mQ, mV, d, q, status, st)
                        : launch_pc<16, D, C>(mK, mQ, mV, d, q, status, st);
    };
    using Yes = std::true_type;
    using No = std::false_type;
    return grad ? (cut ? go(Yes(), Yes()) : go(Yes(), No())) : (cut ? go(No(), Yes()) : go(No(), No()));
}

cudaError_t launch_delta_tc(const m3_dims& d, const DeltaParams& q, int* status, cudaStream_t st) {
    const cudaError_t e = launch_delta_prep(d, q, false, status, st);
    return e == cudaSuccess ? launch_delta_chain(d, q, false, 0, status, st) : e;
}

}  // namespace m3

M3_BOUNDS_EXPORT(delta_tc)
