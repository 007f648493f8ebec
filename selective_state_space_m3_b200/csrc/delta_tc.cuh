// delta_tc.cuh -- what the chunked kernels of the gated delta rule share: the
// gates of a chunk, splitting of float32 values into bfloat16 parts, and the
// records that the gradient's passes hand on.
#pragma once

#include "m3_delta.h"
#include "m3_kernels.h"
#include "tc_ptx.cuh"

namespace m3 {
namespace dtc {

using namespace ptx;

constexpr int kC = 64;             // tokens a chunk
constexpr int kN = 128;
constexpr unsigned kFull = 0xffffffffu;

struct alignas(16) ChainGates {    // what a chunk's chain reads
    float a[kC], at[kC], beta[kC]; // e^G, e^{G_C - G}, beta (0 behind the end)
    float whole;                   // e^{G_C}
    float pad[63];
};
struct alignas(16) Gates : ChainGates {
    float2 G[kC];                  // sum of g in log2 units, as a sum of two floats
    float mid[kC];                 // j < 32: e^{G_31 - G_j}; i >= 32: e^{G_i - G_31}
};
static_assert(sizeof(ChainGates) == 1024, "gates of a record");

__device__ __forceinline__ float clamp_g(float g) { return g < -1.0e4f ? -1.0e4f : g; }
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// two floats -> two bfloat16 (returned), f becomes what the rounding left
__device__ __forceinline__ uint32_t take2(float2& f) {
    const uint32_t w = pack_bf16x2(f.x, f.y);
    f = __ffma2_rn(make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)), make_float2(-1.f, -1.f), f);
    return w;
}
__device__ __forceinline__ uint4 take8(float2* f) {
    return make_uint4(take2(f[0]), take2(f[1]), take2(f[2]), take2(f[3]));
}
__device__ __forceinline__ uint4 round8(const float2* f) {
    return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                      pack_bf16x2(f[3].x, f[3].y));
}
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
    if (M3_SPAN(41, off, 16, limit)) *reinterpret_cast<uint4*>(smem + tile + off) = v;
}

// a + b of sums of two floats (each a pair with a small second part)
__device__ __forceinline__ float2 add_pair(float2 a, float2 b) {
    const float s = a.x + b.x, t = s - a.x;
    const float e = (a.x - (s - t)) + (b.x - t) + (a.y + b.y);
    const float r = s + e;
    return make_float2(r, e - (r - s));
}
__device__ __forceinline__ float diff_pair(float2 a, float2 b) { return (a.x - b.x) + (a.y - b.y); }

// g and beta of a chunk: lane l holds tokens 2 l and 2 l + 1
struct Raw {
    float g[2], beta[2];
};
__device__ __forceinline__ Raw load_raw(const DeltaParams& q, int b, int h, int len, int c) {
    const int lane = threadIdx.x & 31;
    Raw r;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int t = c * kC + 2 * lane + j;
        const size_t o = ((size_t)b * q.seqlen + t) * q.nheads + h;
        const bool ok = t < len && M3_IN(40, o, (long long)q.batch * q.seqlen * q.nheads);
        r.g[j] = (ok && q.g) ? __ldg(q.g + o) : 0.f;
        r.beta[j] = ok ? __ldg(q.beta + o) : 0.f;
    }
    return r;
}
// Sums of g in log2 units.  They run as pairs of floats, so that differences
// keep float32 accuracy after strong decay.
__device__ __forceinline__ void make_gates(const Raw& raw, Gates* out) {
    const int lane = threadIdx.x & 31;
    constexpr float kHi = 1.44269502162933349609f, kLo = 1.92596299112661746887e-8f;    // log2 e
    float2 d[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float g = clamp_g(raw.g[j]);
        const float p = g * kHi;
        d[j] = make_float2(p, fmaf(g, kHi, -p) + g * kLo);
    }
    float2 sum = add_pair(d[0], d[1]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float2 u = make_float2(__shfl_up_sync(kFull, sum.x, o), __shfl_up_sync(kFull, sum.y, o));
        if (lane >= o) sum = add_pair(sum, u);
    }
    const float2 total = make_float2(__shfl_sync(kFull, sum.x, 31), __shfl_sync(kFull, sum.y, 31));
    const float2 mid = make_float2(__shfl_sync(kFull, sum.x, 15), __shfl_sync(kFull, sum.y, 15));
    const float2 G[2] = {add_pair(sum, make_float2(-d[1].x, -d[1].y)), sum};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int i = 2 * lane + j;
        out->G[i] = G[j];
        out->a[i] = ex2(G[j].x + G[j].y);
        out->at[i] = ex2(diff_pair(total, G[j]));
        out->beta[i] = raw.beta[j];
        out->mid[i] = ex2(i < 32 ? diff_pair(mid, G[j]) : diff_pair(G[j], mid));
    }
    if (lane == 0) out->whole = ex2(total.x + total.y);
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(su32(bar)) : "memory");
}
__device__ __forceinline__ void bulk_prefetch(const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// arrival that waits for a value loaded from shared memory: its sign bit goes
// through the address, whose last three bits are cleared again (a barrier has 8
// bytes).  An arrival right behind a load does not wait for it, and the next
// chunk's data may overtake the load.
__device__ __forceinline__ void arrive_after(uint64_t* b, uint32_t loaded) {
    asm volatile(
        "{\n\t.reg .b32 t;\n\t"
        "shr.u32 t, %1, 31;\n\t"
        "add.u32 t, t, %0;\n\t"
        "and.b32 t, t, 0xfffffff8;\n\t"
        "mbarrier.arrive.shared::cta.b64 _, [t];\n\t}" ::"r"(su32(b)), "r"(loaded) : "memory");
}

struct Where {
    int b, h, g, p0, len, nch;     // p0: first column of the CTA
};

// where chain `tile` (a (batch, head) and PC of its columns) is
template <int PC>
__device__ __forceinline__ Where where_is(const DeltaParams& q, int tile) {
    Where w;
    const int slices = q.headdim / PC;
    const int bh = tile / slices;
    w.p0 = (tile % slices) * PC;
    w.b = bh / q.nheads;
    w.h = bh % q.nheads;
    w.g = w.h / (q.nheads / q.ngroups);
    int len = q.seqlen;
    if (q.lengths && M3_IN(42, w.b, q.batch)) len = min(max(q.lengths[w.b], 0), q.seqlen);
    w.len = len;
    w.nch = (len + kC - 1) / kC;
    return w;
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

// Records, one a chunk of a (batch, head), in bfloat16 elements.  Matrices are
// images of shared memory: rows of 128 bytes (64 columns), 16-byte groups
// exchanged by row (sw128).
//   X      [128][64]: T - I rounded; P = scale Gam o Q K^T rounded (zero rows behind the end)
//   TL     [64][64]: what the rounding left of T - I
//   gates  1024 bytes (ChainGates)
// for the gradient also
//   PL     [64][64]: what the rounding left of P
//   then for every 64 columns of the head, each as hi and lo part, groups of 8
//   columns one behind the other (so that a warp with a row a lane writes 512
//   bytes in a piece):
//   S before the chunk and its gradient behind the chunk [2][8][128][8] each, U and dR [2][8][64][8] each
constexpr size_t kTok = 64 * 64, kSt = 128 * 64;
constexpr size_t kRecX = 0, kRecTL = 2 * kTok, kRecGates = 3 * kTok, kRecPL = kRecGates + 512, kRecSlice = kRecPL + kTok;
constexpr size_t kSliceS = 0, kSliceDS = 2 * kSt, kSliceU = 4 * kSt, kSliceDR = 4 * kSt + 2 * kTok;
constexpr size_t kSliceElems = 4 * kSt + 4 * kTok;
// element of row `row`, column `col` of a part with `rows` rows
__host__ __device__ constexpr size_t rec_at(int rows, int row, int col) { return ((size_t)(col >> 3) * rows + row) * 8 + (col & 7); }
__host__ __device__ constexpr size_t rec_elems(int P, bool grad) {
    return grad ? kRecSlice + (size_t)(P / 64) * kSliceElems : kRecPL;
}

}  // namespace dtc
}  // namespace m3
