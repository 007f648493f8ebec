// m3_delta.h -- parameter blocks and launch functions of the gated delta rule's
// kernels (internal to the library; the public ABI is include/m3.h).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>

#include "m3.h"

namespace m3 {

// gated delta rule (k_delta.cu, k_delta_tc.cu); the decode step reads init_h
// and writes final_h (which may be the same buffer)
struct DeltaParams {
    int batch, seqlen, nheads, ngroups, headdim, dstate;
    float scale;
    const void* q;             // [b][t][g][n] io
    const void* k;             // [b][t][g][n] io
    const void* v;             // [b][t][h][p] io
    const float* g;            // [b][t][h] log decay, nullable (0)
    const float* beta;         // [b][t][h]
    const int* lengths;        // [b], nullable (every sequence has seqlen tokens)
    const float* init_h;       // [b][h][n][p], nullable (zeros)
    void* y;                   // [b][t][h][p] io
    float* final_h;            // [b][h][n][p], nullable
    // gradient
    const void* dy;            // [b][t][h][p] io
    const float* d_final_h;    // nullable
    void* dq;                  // io, as q
    void* dk;
    void* dv;
    void* dg;                  // [b][t][h] io, nullable
    void* dbeta;
    float* d_init_h;           // nullable
    int KB, nck;               // tokens a checkpoint, checkpoints a sequence
    float* ckpt;               // [b][h][nck][n][p]
    float* part_qk;            // [column tile][b][t][h][2][n]: parts of dq, dk; chunked: [b][h][chunk][2][n / 4][64][4]
    float* part_g;             // [column tile][b][t][h][2]: parts of dg, dbeta
    __nv_bfloat16* rec;        // chunked path: nck records a (b, h) (delta_tc.cuh)
    float* hand;               // states handed from CTA to CTA [kDeltaSlots][128][64]
    int* flags;                // ... and whether they are there [kDeltaSlots]
};
constexpr int kDeltaSlots = 148;   // most CTAs of the prefill's chains that share chains
// bytes of `hand` and `flags` (0: a CTA each for all chains)
size_t delta_hand_bytes(const m3_dims& d);
constexpr size_t kDeltaFlagBytes = 1024;
int delta_block_tokens(const m3_dims& d);
int delta_tiles(const m3_dims& d);
cudaError_t launch_delta_seq(const m3_dims& d, const DeltaParams& q, cudaStream_t st);
cudaError_t launch_delta_seq_bwd(const m3_dims& d, const DeltaParams& q, cudaStream_t st);
// chunked prefill on the tensor cores (bf16, N = 128, P a multiple of 64);
// `status` is the workspace status word its bounded waits report to
bool delta_tc_eligible(const m3_dims& d);
cudaError_t launch_delta_tc(const m3_dims& d, const DeltaParams& q, int* status, cudaStream_t st);
// its parts: the records of k_delta_prep.cu and the chain (`columns` a CTA, 0: the
// choice is the kernel's; grad: records for the gradient, no y)
cudaError_t launch_delta_prep(const m3_dims& d, const DeltaParams& q, bool grad, int* status, cudaStream_t st);
cudaError_t launch_delta_chain(const m3_dims& d, const DeltaParams& q, bool grad, int columns, int* status, cudaStream_t st);
// bytes of a record, one a chunk of 64 tokens of a (batch, head)
size_t delta_record_bytes(const m3_dims& d, bool grad);
// chunked gradient (same shapes)
cudaError_t launch_delta_rev(const m3_dims& d, const DeltaParams& q, int columns, int* status, cudaStream_t st);
cudaError_t launch_delta_bwd_tc(const m3_dims& d, const DeltaParams& q, int* status, cudaStream_t st);
cudaError_t launch_delta_step(const m3_dims& d, const DeltaParams& q, cudaStream_t st);

}  // namespace m3
