// attend_paged.cu — attention of the newest rows of each sequence over the paged MXFP4 cache.
//
// Mathematics. For a row: s_j = scale q . K_j, o = sum_j exp(s_j - m) V_j /
// sum_j exp(s_j - m), one pass over the keys with a reference m and the two
// sums (see attend_prompt.cu). K_j = 2^(a - 127) k with E2M1 codes k and one
// scale code a per 32 dimensions; V likewise.
//   Keys: codes as f16 (exact); the partial score of each group of 32
//   dimensions is multiplied by its 2^(a - 127) in binary32. Queries become f16
//   times a power of two per row: exact but for parts 2^-28 below the row's
//   largest and smaller.
//   Values: codes times 2^(b - b_ref) in f16, with b_ref the largest scale code
//   that the warp has seen; like m it moves as the pass goes on, and the
//   accumulators are rescaled when it does. Exact down to 2^-23 of the largest.
//   Probabilities: f16, at most 2^15 (the lazy reference of attend_prompt.cu, less
//   2^7 so that small ones keep their bits: exact to 2^-32 of the row's largest).
// All sums are binary32, on the tensor cores (mma.sync m16n8k16, f16 operands).
//
// Bound. A cached token and kv head is D + D/16 bytes against 4 D flops per row
// and head: HBM for single tokens. Decoding the 4-bit codes is CUDA-core work
// whatever multiplies them (2 D conversions a token, at half rate). 128 single
// tokens of 4,000 to 16,000 (D = 128, 32 + 8 heads) take 243 us, 4.83 TB/s or 71 %
// of the copy bandwidth: issue slots are 63 % busy, the ALU pipe 56 %. With 24
// rows of a kv head (steps of six rows, 64 sequences of 1,024 to 5,120, 77 us) it
// is neither: two warps a scheduler (the accumulators take the registers) wait on
// fixed latencies; tensor pipe 36 %, issue 44 %, HBM 30 %. One token over 4,096:
// 10.3 us, launches and the chain lookup - load - join.
// The codes go from shared memory straight into the registers that the MMA
// reads. tcgen05 would need V in 16 bits in shared memory first, since V's scale
// groups do not lie along the product's inner dimension (the keys). K's do: its
// codes and scales could be the operands of a block-scaled MMA as they are, with the
// queries split into 8-bit terms. That has not been built.
//
// Layout. Keys are the MMA's M (scores transposed: 16 keys x 8 rows), so a step
// of 8 rows wastes nothing on padding. The order of a product's inner dimension
// is free when both operands share it, so a lane's operand registers are decoded
// from whole 4-byte (K) and 8-byte (V) pieces of a cached row:
//   S^T = K Q^T   lane (g, t) = (lane / 4, lane % 4) decodes dimensions
//                 32 j + 8 t .. + 7 of keys g and g + 8, for each group j
//   O^T = V^T P^T lane (g, t) decodes dimensions [g D/8, (g + 1) D/8) of keys
//                 2t, 2t + 1, 2t + 8, 2t + 9, two keys' codes interleaved
// P moves from the first product's result layout to the second's operand
// layout by movmatrix. Rows are (token, head) pairs of one kv head's group.
//
// Schedule. The work is a list of items (sequence, kv head, row block), each of
// kOver units for its queries and its join and one for each stage of 32 keys.
// Every block takes an equal, contiguous share of the units, so one long sequence
// spreads over all SMs and a batch of ragged ones stays balanced. Within its share
// of an item a block's warps take the stages in turn. Each copies its own ahead of
// time into a ring of its own (cp.async), so they meet only where an item ends:
// there the accumulators of all warps are joined through shared memory, which the
// drained rings leave free. What a block holds of an item that it shares with
// other blocks goes to the workspace; a second kernel, launched with programmatic
// dependent launch, joins these in a fixed order. Which ones, the main kernel leaves
// in the workspace too (looked up again in the join: 82 us with 64 steps of six rows,
// 25.5 with 24 ragged sequences, now 77 and 20). Results do not depend on timing.
// Tried and slower: one copying warp with bulk copies (128 tokens 479 us against
// 244), the next granule's scores between this one's exponentials and products
// (six rows 94 us against 82), whose registers cost more than the wait.
#include <cuda_runtime.h>
#include <stdint.h>

#include "paged.cuh"

namespace moe {

int64_t attend_paged_workspace(const moe_attend_paged_io_t &io, const moe_kv_cache_t &c, int num_sms) {
  return workspace_of<false>(io, c, num_sms);
}

cudaError_t launch_attend_paged(const moe_attend_paged_io_t &io, const moe_kv_cache_t &c, void *workspace,
                                int64_t workspace_bytes, int32_t *status, int num_sms, cudaStream_t st) {
  return launch_paged<false>(io, nullptr, c, workspace, workspace_bytes, status, num_sms, st);
}

}  // namespace moe
