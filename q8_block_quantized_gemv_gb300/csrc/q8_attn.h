// The attention kernels' launches (defined in q8_attn_decode.cu and q8_attn_prefill.cu) and the layout of their
// workspace.
#pragma once

#include "q8_kv.h"

namespace q8 {

// Workspace: the join counters of both kernels (zero between calls), then the parts, of one kernel or the other (the
// calls that share a workspace run one after another).  Each CTA leaves two parts at most.
constexpr int kAttnMaxCtas = 192;  // more than this GPU's SMs
constexpr long long kPrefillCounterAt = 2048, kAttnCounterBytes = 4096;
constexpr int kDecodeHeads = 16;                                   // most query heads of a decode part
constexpr long long kDecodePartFloats = kDecodeHeads * (128 + 2);  // O, then (m, l)
constexpr long long kPrefillPartAt = kAttnCounterBytes;
constexpr long long kPrefillPartFloats = 256 * (128 + 2);          // O of 256 rows, then (m, l)
constexpr long long kAttnWorkspaceBytes = kAttnCounterBytes + kAttnMaxCtas * 2 * kPrefillPartFloats * 4;
static_assert(kAttnMaxCtas * 4 <= kPrefillCounterAt, "");

cudaError_t launch_attn_decode(const AttnArgs &a, int dim, bool q8, cudaStream_t stream);
cudaError_t launch_attn_prefill(const AttnArgs &a, int dim, bool q8, cudaStream_t stream);
cudaError_t read_attn_fault(unsigned *out, bool clear);  // q8_attn_prefill.cu
cudaError_t sm_count_of_device(int *sms);                // q8_attn.cu

}  // namespace q8
