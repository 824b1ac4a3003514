// The attention kernels' launches (defined in q8_attn_decode.cu and q8_attn_prefill.cu) and the layout of their
// workspace.
#pragma once

#include "q8_kv.h"

namespace q8 {

// Workspace: the join counters of the decode kernel (zero between calls), then the partial results.
constexpr int kAttnMaxCtas = 256;                                  // more than this GPU's SMs
constexpr long long kAttnCounterBytes = 4096;
constexpr int kDecodeHeads = 16;                                   // most query heads of a decode partial
constexpr long long kDecodePartFloats = kDecodeHeads * (128 + 2);  // O, then (m, l)
constexpr long long kAttnWorkspaceBytes = 64ll << 20;
static_assert(kAttnMaxCtas * 4 <= kAttnCounterBytes, "");
static_assert(kAttnCounterBytes + kAttnMaxCtas * 2 * kDecodePartFloats * 4 <= kAttnWorkspaceBytes, "");

cudaError_t launch_attn_decode(const AttnArgs &a, int dim, bool q8, cudaStream_t stream);
cudaError_t sm_count_of_device(int *sms);  // q8_attn.cu

}  // namespace q8
