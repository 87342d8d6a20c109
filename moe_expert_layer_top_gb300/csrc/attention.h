// attention.h — arguments and launchers of the attention kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "moe.h"

namespace moe {

constexpr int kMaxSeqs = 4096;  // sequences of one attention call

// A capacity as the checks of the bounds-checked build see it: half of it under MOE_FLAG_TEST_BOUNDS.
inline int64_t checked_capacity(int64_t n, uint32_t flags) { return flags & MOE_FLAG_TEST_BOUNDS ? n / 2 : n; }

cudaError_t launch_qkv_append(const moe_qkv_append_io_t &io, const moe_kv_cache_t *cache, int32_t *status,
                              int num_sms, cudaStream_t st);
int64_t attend_paged_workspace(const moe_attend_paged_io_t &io, const moe_kv_cache_t &c, int num_sms);
cudaError_t launch_attend_paged(const moe_attend_paged_io_t &io, const moe_kv_cache_t &c, void *workspace,
                                int64_t workspace_bytes, int32_t *status, int num_sms, cudaStream_t st);
int64_t attend_prompt_workspace(const moe_attend_prompt_io_t &io, int num_sms);
cudaError_t launch_attend_prompt(const moe_attend_prompt_io_t &io, int32_t *status, int num_sms, cudaStream_t st);

}  // namespace moe
