// attend_params.cuh -- what the host side (api.cu) and the kernels of the dense attention calls
// (vt_prefill, vt_shared_prefix_decode) share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "vt.h"

namespace vt {

struct AttendParams {
  vt_paged_kv kv;
  int Hkv, G, D;
  int B;             // requests
  int n_groups;      // shared prefix: groups; prompts: 0
  int64_t T;         // rows of q (tokens)
  const __nv_bfloat16* q;
  int64_t sq_t;      // elements between the rows of two tokens
  const int32_t* start;         // q_start [B+1], or group_start [n_groups+1]
  const int32_t* prefix_pages;  // [n_groups]; prompts: NULL
  const int32_t* page_table;
  int64_t pt_stride;
  int64_t max_pages;  // entries of a table row
  const int32_t* seq_lens;
  float qscale;      // sm_scale log2(e)
  int32_t* status;
  __nv_bfloat16* out;
  float* lse;
};

size_t attend_workspace_bytes(const AttendParams& p, int sm_count);
cudaError_t launch_attend(const AttendParams& p, void* ws, int sm_count, cudaStream_t s);

}  // namespace vt
