// pages.cuh -- what the page operations' host side (api.cu) and kernels (pages.cu) share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "vt.h"

namespace vt {

// Lists of up to this many entries are worked on in shared memory; longer ones in the workspace.
constexpr int kListSmem = 2048;

struct PoolView {
  __nv_bfloat16* base;
  int64_t s_p, s_t, s_h;
  int heads, dim;
};

struct PagePools {
  PoolView k, v;
  int64_t num_pages;
  float* centroids;  // or NULL
  int64_t cent_row;  // floats of one page's centroids
};

// A fork (sources: parents, targets: children) or growth (sources: tokens, targets: rows).
struct PageListParams {
  int rows;
  int32_t* page_table;
  int64_t pt_stride;
  int64_t max_pages;  // entries of a table row
  int32_t* seq_lens;
  int32_t* refs;
  int32_t* status;
  int64_t num_pages;
  const int32_t* sources;
  const int32_t* targets;
  int n;
  int32_t* len;   // workspace, n each (a growth of up to kListSmem rows: NULL): the entry's length
                  //   before the call, -1 left out
  int32_t* need;  //   pages it needs
  int32_t* base;  //   pages that the entries before it need
};

struct CompactParams {
  int rows;
  int32_t* page_table;
  int64_t pt_stride;
  int64_t max_pages;  // entries of a table row
  const int32_t* seq_lens;
  int32_t* refs;
  int32_t* status;
  int64_t num_pages;
  int32_t* n_used;
  int32_t* n_moves;  // workspace: one word, then num_pages words each
  int32_t* src;      //   the page of move m
  int32_t* dst;      //   where it goes
  int32_t* move_of;  //   -1 for a free page; the move of a used one at or above n_used, else 0
};

cudaError_t launch_copy_pages(const PagePools& pools, const int32_t* src, const int32_t* dst, int n,
                              int sides, int32_t* status, cudaStream_t s);
cudaError_t launch_fork(const PagePools& pools, const PageListParams& p, int sides, cudaStream_t s);
cudaError_t launch_extend(const PageListParams& p, cudaStream_t s);
cudaError_t launch_free(const vt_page_books& b, int64_t max_pages, int64_t num_pages,
                        const int32_t* requests, int n, cudaStream_t s);
cudaError_t launch_compact(const PagePools& pools, const CompactParams& p, int sides, int sm_count,
                           cudaStream_t s);

}  // namespace vt
