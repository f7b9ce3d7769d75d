// pages.cu -- the pages of the cache on the device: copying, forking, growing, ending and
// compacting requests over a pool of reference-counted pages.
//
// The books are page_table [R, max_pages] (rows pt_stride apart), seq_lens [R] and refs [P].  A
// page is free where its count is 0, and the k-th page that a call takes is the free page of
// rank k,
//   rank(x) = #{y < x : refs[y] == 0},
// so what a call does follows from the books alone: the only atomics are sums and minima of
// integers, whose order does not show.
//
// Finding ranks is one scan of refs.  One cluster of kScanCtas CTAs does it in one launch: each
// CTA counts its contiguous share, the counts are exchanged over distributed shared memory, and
// a second walk over the share (now in L1/L2) hands out the ranks.  A grid-wide scan would take
// a second launch for the same exchange, and a single CTA reads 1 MB of counts (a pool of 262144
// pages) at one SM's rate.  What has to be copied then goes over the whole GPU in a second launch,
// a side (K or V) of a page per CTA: 6.0 TB/s, 0.92 of a plain copy's rate, for 6000 pages of 64 KB.
// Small calls are bound by their launches: a fork of 4 requests of a pool of 1000 pages takes two
// of ~5 us each on the GPU, and 13 us on the host.
#include "common.cuh"
#include "pages.cuh"

namespace vt {

namespace {

constexpr int kScanCtas = 8;
constexpr int kScanThreads = 1024;
constexpr int kScanTile = kScanThreads * 4;  // counts per step: an int4 each
// A pool of up to this many pages is scanned by one CTA: one step of its threads, against a
// cluster's launch and barriers of eight CTAs.  One CTA and a cluster, in a chain of calls: a
// compaction in which nothing moves 7.4 and 8.4 us (500 pages), 8.8 and 9.8 (4096), 11.5 and 9.9
// (8192), 14.0 and 10.1 (12000), 21.9 and 10.2 (24000); a growth of 4 rows 9.1 and 9.4 (4096), 9.6
// and 9.8 (8192), 10.3 and 9.8 (12000), 10.7 and 9.6 (24000).
constexpr int64_t kOneCta = kScanTile;

// Page count of `len` tokens (len >= 0, also close to 2^31).
__device__ __forceinline__ int pages_of(int len) { return len / kPage + (len % kPage != 0); }

// Exclusive prefix sum over the block's threads; `total` gets the sum.  Two barriers.
__device__ __forceinline__ int block_excl(int v, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // s_warp is free again
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
    const int c = s_warp[w];
    before += w < warp ? c : 0;
    all += c;
  }
  total = all;
  return before + x - v;
}

__device__ __forceinline__ int block_sum(int v, int* s_warp) {
  int total;
  block_excl(v, s_warp, total);
  return total;
}

// refs[x .. x+3], entries at or behind `end` read as `fill`.
__device__ __forceinline__ int4 load4(const int32_t* refs, int64_t x, int64_t end, int fill) {
  int4 r;
  if (x + 4 <= end && ((reinterpret_cast<uintptr_t>(refs + x) & 15u) == 0))
    return *reinterpret_cast<const int4*>(refs + x);
  r.x = x < end ? refs[x] : fill;
  r.y = x + 1 < end ? refs[x + 1] : fill;
  r.z = x + 2 < end ? refs[x + 2] : fill;
  r.w = x + 3 < end ? refs[x + 3] : fill;
  return r;
}

// Used pages in [lo, hi), counted by the block.
__device__ __forceinline__ int count_used(const int32_t* refs, int64_t lo, int64_t hi,
                                          int* s_warp) {
  int c = 0;
  for (int64_t x = lo + (int64_t)threadIdx.x * 4; x < hi; x += kScanTile) {
    const int4 r = load4(refs, x, hi, 0);
    c += (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
  }
  return block_sum(c, s_warp);
}

struct Share {
  int64_t lo, hi;  // this CTA's pages
};

template <int CTAS>
__device__ __forceinline__ Share my_share(int64_t P, int rank) {
  const int64_t tiles = (P + kScanTile - 1) / kScanTile;
  const int64_t per = (tiles + CTAS - 1) / CTAS * kScanTile;
  Share s;
  s.lo = min(P, per * rank);
  s.hi = min(P, s.lo + per);
  return s;
}

// The list side of a fork or growth, by CTA 0: which entries count, how many pages each needs
// (base: exclusive sums of the needs), and the total.  A target row carries -(n - i) while the
// call runs: the minimum over the entries that name it is its first entry.
//
// Lists of up to kListSmem entries stay in shared memory (and reach the other CTAs from there):
// the search of a free page's entry takes a step per bit of n, and in global memory each was a
// trip to L2 (a fork of 256: 28 us).
struct Lists {
  int *len, *need, *base;
};

template <bool FORK>
__device__ int read_list(const PageListParams& p, const Lists& a, int* s_warp) {
  const int n = p.n;
  for (int i = threadIdx.x; i < n; i += kScanThreads) {
    const int row = p.targets[i], source = p.sources[i];
    int len = -1, need = 0, bad = 0;
    if (row < 0 || row >= p.rows) {
      bad = VT_DEV_BAD_REQ;
    } else if (FORK) {
      if (source < 0 || source >= p.rows || p.seq_lens[row] != 0) {
        bad = VT_DEV_BAD_REQ;
      } else {
        len = p.seq_lens[source];
        if (len <= 0) bad = VT_DEV_BAD_REQ;
        else if (pages_of(len) > p.max_pages) bad = VT_DEV_BAD_LEN;
        need = len % kPage != 0;
      }
    } else {
      len = p.seq_lens[row];
      const int64_t grown = (int64_t)len + source;
      if (len < 0 || source < 0 || grown > p.max_pages * kPage || grown > INT32_MAX)
        bad = VT_DEV_BAD_LEN;
      else
        need = pages_of((int)grown) - pages_of(len);
    }
    if (bad) flag(p.status, bad);
    a.len[i] = bad ? -1 : len;
    a.need[i] = need;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kScanThreads)
    if (a.len[i] >= 0) atomicMin(&p.seq_lens[p.targets[i]], i - n);
  __threadfence();
  __syncthreads();
  int carry = 0;
  for (int i0 = 0; i0 < n; i0 += kScanThreads) {
    const int i = i0 + threadIdx.x;
    int need = 0;
    if (i < n && a.len[i] >= 0) {
      if (__ldcg(&p.seq_lens[p.targets[i]]) == i - n) {
        need = a.need[i];
      } else {  // an earlier entry has the row
        a.len[i] = -1;
        flag(p.status, VT_DEV_BAD_REQ);
      }
    }
    int total;
    const int base = block_excl(need, s_warp, total);
    // sums saturate: one past 2^31 is above every pool's free pages
    if (i < n) {
      a.need[i] = need;
      a.base[i] = (int)min((int64_t)INT32_MAX, (int64_t)carry + base);
    }
    carry = (int)min((int64_t)INT32_MAX, (int64_t)carry + total);
  }
  return carry;
}

template <bool FORK, int CTAS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kScanThreads, 1)
    page_list_kernel(const PageListParams p) {
  __shared__ int s_warp[kScanThreads / 32];
  __shared__ int s_free, s_need;
  __shared__ int s_list[3][kListSmem];
  cg::cluster_group cluster = cg::this_cluster();
  let_next_launch();
  const int rank = (int)cluster.block_rank();
  const Share sh = my_share<CTAS>(p.num_pages, rank);
  const bool small = p.n <= kListSmem;
  const Lists a = small ? Lists{s_list[0], s_list[1], s_list[2]} : Lists{p.len, p.need, p.base};
  if (rank == 0) {
    const int need = read_list<FORK>(p, a, s_warp);
    if (threadIdx.x == 0) s_need = need;
  }
  const int n_used = count_used(p.refs, sh.lo, sh.hi, s_warp);
  if (threadIdx.x == 0) s_free = (int)(sh.hi - sh.lo) - n_used;
  cluster.sync();
  int before = 0, n_free = 0;
  for (int r = 0; r < CTAS; ++r) {
    const int c = *cluster.map_shared_rank(&s_free, r);
    before += r < rank ? c : 0;
    n_free += c;
  }
  const int total = *cluster.map_shared_rank(&s_need, 0);
  const int want = min(total, n_free);
  if (small && rank != 0 && before < want) {
    const int* from = cluster.map_shared_rank(&s_list[0][0], 0);
    for (int k = 0; k < 3; ++k)
      for (int i = threadIdx.x; i < p.n; i += kScanThreads)
        s_list[k][i] = from[k * kListSmem + i];
    __syncthreads();
  }
  // hand the free pages of this share out, lowest first
  int at = before;
  for (int64_t x0 = sh.lo; x0 < sh.hi && at < want; x0 += kScanTile) {
    const int64_t x = x0 + (int64_t)threadIdx.x * 4;
    const int4 r = load4(p.refs, x, sh.hi, 1);
    const int f[4] = {r.x <= 0, r.y <= 0, r.z <= 0, r.w <= 0};
    int sum;
    int k = at + block_excl(f[0] + f[1] + f[2] + f[3], s_warp, sum);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (!f[e]) continue;
      if (k < want) {
        int lo = 0, hi = p.n - 1;  // the last entry whose base is <= k needs this page
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (a.base[mid] <= k) lo = mid; else hi = mid - 1;
        }
        const int need = a.need[lo], base = a.base[lo];
        if ((int64_t)base + need <= n_free) {
          const int len = a.len[lo];
          const int page = (int)(x + e);
          // a fork's own page stands for the parent's partly filled last one
          const int slot = FORK ? len / kPage : pages_of(len) + (k - base);
          p.page_table[(int64_t)p.targets[lo] * p.pt_stride + slot] = page;
          p.refs[page] = 1;
        }
      }
      ++k;
    }
    at += sum;
  }
  if (rank == 0) {
    for (int i = threadIdx.x; i < p.n; i += kScanThreads) {
      const int len = a.len[i];
      bool served = false;
      if (len >= 0) {
        served = (int64_t)a.base[i] + a.need[i] <= n_free || a.need[i] == 0;
        if (!served) flag(p.status, VT_DEV_NO_PAGE);
        p.seq_lens[p.targets[i]] = FORK ? (served ? len : 0) : (served ? len + p.sources[i] : len);
      }
      if (FORK) p.len[i] = served ? len : -1;  // for the copies
    }
  }
  cluster.sync();  // (no CTA leaves while another reads its shared memory)
}

// One page's rows of one pool, by the whole block: 16-byte pieces, kUnroll of them in flight in
// each thread.
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;
// CTAs of a compaction's second launch, per SM and side; each takes several moves and rows.  2, 4
// and 8 take the same time (158 us for 5.6 k moves, 18 for a small pool), 16 2 us more.
constexpr int kApplyCtas = 8;

__device__ __forceinline__ void copy_page(const PoolView& v, int64_t dst, int64_t src) {
  const int per_head = v.dim / 8, per_tok = v.heads * per_head, total = kPage * per_tok;
  const __nv_bfloat16* s = v.base + src * v.s_p;
  __nv_bfloat16* d = v.base + dst * v.s_p;
  for (int i0 = threadIdx.x; i0 < total; i0 += kCopyThreads * kCopyUnroll) {
    uint4 r[kCopyUnroll];
    int64_t off[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
      const int i = i0 + u * kCopyThreads;
      const int t = i / per_tok, c = i - t * per_tok, h = c / per_head;
      off[u] = t * v.s_t + h * v.s_h + (int64_t)(c - h * per_head) * 8;
      if (i < total) r[u] = ld_stream_u4(s + off[u]);
    }
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
      if (i0 + u * kCopyThreads < total) *reinterpret_cast<uint4*>(d + off[u]) = r[u];
  }
}

// what is behind a page's first kCopyThreads pieces of centroids
__device__ __forceinline__ void copy_centroids(float* c, int64_t row, int64_t dst, int64_t src) {
  for (int64_t i = threadIdx.x + kCopyThreads; i < row / 4; i += kCopyThreads)
    reinterpret_cast<float4*>(c + dst * row)[i] = ld_stream_f4(c + src * row + i * 4);
}

// blockIdx.y: 0 the K pool (and the centroids), 1 the V pool
__device__ __forceinline__ void copy_side(const PagePools& pools, int side, int64_t dst,
                                          int64_t src) {
  if (side == 0) {
    // (the centroids' first piece is in flight beside the page)
    const bool cent = pools.centroids && threadIdx.x < pools.cent_row / 4;
    float4 first;
    if (cent)
      first = ld_stream_f4(pools.centroids + src * pools.cent_row + threadIdx.x * 4);
    copy_page(pools.k, dst, src);
    if (cent)
      reinterpret_cast<float4*>(pools.centroids + dst * pools.cent_row)[threadIdx.x] = first;
    if (pools.centroids) copy_centroids(pools.centroids, pools.cent_row, dst, src);
  } else {
    copy_page(pools.v, dst, src);
  }
}

__global__ void __launch_bounds__(kCopyThreads)
    copy_pages_kernel(const PagePools pools, const int32_t* src, const int32_t* dst,
                      int32_t* status) {
  const int s = src[blockIdx.x], d = dst[blockIdx.x];
  if (s < 0 || d < 0 || s >= pools.num_pages || d >= pools.num_pages) {
    if (threadIdx.x == 0) flag(status, VT_DEV_BAD_PAGE);
    return;
  }
  copy_side(pools, blockIdx.y, d, s);
}

// The rows and shared references of the forks that were served (blockIdx.y 0), and their copies
// of a partly filled last page.
__global__ void __launch_bounds__(kCopyThreads)
    fork_apply_kernel(const PagePools pools, const PageListParams p) {
  const int i = blockIdx.x;
  wait_for_previous();
  const int len = p.len[i];
  if (len < 0) return;
  const int32_t* from = p.page_table + (int64_t)p.sources[i] * p.pt_stride;
  int32_t* to = p.page_table + (int64_t)p.targets[i] * p.pt_stride;
  const int full = len / kPage;
  if (blockIdx.y == 0)
    for (int k = threadIdx.x; k < full; k += kCopyThreads) {
      const int page = from[k];
      to[k] = page;
      if (page < 0 || page >= pools.num_pages) flag(p.status, VT_DEV_BAD_PAGE);
      else atomicAdd(&p.refs[page], 1);
    }
  if (len % kPage != 0) {
    const int s = from[full], d = to[full];
    if (s < 0 || s >= pools.num_pages) {
      if (threadIdx.x == 0) flag(p.status, VT_DEV_BAD_PAGE);
    } else {
      copy_side(pools, blockIdx.y, d, s);
    }
  }
}

__global__ void __launch_bounds__(kCopyThreads)
    free_kernel(int rows, const int32_t* page_table, int64_t pt_stride, int64_t max_pages,
                int32_t* seq_lens, int32_t* refs, int64_t num_pages, const int32_t* requests,
                int32_t* status) {
  __shared__ int s_len;
  const int row = requests[blockIdx.x];
  if (row < 0 || row >= rows) {
    if (threadIdx.x == 0) flag(status, VT_DEV_BAD_REQ);
    return;
  }
  if (threadIdx.x == 0) s_len = atomicExch(&seq_lens[row], 0);  // of two entries, one frees it
  __syncthreads();
  if (s_len <= 0) return;
  int n = pages_of(s_len);
  if (n > max_pages) {
    if (threadIdx.x == 0) flag(status, VT_DEV_BAD_LEN);
    n = (int)max_pages;
  }
  for (int k = threadIdx.x; k < n; k += kCopyThreads) {
    const int page = page_table[(int64_t)row * pt_stride + k];
    if (page < 0 || page >= num_pages) {
      flag(status, VT_DEV_BAD_PAGE);
    } else if (atomicSub(&refs[page], 1) <= 0) {
      atomicAdd(&refs[page], 1);
      flag(status, VT_DEV_BAD_REF);
    }
  }
}

// Moves of a compaction.  With used(x) = #{y < x : refs[y] > 0} and u = used(P): the free page
// x < u has rank x - used(x) among the free ones, the used page x >= u has rank
// used(x) - used(u) among those that move.
template <int CTAS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kScanThreads, 1)
    compact_plan_kernel(const CompactParams p) {
  __shared__ int s_warp[kScanThreads / 32];
  __shared__ int s_used, s_below;
  cg::cluster_group cluster = cg::this_cluster();
  let_next_launch();
  const int rank = (int)cluster.block_rank();
  const Share sh = my_share<CTAS>(p.num_pages, rank);
  const int mine = count_used(p.refs, sh.lo, sh.hi, s_warp);
  if (threadIdx.x == 0) s_used = mine;
  cluster.sync();
  int before = 0, u = 0;
  for (int r = 0; r < CTAS; ++r) {
    const int c = *cluster.map_shared_rank(&s_used, r);
    before += r < rank ? c : 0;
    u += c;
  }
  // this share's part of used(u)
  const int64_t cut = min(sh.hi, (int64_t)u);
  const int below = cut >= sh.hi ? mine : cut <= sh.lo ? 0 : count_used(p.refs, sh.lo, cut, s_warp);
  if (threadIdx.x == 0) s_below = below;
  cluster.sync();
  int used_u = 0;
  for (int r = 0; r < CTAS; ++r) used_u += *cluster.map_shared_rank(&s_below, r);
  if (rank == 0 && threadIdx.x == 0) {
    *p.n_used = u;
    *p.n_moves = u - used_u;
  }
  int at = before;
  for (int64_t x0 = sh.lo; x0 < sh.hi; x0 += kScanTile) {
    const int64_t x = x0 + (int64_t)threadIdx.x * 4;
    const int4 r = load4(p.refs, x, sh.hi, 0);
    const int f[4] = {r.x > 0, r.y > 0, r.z > 0, r.w > 0};
    int sum;
    int k = at + block_excl(f[0] + f[1] + f[2] + f[3], s_warp, sum);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t id = x + e;
      if (id < sh.hi) {
        p.move_of[id] = !f[e] ? -1 : id < u ? 0 : k - used_u;
        if (id >= u) {
          if (f[e]) p.src[k - used_u] = (int)id;
        } else if (!f[e]) {
          p.dst[id - k] = (int)id;
        }
      }
      k += f[e];
    }
    at += sum;
  }
  cluster.sync();
}

__global__ void __launch_bounds__(kCopyThreads)
    compact_apply_kernel(const PagePools pools, const CompactParams p) {
  wait_for_previous();
  const int moves = *p.n_moves, u = *p.n_used;
  for (int m = blockIdx.x; m < moves; m += gridDim.x) {
    const int s = p.src[m], d = p.dst[m];
    copy_side(pools, blockIdx.y, d, s);
    if (blockIdx.y == 0 && threadIdx.x == 0) {
      p.refs[d] = p.refs[s];
      p.refs[s] = 0;
    }
  }
  if (blockIdx.y != 0) return;
  for (int row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const int len = p.seq_lens[row];
    if (len <= 0) continue;
    int n = pages_of(len);
    if (n > p.max_pages) {
      if (threadIdx.x == 0) flag(p.status, VT_DEV_BAD_LEN);
      n = (int)p.max_pages;
    }
    int32_t* t = p.page_table + (int64_t)row * p.pt_stride;
    for (int k = threadIdx.x; k < n; k += kCopyThreads) {
      const int page = t[k];
      if (page < 0 || page >= p.num_pages) {
        flag(p.status, VT_DEV_BAD_PAGE);
      } else {  // (the counts change meanwhile; what the plan noted of them does not)
        const int m = p.move_of[page];
        if (m < 0) flag(p.status, VT_DEV_BAD_REF);
        else if (page >= u) t[k] = p.dst[m];
      }
    }
  }
}

}  // namespace

cudaError_t launch_copy_pages(const PagePools& pools, const int32_t* src, const int32_t* dst, int n,
                              int sides, int32_t* status, cudaStream_t s) {
  copy_pages_kernel<<<dim3(n, sides), kCopyThreads, 0, s>>>(pools, src, dst, status);
  return cudaGetLastError();
}

cudaError_t launch_fork(const PagePools& pools, const PageListParams& p, int sides,
                        cudaStream_t s) {
  if (p.num_pages <= kOneCta) page_list_kernel<true, 1><<<1, kScanThreads, 0, s>>>(p);
  else page_list_kernel<true, kScanCtas><<<kScanCtas, kScanThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_after(fork_apply_kernel, dim3(p.n, sides), kCopyThreads, s, pools, p);
}

cudaError_t launch_extend(const PageListParams& p, cudaStream_t s) {
  if (p.num_pages <= kOneCta) page_list_kernel<false, 1><<<1, kScanThreads, 0, s>>>(p);
  else page_list_kernel<false, kScanCtas><<<kScanCtas, kScanThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_free(const vt_page_books& b, int64_t max_pages, int64_t num_pages,
                        const int32_t* requests, int n, cudaStream_t s) {
  free_kernel<<<n, kCopyThreads, 0, s>>>(b.rows, b.page_table, b.pt_stride, max_pages, b.seq_lens,
                                         b.refs, num_pages, requests, b.status);
  return cudaGetLastError();
}

cudaError_t launch_compact(const PagePools& pools, const CompactParams& p, int sides, int sm_count,
                           cudaStream_t s) {
  if (p.num_pages <= kOneCta) compact_plan_kernel<1><<<1, kScanThreads, 0, s>>>(p);
  else compact_plan_kernel<kScanCtas><<<kScanCtas, kScanThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_after(compact_apply_kernel, dim3(sm_count * kApplyCtas, sides), kCopyThreads, s, pools, p);
}

}  // namespace vt
