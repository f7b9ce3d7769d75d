// attend.cu -- dense attention over the paged cache: packed causal prompts (vt_prefill) and
// decode with shared prefixes (vt_shared_prefix_decode).
//
// One warp per (token, query head): the lanes split the head's dims, keys come one after the
// other, and the softmax runs with a running maximum and sum in base 2.
#include "attend_params.cuh"
#include "common.cuh"

namespace vt {

namespace {

// The page-table row, and the number of keys, of token t's query row; false: not computed.
struct RowKeys {
  const int32_t* table;    // its own row
  const int32_t* shared;   // where the first `n_shared` entries are
  int n_shared, keys;
  bool ok, bad;
};

__device__ bool starts_ok(const int32_t* start, int n, int64_t bound) {
  if (start[0] != 0) return false;
  for (int i = 0; i < n; ++i)
    if (start[i + 1] < start[i]) return false;
  return start[n] <= bound;
}

__device__ RowKeys row_keys(const AttendParams& p, int64_t t) {
  RowKeys r{};
  const int n = p.prefix_pages ? p.n_groups : p.B;
  if (t >= p.start[n]) return r;
  int lo = 0, hi = n - 1;  // the last entry that starts at or before t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.start[mid] <= t) lo = mid; else hi = mid - 1;
  }
  r.ok = true;
  const int b = p.prefix_pages ? (int)t : lo;
  const int len = p.seq_lens[b];
  r.table = r.shared = p.page_table + (int64_t)b * p.pt_stride;
  r.bad = len < 0 || len > p.pt_stride * kPage;
  if (p.prefix_pages) {
    r.shared = p.page_table + (int64_t)p.start[lo] * p.pt_stride;
    r.n_shared = p.prefix_pages[lo];
    r.bad |= r.n_shared < 0 || r.n_shared > p.pt_stride || len < 1 || len / kPage < r.n_shared;
    r.keys = len;
  } else {
    const int nq = p.start[lo + 1] - p.start[lo];
    r.bad |= len < nq;
    r.keys = len - nq + (int)(t - p.start[lo]) + 1;
  }
  if (r.bad) r.keys = 0;
  return r;
}

template <int D>
__global__ void __launch_bounds__(256) attend_rows_kernel(const AttendParams p) {
  constexpr int E = D / 32;  // dims of a lane: lane * E ..
  __shared__ int s_ok;
  if (threadIdx.x == 0)
    s_ok = starts_ok(p.start, p.prefix_pages ? p.n_groups : p.B, p.T);
  __syncthreads();
  if (!s_ok) {
    if (threadIdx.x == 0) flag(p.status, VT_DEV_BAD_START);
    return;
  }
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int Hq = p.Hkv * p.G;
  const int64_t t = w / Hq;
  if (t >= p.T) return;
  const int hq = (int)(w - t * Hq), h = hq / p.G;
  const RowKeys rk = row_keys(p, t);
  if (!rk.ok) return;
  if (rk.bad && lane == 0) flag(p.status, VT_DEV_BAD_LEN);
  float q[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(p.q[t * p.sq_t + (int64_t)hq * D + lane * E + e]);
    o[e] = 0.0f;
  }
  const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(p.kv.k_pool) + h * p.kv.sk_h;
  const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(p.kv.v_pool) + h * p.kv.sv_h;
  float m = -INFINITY, l = 0.0f;
  for (int j = 0; j < rk.keys; ++j) {
    const int page = (j / kPage < rk.n_shared ? rk.shared : rk.table)[j / kPage];
    if (page < 0 || page >= p.kv.num_pages) {
      if (lane == 0) flag(p.status, VT_DEV_BAD_PAGE);
      j |= kPage - 1;
      continue;
    }
    const __nv_bfloat16* kr = kp + page * p.kv.sk_p + (j % kPage) * p.kv.sk_t + lane * E;
    const __nv_bfloat16* vr = vp + page * p.kv.sv_p + (j % kPage) * p.kv.sv_t + lane * E;
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], __bfloat162float(kr[e]), s);
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(kFull, s, x);
    s *= p.qscale;
    const float mn = fmaxf(m, s);
    const float f = exp2f(m - mn), pr = exp2f(s - mn);
    l = fmaf(l, f, pr);
    m = mn;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(pr, __bfloat162float(vr[e]), o[e] * f);
  }
  const int64_t row = t * Hq + hq;
#pragma unroll
  for (int e = 0; e < E; ++e)
    p.out[row * D + lane * E + e] = __float2bfloat16(l > 0.0f ? o[e] / l : 0.0f);
  if (p.lse && lane == 0) p.lse[row] = l > 0.0f ? m * kLn2 + logf(l) : -INFINITY;
}

}  // namespace

size_t attend_workspace_bytes(const AttendParams&, int) { return 256; }

cudaError_t launch_attend(const AttendParams& p, void*, int, cudaStream_t s) {
  const int64_t blocks = (p.T * p.Hkv * p.G + 7) / 8;
  if (p.D == 128) attend_rows_kernel<128><<<(unsigned)blocks, 256, 0, s>>>(p);
  else attend_rows_kernel<64><<<(unsigned)blocks, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace vt
