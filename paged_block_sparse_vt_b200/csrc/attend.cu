// attend.cu -- dense attention over the paged cache on the fifth-generation tensor cores: packed
// causal prompts (vt_prefill) and decode with shared prefixes (vt_shared_prefix_decode).
//
// Rows.  The G query heads of a KV head see the same keys, so the rows of a tile are (token,
// head) pairs, token first: 128 rows hold 128/G tokens, and one token of a decode call fills G of
// them.  An item is two row tiles (256 rows), or one where there are no more tokens, against its
// keys in steps of 128 (eight pages).
//
// One step, for either row tile t, with everything fp32 but the operands of the products:
//   S_t = Q_t K^T                (tcgen05, 128 x 128 in tensor memory)
//   m   = max(m, max_j S_t[r, j]), l = l f + sum_j p_j, p_j = 2^(c S_t[r, j] - c m), c = scale log2 e
//   P_t = bf16(p)                (over the columns of S_t)
//   O_t = O_t f + P_t V          (tcgen05, P_t read from tensor memory)
// A warpgroup has one tile, a thread one row, so no sum or maximum crosses lanes.  f = 1 unless
// the maximum rose: O_t is rescaled only when it rose by more than 2^kLazy since the last time
// (until then p <= 2^kLazy, which loses nothing in bf16 or in fp32).
//
// One warp loads: K and V tiles alternate in a ring of shared-memory stages, each of them 8
// pages by TMA in 128-byte swizzled boxes of 16 tokens x 64 dims, straight from the pools through
// the page table.  The page that holds a request's last token is loaded from a negative token
// coordinate, so that its tokens stand at the END of its 16 rows and the hardware fills the rest
// with zeros: whatever the pool holds behind a request's end never gets into a product (0 x NaN
// would spoil the row).  One warp issues all products; they complete in the order of issue,
// which is why S_t of the next step may overwrite P_t as soon as P_t V is issued.
//
// Work is cut into equal shares of the whole batch, across items where need be (attend_plan.cuh);
// an item that falls into several shares leaves unnormalised partial rows with their m and l, and
// a second launch joins those: out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i.
#include <cuda.h>

#include "attend_params.cuh"
#include "attend_plan.cuh"
#include "common.cuh"
#include "umma.cuh"

namespace vt {

namespace {

constexpr int kThreads = 384;   // two softmax warpgroups, and one with the loading and product warps
// Registers: a softmax thread holds its row of scores, 128 of them, beside the rest; what the
// third warpgroup gives up goes to the other two (2 * 200 + 104 = 3 * 168, the launch's share).
constexpr int kRegsSoftmax = 200, kRegsOther = 104;
constexpr int kLoadWarp = 8, kMmaWarp = 9;
constexpr int kDescs = 6;       // items described ahead
constexpr int kBadRing = 16;    // key tiles whose page checks are kept (> tiles in flight)
constexpr int kPlan = 1024;     // entries of the cost table in shared memory
constexpr float kLazy = 8.0f;
constexpr int kPagesTile = kKeys / kPage;
constexpr int kSoftWarps = 8;
constexpr int kSmall = 32;      // rows of a small item
constexpr int kStage = 32 * 128;  // a softmax warp's staging: 128 bytes of each of its rows

template <int D>
struct Cfg {
  static constexpr int HALVES = D / 64;              // 64-dim boxes of a row
  static constexpr int BOX = kKeys * 128;            // bytes of one half of a tile
  static constexpr int TILE = HALVES * BOX;          // bytes of a Q, K or V tile
  // wide: two Q tiles, 128 KB of K and V, staging of all softmax warps
  static constexpr int STAGES = D == 128 ? 4 : 8;
  static constexpr int WIDE = 2 * TILE + kSoftWarps * kStage + STAGES * TILE;
  // narrow: one Q tile, 192 KB of K and V.  Items of up to kSmall rows fill only the first of the
  // four parts of that tile; the second stages their results.  (The product reads 128 rows of Q
  // all the same; the others are what stands there, and nobody looks at their results.)  Larger
  // ones stage theirs over their own Q, so the next Q waits for them.
  static constexpr int Q_SMALL = kSmall * 128;  // bytes of one half
  static constexpr int STAGES_NARROW = D == 128 ? 6 : 12;
  static constexpr int NARROW = TILE + STAGES_NARROW * TILE;
  static constexpr int SMEM = 1024 + (WIDE > NARROW ? WIDE : NARROW);
};

// What the loading warp tells the others about a piece of an item.
struct Desc {
  int tok0;            // first query token
  int n_tok;           // tokens of the item; 0: no more items
  int h;               // KV head
  int j0, j1;          // key tiles [j0, j1)
  int vis0, step;      // keys seen by token i of the item: vis0 + i step
  int kv_len;          // valid keys
  int slot;            // where a partial result goes: -1 none (write out), else see below
  int whole;           // 1: all key tiles
  int prefix;          // the item is a shared prefix
};

// A header of a partial slot.
struct Head {
  int tok0, n_tok, h, j0, j1, n_tiles, valid, pad;
};

struct Work {          // the workspace
  Head* head;          // [2 ctas]
  float* part;         // prompts: [2 ctas][256][D + 4]: slot 2c continues an item in CTA c, slot
                       //   2c + 1 begins one; shared prefixes: [ctas][256][D + 4], slot c continues
  float* first;        // shared prefixes: [2][B Hq][D + 4], the rows of items' first pieces:
                       //   prefixes, then own pages
  int64_t* line;       // shared prefixes: [units + 2] where each unit begins in its line, and the
                       //   lengths of the two lines
};

// A partial row: O, then m (scaled, base 2) and l; padded to 16 bytes.
template <int D>
constexpr int kRowF = D + 4;

struct Shared {
  Desc desc[kDescs];
  int bad[kBadRing];
  uint64_t q_full, q_empty, s_full[2], p_ready[2][2], o_full[2], desc_full[kDescs],
      desc_empty[kDescs], kv_full[12], kv_empty[12], hand[4], back[4], out_done[2], drain;
  float2 ml[kTile];  // m and l of the second warpgroup's rows, where it shares the first's
  uint32_t tmem;
  int abort;
};

// ---- the units ------------------------------------------------------------------------------

template <bool SHARED>
__device__ __forceinline__ int unit_count(const AttendParams& p) {
  return SHARED ? p.n_groups + p.B : p.B;
}

// The group of request b, or -1: groups are few and their starts stay in L1.
__device__ __forceinline__ int group_of(const AttendParams& p, int b) {
  if (b >= p.start[p.n_groups]) return -1;
  int lo = 0, hi = p.n_groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.start[mid] <= b) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Pages that a group shares as far as this call goes (a group of one shares with nobody); -1 bad.
__device__ __forceinline__ int group_prefix(const AttendParams& p, int g) {
  const int pages = p.prefix_pages[g];
  if (pages < 0 || pages > p.pt_stride) return -1;
  return p.start[g + 1] - p.start[g] >= 2 ? pages : 0;
}

template <bool SHARED>
__device__ Unit load_unit_raw(const AttendParams& p, int u) {
  Unit x{};
  if (!SHARED) {
    const int len = p.seq_lens[u];
    x.tok0 = p.start[u];
    x.n = p.start[u + 1] - x.tok0;
    x.row = u;
    if (x.n == 0) return x;  // whatever its length
    x.bad = len < x.n || len > p.pt_stride * kPage;
    x.kv_len = x.bad ? 0 : len;
    x.vis0 = x.bad ? 0 : len - x.n + 1;
    x.step = x.bad ? 0 : 1;
  } else if (u < p.n_groups) {
    const int pages = group_prefix(p, u);
    x.tok0 = x.row = p.start[u];
    if (pages > 0) x.n = p.start[u + 1] - x.tok0;
    x.kv_len = x.vis0 = max(pages, 0) * kPage;
  } else {
    const int b = u - p.n_groups, g = group_of(p, b);
    x.tok0 = x.row = b;
    if (g < 0) return x;
    x.n = 1;
    const int len = p.seq_lens[b], pages = group_prefix(p, g);
    x.bad = pages < 0 || len < 1 || len > p.pt_stride * kPage ||
            len < p.prefix_pages[g] * kPage;
    x.page0 = max(pages, 0);
    x.kv_len = x.vis0 = x.bad ? 0 : len - x.page0 * kPage;
  }
  return x;
}

template <bool SHARED>
__device__ __forceinline__ Unit load_unit(const AttendParams& p, int u) {
  Unit x = load_unit_raw<SHARED>(p, u);
  x.narrow = x.n <= kTile / p.G;
  return x;
}

// ---- bounded waits --------------------------------------------------------------------------

__device__ __forceinline__ bool wait(uint32_t bar, uint32_t phase, volatile int* abort_flag) {
  for (int i = 0; i < 64; ++i)
    if (umma::mbar_try_wait(bar, phase)) return true;
  const unsigned long long t0 = global_ns();
  while (!umma::mbar_try_wait(bar, phase)) {
    if (*abort_flag) return false;
    if (global_ns() - t0 > kWaitNs) {
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two floats in one register pair, and the two-wide arithmetic on them
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float total2(uint64_t a, uint64_t b) {
  float x0, y0, x1, y1;
  unpair(a, x0, y0);
  unpair(b, x1, y1);
  return (x0 + y0) + (x1 + y1);
}
// 2^x of a pair on the special-function units
__device__ __forceinline__ uint64_t exp2_unit(uint64_t x) {
  float a, b;
  unpair(x, a, b);
  return pair(ex2(a), ex2(b));
}
// two floats rounded to a bf16 pair, `lo` in the low half
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t pack2(uint64_t p) {
  float lo, hi;
  unpair(p, lo, hi);
  return pack2(lo, hi);
}

__device__ __forceinline__ void st_shared16(uint32_t a, uint32_t x, uint32_t y, uint32_t z,
                                            uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n"
               :
               : "r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// 32 bits, one for each key slot of a 32-wide column block that the row may use.
struct RowMask {
  int lim;            // slots below lim are visible ...
  int hole0, hole1;   // ... but for these
  uint32_t bad;       // pages of the tile that take no part, one bit each
  __device__ __forceinline__ static uint32_t below(int n) {  // the n low bits
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
  }
  __device__ __forceinline__ uint32_t word(int w) const {
    uint32_t m = below(lim - 32 * w);
    m &= ~(below(hole1 - 32 * w) & ~below(hole0 - 32 * w));
    if (bad >> (2 * w) & 1u) m &= 0xffff0000u;
    if (bad >> (2 * w + 1) & 1u) m &= 0x0000ffffu;
    return m;
  }
};

// ---- the kernel -----------------------------------------------------------------------------

template <int N>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" : : "n"(N));
}
template <int N>
__device__ __forceinline__ void regs_less() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" : : "n"(N));
}

template <int D, bool SHARED>
__global__ void __launch_bounds__(kThreads, 1)
    attend_kernel(const AttendParams p, const Work w, const __grid_constant__ CUtensorMap q_map,
                  const __grid_constant__ CUtensorMap q1_map,
                  const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map) {
  using C = Cfg<D>;
  extern __shared__ unsigned char raw[];
  __shared__ Shared sh;
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tpt = kTile / p.G;
  const int cta = blockIdx.x;
  volatile int* abort_flag = &sh.abort;
  // the cost tables of both lines lie where q comes later
  int64_t* table0 = reinterpret_cast<int64_t*>(raw + (base - smem_u32(raw)));
  int64_t* table1 = table0 + kPlan + 1;

  // The starts, then the cost of every unit, summed up over entries of `per` units each.
  const int units = unit_count<SHARED>(p);
  const int n_start = SHARED ? p.n_groups : p.B;
  bool fine = true;
  for (int i = threadIdx.x; i < n_start; i += kThreads)
    fine &= p.start[i + 1] >= p.start[i] && (i > 0 || p.start[0] == 0);
  fine &= p.start[n_start] <= p.T;
  if (warp == kMmaWarp) umma::tmem_alloc(smem_u32(&sh.tmem), 512);
  if (threadIdx.x == 0) {
    sh.abort = 0;
    umma::mbar_init(smem_u32(&sh.q_full), 1);
    umma::mbar_init(smem_u32(&sh.q_empty), 1);
    umma::mbar_init(smem_u32(&sh.out_done[0]), 4);
    umma::mbar_init(smem_u32(&sh.out_done[1]), 4);
    umma::mbar_init(smem_u32(&sh.drain), 1);
    for (int t = 0; t < 2; ++t) {
      umma::mbar_init(smem_u32(&sh.s_full[t]), 1);
      umma::mbar_init(smem_u32(&sh.p_ready[t][0]), 4);
      umma::mbar_init(smem_u32(&sh.p_ready[t][1]), 4);
      umma::mbar_init(smem_u32(&sh.o_full[t]), 1);
    }
    for (int i = 0; i < 4; ++i) {
      umma::mbar_init(smem_u32(&sh.hand[i]), 1);
      umma::mbar_init(smem_u32(&sh.back[i]), 1);
    }
    for (int i = 0; i < kDescs; ++i) {
      umma::mbar_init(smem_u32(&sh.desc_full[i]), 1);
      umma::mbar_init(smem_u32(&sh.desc_empty[i]), 9);
    }
    for (int i = 0; i < 12; ++i) {
      umma::mbar_init(smem_u32(&sh.kv_full[i]), 1);
      umma::mbar_init(smem_u32(&sh.kv_empty[i]), 1);
    }
    umma::mbar_fence_init();
  }
  umma::fence_before_sync();
  fine = __syncthreads_and(fine);
  umma::fence_after_sync();
  const uint32_t tm = sh.tmem;

  const int per = (units + kPlan - 1) / kPlan, entries = (units + per - 1) / per;
  if (fine)
    for (int e = threadIdx.x; e < entries; e += kThreads) {
      int64_t c[2] = {0, 0};
      for (int u = e * per; u < min(units, (e + 1) * per); ++u) {
        const Unit x = load_unit<SHARED>(p, u);
        if (x.bad && cta == 0) flag(p.status, VT_DEV_BAD_LEN);
        c[x.narrow] += p.Hkv * cost_before(x, tpt, unit_items(x, tpt));
      }
      table0[e + 1] = c[0];
      table1[e + 1] = c[1];
    }
  __syncthreads();
  if (fine && warp < 2) {
    int64_t* line = warp ? table1 : table0;
    const int run = (entries + 31) / 32;
    int64_t sum = 0;
    for (int e = lane * run; e < min(entries, (lane + 1) * run); ++e) sum += line[e + 1];
    int64_t before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(kFull, before, o);
      if (lane >= o) before += y;
    }
    before -= sum;
    for (int e = lane * run; e < min(entries, (lane + 1) * run); ++e) {
      const int64_t c = line[e + 1];
      line[e + 1] = before + c;
      before += c;
    }
    if (lane == 0) line[0] = 0;
  }
  __syncthreads();
  if (!fine && cta == 0 && threadIdx.x == 0) flag(p.status, VT_DEV_BAD_START);
  const int64_t wide = fine ? table0[entries] : 0, thin = fine ? table1[entries] : 0;
  // this CTA's line, its number there and how many share it
  const int split = first_narrow(wide, thin, gridDim.x);
  const bool narrow = cta >= split;
  const int64_t* line = narrow ? table1 : table0;
  const int64_t total = narrow ? thin : wide;
  const int rank = narrow ? cta - split : cta;
  const int n_cta = share_count(total, narrow ? gridDim.x - split : split);

  if (SHARED && cta == 0) {  // where the units begin, for the joining kernel; -1: nothing was done
    if (fine) {
      for (int e = threadIdx.x; e < entries; e += kThreads) {
        int64_t c[2] = {table0[e], table1[e]};
        for (int u = e * per; u < min(units, (e + 1) * per); ++u) {
          const Unit x = load_unit<SHARED>(p, u);
          w.line[u] = c[x.narrow];
          c[x.narrow] += p.Hkv * cost_before(x, tpt, unit_items(x, tpt));
        }
      }
    }
    if (threadIdx.x == 0) {
      w.line[units] = fine ? wide : -1;
      w.line[units + 1] = thin;
    }
    __syncthreads();  // (before q overwrites the tables)
  }

  // shared memory of the two kinds
  const uint32_t q_smem = base;
  const uint32_t kv_smem = base + (narrow ? C::TILE : 2 * C::TILE + kSoftWarps * kStage);
  auto is_small = [&](int n_tok) { return narrow && n_tok * p.G <= kSmall; };
  const int stages = narrow ? C::STAGES_NARROW : C::STAGES;

  const bool work = total > 0 && rank < n_cta;
  if (warp >= kLoadWarp) {
  regs_less<kRegsOther>();
  if (warp == kLoadWarp) {
    // ---- loading -----------------------------------------------------------------------------
    if (lane == 0 && !SHARED) {
      w.head[2 * cta].valid = 0;
      w.head[2 * cta + 1].valid = 0;
    }
    int n_desc = 0, n_item = 0, n_tile = 0;
    int n_out = 0;        // items whose results are known to be out
    bool small_before = true;
    int st = 0;           // the ring's next stage and its phase
    uint32_t ph = 0, filled = 0;
    bool go = true;
    if (work) {
      const int64_t x0 = share_begin(total, n_cta, rank), x1 = share_begin(total, n_cta, rank + 1);
      int lo = 0, hi = entries - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (line[mid] <= x0) lo = mid; else hi = mid - 1;
      }
      int u = lo * per;
      int64_t pos = line[lo];
      Unit un = load_unit<SHARED>(p, u);
      int items = un.narrow == narrow ? unit_items(un, tpt) : 0;
      int64_t head_cost = cost_before(un, tpt, items);
      while (pos + p.Hkv * head_cost <= x0) {  // x0 < total, so this ends at a unit with items
        pos += p.Hkv * head_cost;
        un = load_unit<SHARED>(p, ++u);
        items = un.narrow == narrow ? unit_items(un, tpt) : 0;
        head_cost = cost_before(un, tpt, items);
      }
      int h = (int)((x0 - pos) / head_cost);
      pos += h * head_cost;
      int t = 0;
      {
        int a = 0, b = items - 1;
        while (a < b) {
          const int mid = (a + b + 1) >> 1;
          if (cost_before(un, tpt, mid) <= x0 - pos) a = mid; else b = mid - 1;
        }
        t = a;
        pos += cost_before(un, tpt, t);
      }
      umma::fence_async_smem();  // the table has been read
      while (go && pos < x1) {
        const int64_t cost = item_cost(un, tpt, t);
        const int keys = item_keys(un, tpt, t), wt = item_weight(un, tpt, t);
        const int tiles = (keys + kKeys - 1) / kKeys;
        const int j0 = cut_tile(x0 - pos, cost, wt, tiles), j1 = cut_tile(x1 - pos, cost, wt, tiles);
        if (j0 < j1 || (tiles == 0 && pos >= x0)) {
          // describe it
          const int di = n_desc % kDescs;
          go = wait(smem_u32(&sh.desc_empty[di]), ((n_desc / kDescs) & 1) ^ 1, abort_flag);
          if (!go) break;
          const int first = t * 2 * tpt, n_tok = min(un.n - first, 2 * tpt);
          const bool whole = j0 == 0 && j1 == tiles;
          const bool prefix = SHARED && u < p.n_groups;
          if (lane == 0) {
            Desc d;
            d.tok0 = un.tok0 + first;
            d.n_tok = n_tok;
            d.h = h;
            d.j0 = j0;
            d.j1 = j1;
            d.vis0 = un.vis0 + first * un.step;
            d.step = un.step;
            d.kv_len = un.kv_len;
            d.whole = whole;
            d.prefix = prefix;
            d.slot = SHARED ? cta : whole ? -1 : 2 * cta + (j0 == 0);
            sh.desc[di] = d;
            if (!SHARED && !whole) {
              Head hd{un.tok0 + first, n_tok, h, j0, j1, tiles, 1, 0};
              w.head[d.slot] = hd;
            }
            umma::mbar_arrive(smem_u32(&sh.desc_full[di]));
          }
          ++n_desc;
          // its tiles
          const int n_pages = (un.kv_len + kPage - 1) / kPage;
          const int last = un.kv_len - kPage * (n_pages - 1);  // tokens on the last page
          const int32_t* table = p.page_table + (int64_t)un.row * p.pt_stride + un.page0;
          auto page_id = [&](int j) {  // of lane's page among the four tiles from j
            const int i = j * kPagesTile + lane;
            return i < n_pages && j < j1 ? table[i] : -1;
          };
          int ids = 0, next = j0 < j1 ? page_id(j0) : 0;
          for (int j = j0; go && j < j1; ++j, ++n_tile) {
            if ((j - j0) % 4 == 0) {
              ids = next;
              next = page_id(j + 4);
            }
            const int mine = ((j - j0) & 3) * kPagesTile + (lane & 7);
            int id = __shfl_sync(kFull, ids, mine);
            const int i = j * kPagesTile + (lane & 7);
            const bool there = i < n_pages;
            const bool bad = there && (id < 0 || id >= p.kv.num_pages);
            const uint32_t bads = __ballot_sync(kFull, bad) & 0xffu;
            // tokens [0, 16), the last page's from a negative one; [16, 32): all zeros
            int c_tok = i == n_pages - 1 ? last - kPage : 0;
            if (!there || bad) {
              id = 0;
              c_tok = kPage;
            }
            if (lane == 0) {
              sh.bad[n_tile % kBadRing] = (int)bads;
              if (bads) flag(p.status, VT_DEV_BAD_PAGE);
            }
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
              const uint32_t full = smem_u32(&sh.kv_full[st]);
              go = go && wait(smem_u32(&sh.kv_empty[st]), ph ^ 1, abort_flag);
              if (!go) break;
              if (lane == 0) umma::mbar_expect_tx(full, C::TILE);
              __syncwarp();
              if (lane < kPagesTile * C::HALVES) {
                const int half = lane / kPagesTile;
                umma::tma_load_4d(kv_smem + st * C::TILE + half * C::BOX +
                                      (lane & 7) * (kPage * 128),
                                  kv ? &v_map : &k_map, half * 64, c_tok, h, id, full);
              }
              ++filled;
              if (++st == stages) {
                st = 0;
                ph ^= 1;
              }
              if (kv == 0 && j == j0) {
                // q goes behind the first K tile: its buffer is free only when the last item's
                // scores are done
                go = wait(smem_u32(&sh.q_empty), (n_item & 1) ^ 1, abort_flag);
                if (!go) break;
                const int tiles_q = n_tok > tpt ? 2 : 1;
                const bool small = is_small(n_tok);
                // results out: of the last item where the two meet in shared memory, else of the
                // one before, so that no phase of the two barriers is passed unseen
                const int outs = !narrow ? 0 : small && small_before ? n_item - 1 : n_item;
                for (; go && n_out < outs; ++n_out)
                  go = wait(smem_u32(&sh.out_done[n_out & 1]), n_out >> 1 & 1, abort_flag);
                if (!go) break;
                small_before = small;
                if (lane == 0) {
                  const uint32_t bar = smem_u32(&sh.q_full);
                  const int box = p.G * (small ? kSmall / p.G : tpt) * 128;
                  umma::mbar_expect_tx(bar, box * C::HALVES * tiles_q);
                  for (int tt = 0; tt < tiles_q; ++tt)
                    for (int half = 0; half < C::HALVES; ++half)
                      umma::tma_load_3d(q_smem + tt * C::TILE + half * (small ? C::Q_SMALL : C::BOX),
                                        small ? &q1_map : &q_map, half * 64, h * p.G,
                                        un.tok0 + first + tt * tpt, bar);
                }
                ++n_item;
              }
            }
          }
        }
        // the next item
        pos += cost;
        if (++t == items) {
          t = 0;
          if (++h == p.Hkv) {
            h = 0;
            do {
              if (++u == units) break;
              un = load_unit<SHARED>(p, u);
              items = un.narrow == narrow ? unit_items(un, tpt) : 0;
            } while (items == 0);
            if (u == units) break;
          }
        }
      }
    }
    if (go) {
      const int di = n_desc % kDescs;
      go = wait(smem_u32(&sh.desc_empty[di]), ((n_desc / kDescs) & 1) ^ 1, abort_flag);
      if (go && lane == 0) {
        sh.desc[di].n_tok = 0;
        umma::mbar_arrive(smem_u32(&sh.desc_full[di]));
      }
    }
    if (!go) {  // copies in flight must land before the shared memory goes away
      for (uint32_t i = 0; i < min(filled, (uint32_t)stages); ++i) {
        if (st-- == 0) {
          st = stages - 1;
          ph ^= 1;
        }
        const unsigned long long t0 = global_ns();
        while (!umma::mbar_try_wait(smem_u32(&sh.kv_full[st]), ph) && global_ns() - t0 < kWaitNs) {
        }
      }
      const unsigned long long t0 = global_ns();
      while (n_item > 0 && !umma::mbar_try_wait(smem_u32(&sh.q_full), (n_item - 1) & 1) &&
             global_ns() - t0 < kWaitNs) {
      }
    }
  } else if (warp == kMmaWarp) {
    // ---- products ----------------------------------------------------------------------------
    constexpr uint32_t kIdS = umma::idesc_bf16(kTile, kKeys, false, false);
    constexpr uint32_t kIdO = umma::idesc_bf16(kTile, D, false, true);
    int n_desc = 0, n_item = 0;
    int k_st = 0, v_st = 1;  // the ring's next K and V stage, and their phases
    uint32_t k_ph = 0, v_ph = 0, p_phase[2] = {0, 0};
    bool go = true;
    auto scores = [&](int t, int q_tile, uint32_t q_half, int st) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t at = (k % 4) * 32;
        umma::mma_bf16(
            tm + t * kKeys,
            umma::sdesc_sw128(q_smem + q_tile * C::TILE + (k / 4) * q_half + at, 0, 1024),
            umma::sdesc_sw128(kv_smem + st * C::TILE + (k / 4) * C::BOX + at, 0, 1024), kIdS,
            k > 0);
      }
      umma::commit(smem_u32(&sh.s_full[t]));
    };
    auto values = [&](int t, int st, int half, bool more) {
#pragma unroll
      for (int k = half * (kKeys / 32); k < (half + 1) * (kKeys / 32); ++k)
        umma::mma_bf16_ta(tm + 2 * kKeys + t * D, tm + t * kKeys + k * 8,
                          umma::sdesc_sw128(kv_smem + st * C::TILE + k * 2048, C::BOX, 1024), kIdO,
                          more || k > 0);
    };
    while (true) {
      const int di = n_desc % kDescs;
      go = wait(smem_u32(&sh.desc_full[di]), (n_desc / kDescs) & 1, abort_flag);
      if (!go) break;
      const int n_tok = sh.desc[di].n_tok, j0 = sh.desc[di].j0, j1 = sh.desc[di].j1;
      __syncwarp();
      if (lane == 0) umma::mbar_arrive(smem_u32(&sh.desc_empty[di]));
      ++n_desc;
      if (n_tok == 0) break;
      if (j0 == j1) continue;
      // Step k: the values of key tile k - lag, then the scores of key tile k.  Two row tiles take
      // every key tile one after the other.  One row tile alone would leave the tensor cores
      // idle while its softmax runs, so it takes key tiles in turn as two: even ones in S_0 and
      // O_0, odd ones in S_1 and O_1, each with its own maxima and sums, joined at the end.
      const bool two = n_tok > tpt;
      const int n = j1 - j0, lag = two ? 1 : 2;
      const uint32_t q_half = is_small(n_tok) ? C::Q_SMALL : C::BOX;
      go = wait(smem_u32(&sh.q_full), n_item & 1, abort_flag);
      for (int k = 0; go && k < n + lag; ++k) {
        const bool has_k = k < n, has_v = k >= lag && k - lag < n;
        if (has_k)
          go = wait(smem_u32(&sh.kv_full[k_st]), k_ph, abort_flag);
        if (go && has_v) go = wait(smem_u32(&sh.kv_full[v_st]), v_ph, abort_flag);
        const int t0 = two ? 0 : k & 1, t1 = two ? 1 : t0;
        for (int t = t0; go && t <= t1; ++t) {
          if (has_v) {
            go = wait(smem_u32(&sh.p_ready[t][0]), p_phase[t], abort_flag);
            if (!go) break;
            umma::fence_after_sync();
            values(t, v_st, 0, k >= 2 * lag);
            go = wait(smem_u32(&sh.p_ready[t][1]), p_phase[t], abort_flag);
            if (!go) break;
            umma::fence_after_sync();
            values(t, v_st, 1, true);
            p_phase[t] ^= 1;
            if (!has_k) umma::commit(smem_u32(&sh.o_full[t]));
          } else {
            umma::fence_after_sync();
          }
          if (has_k) scores(t, two ? t : 0, q_half, k_st);
        }
        if (!go) break;
        if (has_v) {
          umma::commit(smem_u32(&sh.kv_empty[v_st]));
          if ((v_st += 2) >= stages) {
            v_st = 1;
            v_ph ^= 1;
          }
        }
        if (has_k) {
          umma::commit(smem_u32(&sh.kv_empty[k_st]));
          if (k == n - 1) umma::commit(smem_u32(&sh.q_empty));
          if ((k_st += 2) >= stages) {
            k_st = 0;
            k_ph ^= 1;
          }
        }
      }
      if (!go) break;
      ++n_item;
    }
    if (!go) {  // let what was issued finish
      umma::commit(smem_u32(&sh.drain));
      const unsigned long long t0 = global_ns();
      while (!umma::mbar_try_wait(smem_u32(&sh.drain), 0) && global_ns() - t0 < kWaitNs) {
      }
    }
  }
  } else {
    regs_more<kRegsSoftmax>();
    // ---- softmax and results -----------------------------------------------------------------
    const int t = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t tm_row = tm + ((uint32_t)(warp & 3) << 21);  // this warp's lanes
    const uint32_t tm_s = tm_row + t * kKeys, tm_o = tm_row + 2 * kKeys + t * D;
    const float c = p.qscale, lazy = kLazy / c;
    const int Hq = p.Hkv * p.G;
    const int tok_row = row / p.G, head_row = row - tok_row * p.G;
    uint32_t s_phase = 0, o_phase = 0, hand_phase = 0;
    bool lent = false;  // O_1 is the first warpgroup's to read
    int n_tile = 0, n_item = 0;
    for (int n_desc = 0;; ++n_desc) {
      const int di = n_desc % kDescs;
      if (!wait(smem_u32(&sh.desc_full[di]), (n_desc / kDescs) & 1, abort_flag)) break;
      const Desc d = sh.desc[di];
      __syncwarp();
      if (lane == 0) umma::mbar_arrive(smem_u32(&sh.desc_empty[di]));
      if (d.n_tok == 0) break;
      const bool two = d.n_tok > tpt;
      const int rt = two ? t : 0;  // row tile
      const int n_tok = min(tpt, d.n_tok - rt * tpt);
      const bool active = (warp & 3) * 32 < n_tok * p.G, mine = row < n_tok * p.G;
      const int tok = rt * tpt + min(tok_row, n_tok - 1);
      const int vis = d.vis0 + tok * d.step;
      const int vis_warp = d.vis0 + (rt * tpt + min((warp & 3) * 32 / p.G, n_tok - 1)) * d.step;
      const int n_pages = (d.kv_len + kPage - 1) / kPage;
      const int gap = n_pages * kPage - d.kv_len;   // zero rows ahead of the last page's tokens
      float m = -INFINITY, l = 0.0f;
      bool ok = true;
      const int begin = two ? d.j0 : d.j0 + t, stride = two ? 1 : 2;
      for (int j = begin; j < d.j1; j += stride) {
        ok = wait(smem_u32(&sh.s_full[t]), s_phase, abort_flag);
        if (!ok) break;
        s_phase ^= 1;
        if (active) {
          umma::fence_after_sync();
          const uint32_t bad = (uint32_t)*(volatile int*)&sh.bad[(n_tile + j - d.j0) % kBadRing];
          const int slot0 = j * kKeys;
          const bool masked = slot0 + kKeys > vis_warp || bad;
          if (masked) {  // what a row may not see becomes -inf in place
            RowMask rm;
            const int last0 = (n_pages - 1) * kPage;  // the last page's first slot
            rm.lim = (vis > last0 ? vis + gap : vis) - slot0;
            rm.hole0 = last0 - slot0;
            rm.hole1 = rm.hole0 + gap;
            rm.bad = bad;
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              uint32_t s[32];
              umma::tmem_ld32_async(tm_s + 32 * i, s);
              const uint32_t ms = rm.word(i);
              umma::tmem_wait_ld();
              umma::tmem_landed(s);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(ms >> e & 1u)) s[e] = __float_as_uint(-INFINITY);
              umma::tmem_st32_async(tm_s + 32 * i, s);
            }
            umma::tmem_wait_st();
          }
          // The scores are read twice, for the maximum and for the weights: a row of 128 does not
          // stay in registers without spills, and a second read costs 32 cycles per 32 columns.
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          {
            uint32_t s[4][32];
#pragma unroll
            for (int i = 0; i < 4; ++i) umma::tmem_ld32_async(tm_s + 32 * i, s[i]);
            umma::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 4; ++i) umma::tmem_landed(s[i]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int e = 0; e < 32; e += 8)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mx[k] = fmaxf(mx[k], fmaxf(__uint_as_float(s[i][e + k]),
                                             __uint_as_float(s[i][e + 4 + k])));
          }
          uint32_t s[2][32];
          umma::tmem_ld32_async(tm_s, s[0]);
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          if (__any_sync(kFull, mine && (top > m + lazy || (m == -INFINITY && top > m)))) {
            const float mn = fmaxf(m, top);
            const float f = m == -INFINITY ? 0.0f : ex2((m - mn) * c);
            m = mn;
            l *= f;
            if (j > begin) {
#pragma unroll 1
              for (int i = 0; i < D / 16; ++i) {
                uint32_t o[16];
                umma::tmem_ld16(tm_o + 16 * i, o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                umma::tmem_st16_async(tm_o + 16 * i, o);
              }
            }
          }
          const float mc = m == -INFINITY ? 0.0f : m * c;
          const uint64_t c2 = pair(c, c), mc2 = pair(-mc, -mc);
          uint64_t sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            umma::tmem_wait_ld();
            umma::tmem_landed(s[i & 1]);
            if (i < 3) umma::tmem_ld32_async(tm_s + 32 * (i + 1), s[(i + 1) & 1]);
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              uint64_t x = fma2(pair(__uint_as_float(s[i & 1][2 * e]),
                                     __uint_as_float(s[i & 1][2 * e + 1])),
                                c2, mc2);
              x = exp2_unit(x);
              sum[e & 1] = add2(sum[e & 1], x);
              pk[e] = pack2(x);
            }
            umma::tmem_st16_async(tm_s + 16 * i, pk);  // (over scores that were read)
            if (i & 1) {  // half of the keys: the product with their values can start
              if (lent) {
                wait(smem_u32(&sh.back[warp & 3]), hand_phase, abort_flag);
                hand_phase ^= 1;
                lent = false;
              }
              umma::tmem_wait_st();
              umma::fence_before_sync();
              __syncwarp();
              if (lane == 0) umma::mbar_arrive(smem_u32(&sh.p_ready[t][i >> 1]));
            }
          }
          l += total2(sum[0], sum[1]);
        } else {
          if (lent) {
            wait(smem_u32(&sh.back[warp & 3]), hand_phase, abort_flag);
            hand_phase ^= 1;
            lent = false;
          }
          if (lane == 0) {
            umma::mbar_arrive(smem_u32(&sh.p_ready[t][0]));
            umma::mbar_arrive(smem_u32(&sh.p_ready[t][1]));
          }
        }
      }
      if (!ok) break;
      n_tile += d.j1 - d.j0;
      n_item += d.j0 < d.j1;
      if (begin < d.j1) {
        if (!wait(smem_u32(&sh.o_full[t]), o_phase, abort_flag)) break;
        o_phase ^= 1;
        umma::fence_after_sync();
      }
      // One row tile: the second warpgroup leaves its rows to the first, and its next weights wait
      // until the first has read O_1.
      const bool odd = !two && d.j1 - d.j0 > 1;  // there are rows in O_1
      if (!two && t == 1) {
        if (odd) {
          sh.ml[row] = make_float2(m, l);
          umma::fence_before_sync();
          __syncwarp();
          if (lane == 0) umma::mbar_arrive(smem_u32(&sh.hand[warp & 3]));
          lent = true;
        }
        continue;
      }
      float f0 = 1.0f, f1 = 0.0f;
      if (odd) {
        if (!wait(smem_u32(&sh.hand[warp & 3]), hand_phase, abort_flag)) break;
        hand_phase ^= 1;
        umma::fence_after_sync();
        const float2 other = sh.ml[row];  // (the wait above keeps the compiler from moving this)
        const float mn = fmaxf(m, other.x);
        f0 = m == -INFINITY ? 0.0f : ex2((m - mn) * c);
        f1 = other.x == -INFINITY ? 0.0f : ex2((other.x - mn) * c);
        m = mn;
        l = l * f0 + other.y * f1;
      }
      if (!active) {
        __syncwarp();
        if (odd && lane == 0) umma::mbar_arrive(smem_u32(&sh.back[warp & 3]));
        if (narrow && d.j0 < d.j1 && lane == 0)
          umma::mbar_arrive(smem_u32(&sh.out_done[(n_item - 1) & 1]));
        continue;
      }
      // Results leave through shared memory, 128 bytes of each row at a time (16-byte piece c of
      // row r at c ^ (r % 8)), so that a store covers whole lines: straight from a thread's own
      // row it would touch 32 of them.
      const bool whole = !SHARED && d.whole;
      const int64_t orow = (int64_t)(d.tok0 + tok) * Hq + d.h * p.G + head_row;
      const float mc = m == -INFINITY ? -INFINITY : m * c;
      const float inv = l > 0.0f ? 1.0f / l : 0.0f;
      const int rows = min(32, n_tok * p.G - (warp & 3) * 32);  // of this warp, the valid ones
      // each lane's eight rows r0, r0 + 4, .. in the stores: byte offsets from the result's base
      const int r0 = lane >> 3, piece = lane & 7;
      unsigned char* base_out =
          whole ? reinterpret_cast<unsigned char*>(p.out)
                : reinterpret_cast<unsigned char*>(
                      SHARED && d.j0 == 0
                          ? w.first + (d.prefix ? 0 : (int64_t)p.B * Hq) * kRowF<D>
                          : w.part + ((int64_t)d.slot * 2 * kTile + t * kTile) * kRowF<D>);
      const int64_t row_at = whole ? orow * D * 2
                             : (SHARED && d.j0 == 0 ? orow : (int64_t)row) * kRowF<D> * 4;
      const uint32_t stage = (!narrow                ? base + 2 * C::TILE
                              : is_small(d.n_tok) ? q_smem + C::HALVES * C::Q_SMALL
                                                  : q_smem) +
                             warp * kStage;
      const int passes = whole ? D / 64 : D / 32;
      // 32 dims of the row from dim `at`, joined where there are two parts
      auto result = [&](int at, uint32_t (&o)[2][16]) {
        if (d.j0 < d.j1) {
          umma::tmem_ld16_async(tm_o + at, o[0]);
          umma::tmem_ld16_async(tm_o + at + 16, o[1]);
          umma::tmem_wait_ld();
          umma::tmem_landed(o[0]);
          umma::tmem_landed(o[1]);
          if (odd) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t x[16];
              umma::tmem_ld16_async(tm_o + D + at + 16 * i, x);
              umma::tmem_wait_ld();
              umma::tmem_landed(x);
#pragma unroll
              for (int e = 0; e < 16; ++e)
                o[i][e] = __float_as_uint(
                    fmaf(__uint_as_float(o[i][e]), f0, __uint_as_float(x[e]) * f1));
            }
          }
        }
        if (!(l > 0.0f)) {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e >> 4][e & 15] = 0u;
        }
      };
#pragma unroll 1
      for (int i = 0; i < passes; ++i) {
        uint32_t o[2][16];
        if (whole) {
#pragma unroll 1
          for (int part = 0; part < 2; ++part) {
            result(64 * i + 32 * part, o);
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
              uint32_t v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                v[e] = pack2(__uint_as_float(o[q4 >> 1][8 * (q4 & 1) + 2 * e]) * inv,
                             __uint_as_float(o[q4 >> 1][8 * (q4 & 1) + 2 * e + 1]) * inv);
              st_shared16(stage + lane * 128 + (((4 * part + q4) ^ (lane & 7)) << 4), v[0], v[1],
                          v[2], v[3]);
            }
          }
        } else {
          result(32 * i, o);
#pragma unroll
          for (int q8 = 0; q8 < 8; ++q8)
            st_shared16(stage + lane * 128 + ((q8 ^ (lane & 7)) << 4),
                        o[q8 >> 2][4 * (q8 & 3)], o[q8 >> 2][4 * (q8 & 3) + 1],
                        o[q8 >> 2][4 * (q8 & 3) + 2], o[q8 >> 2][4 * (q8 & 3) + 3]);
        }
        if (odd && i == passes - 1) {  // O_1 has been read
          umma::fence_before_sync();
          __syncwarp();
          if (lane == 0) umma::mbar_arrive(smem_u32(&sh.back[warp & 3]));
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = r0 + 4 * k;
          const int64_t at = __shfl_sync(kFull, row_at, r);
          const uint4 v = ld_shared16(stage + r * 128 + ((piece ^ (r & 7)) << 4));
          if (r < rows) *reinterpret_cast<uint4*>(base_out + at + 128 * i + 16 * piece) = v;
        }
        __syncwarp();
      }
      if (lane < rows) {
        if (!whole)
          *reinterpret_cast<float2*>(base_out + row_at + D * 4) = make_float2(mc, l);
        else if (p.lse)
          p.lse[orow] = l > 0.0f ? mc * kLn2 + logf(l) : -INFINITY;
      }
      if (narrow && d.j0 < d.j1) {  // (the copy of the next Q is another proxy's write)
        umma::fence_async_smem();
        __syncwarp();
        if (lane == 0) umma::mbar_arrive(smem_u32(&sh.out_done[(n_item - 1) & 1]));
      }
    }
  }
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  if (sh.abort && threadIdx.x == 0) flag(p.status, VT_DEV_TIMEOUT);
  if (warp == kMmaWarp) umma::tmem_dealloc(tm, 512);
}

// ---- joining partial rows -------------------------------------------------------------------

// A warp's running join of partial rows of D floats (lane: D/32 of them).
template <int D>
struct Join {
  static constexpr int E = D / 32;
  float o[E], m = -INFINITY, l = 0.0f;
  __device__ __forceinline__ Join() {
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;
  }
  __device__ __forceinline__ void add(const float* r, int lane) {
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(r + D));
    float x[E];
    if (E == 4) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(r) + lane);
      x[0] = v.x; x[1] = v.y; x[E - 2] = v.z; x[E - 1] = v.w;
    } else {
      const float2 v = __ldcg(reinterpret_cast<const float2*>(r) + lane);
      x[0] = v.x; x[1] = v.y;
    }
    float M, fa, fb;
    merge_scale(m, ml.x, M, fa, fb);
    m = M;
    l = l * fa + ml.y * fb;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * fa + x[e] * fb;
  }
  __device__ __forceinline__ void write(__nv_bfloat16* out, float* lse, int64_t row, int lane) {
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    uint32_t* dst = reinterpret_cast<uint32_t*>(out + row * D) + lane * (E / 2);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) dst[e] = pack2(o[2 * e] * inv, o[2 * e + 1] * inv);
    if (lse && lane == 0) lse[row] = l > 0.0f ? m * kLn2 + logf(l) : -INFINITY;
  }
};

constexpr int kJoinThreads = 256;
constexpr int kJoinRows = kJoinThreads / 32;

// Prompts: block (c, y) joins rows y * 8 .. of the item that begins in CTA c and ends in another.
template <int D>
__global__ void __launch_bounds__(kJoinThreads)
    join_items_kernel(const AttendParams p, const Work w) {
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Head h0 = w.head[2 * c + 1];
  if (!h0.valid) return;
  const int tpt = kTile / p.G, Hq = p.Hkv * p.G;
  const int r = blockIdx.y * kJoinRows + warp;  // row of the item
  const int tile = r / kTile, in = r - tile * kTile;
  const int tok = tile * tpt + in / p.G;
  if (in >= tpt * p.G || tok >= h0.n_tok) return;
  Join<D> a;
  a.add(w.part + ((int64_t)(2 * c + 1) * 2 * kTile + r) * kRowF<D>, lane);
  int done = h0.j1;
  for (int k = c + 1; done < h0.n_tiles && k < (int)gridDim.x; ++k) {
    const Head hk = w.head[2 * k];
    if (!hk.valid) continue;  // its share lay within a key tile of another's
    a.add(w.part + ((int64_t)2 * k * 2 * kTile + r) * kRowF<D>, lane);
    done = hk.j1;
  }
  a.write(p.out, p.lse, (int64_t)(h0.tok0 + tok) * Hq + h0.h * p.G + in % p.G, lane);
}

// Shared prefixes: a warp joins one row: the pieces of its group's prefix, and of its own pages.
template <int D>
__global__ void __launch_bounds__(kJoinThreads)
    join_rows_kernel(const AttendParams p, const Work w, int ctas) {
  const int units = p.n_groups + p.B;
  const int64_t wide = w.line[units], thin = w.line[units + 1];
  if (wide < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hq = p.Hkv * p.G, tpt = kTile / p.G;
  const int64_t orow = (int64_t)blockIdx.x * kJoinRows + warp;
  if (orow >= (int64_t)p.B * Hq) return;
  const int b = (int)(orow / Hq), hq = (int)(orow - (int64_t)b * Hq);
  const int h = hq / p.G;
  const int g = group_of(p, b);
  if (g < 0) return;
  const Unit own = load_unit<true>(p, p.n_groups + b);
  Join<D> a;
  const int split = first_narrow(wide, thin, ctas);
#pragma unroll 1
  for (int part = 0; part < 2 && !own.bad; ++part) {
    const int u = part ? p.n_groups + b : g;
    const Unit un = part ? own : load_unit<true>(p, g);
    if (un.n == 0) continue;
    const int64_t total = un.narrow ? thin : wide;
    const int cta0 = un.narrow ? split : 0;
    const int n_cta = share_count(total, un.narrow ? ctas - split : split);
    const int t = (b - un.tok0) / (2 * tpt), i = (b - un.tok0) - t * 2 * tpt;
    const int r = i / tpt * kTile + i % tpt * p.G + (hq - h * p.G);  // the row within the item
    const int64_t cost = item_cost(un, tpt, t);
    const int64_t pos = w.line[u] + h * cost_before(un, tpt, unit_items(un, tpt)) +
                        cost_before(un, tpt, t);
    const int wt = item_weight(un, tpt, t);
    const int tiles = (item_keys(un, tpt, t) + kKeys - 1) / kKeys;
    if (tiles == 0) continue;
    for (int c = share_of(total, n_cta, pos); c < n_cta; ++c) {
      const int64_t x0 = share_begin(total, n_cta, c), x1 = share_begin(total, n_cta, c + 1);
      if (x0 >= pos + cost) break;
      const int j0 = cut_tile(x0 - pos, cost, wt, tiles), j1 = cut_tile(x1 - pos, cost, wt, tiles);
      if (j0 >= j1) continue;
      a.add(j0 == 0 ? w.first + ((part ? (int64_t)p.B * Hq : 0) + orow) * kRowF<D>
                    : w.part + ((int64_t)(cta0 + c) * 2 * kTile + r) * kRowF<D>,
            lane);
    }
  }
  a.write(p.out, p.lse, orow, lane);
}

// ---- host -----------------------------------------------------------------------------------

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Fills w from ws (NULL: only the size is wanted) and returns the bytes.
size_t lay_out(const AttendParams& p, int ctas, void* ws, Work* w) {
  const bool shared = p.prefix_pages != nullptr;
  const size_t row = (size_t)(p.D + 4) * 4;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* r = ws ? static_cast<char*>(ws) + at : nullptr;
    at += up256(bytes);
    return r;
  };
  Work x{};
  x.head = reinterpret_cast<Head*>(take(shared ? 0 : 2 * sizeof(Head) * ctas));
  x.part = reinterpret_cast<float*>(take((size_t)(shared ? 1 : 2) * ctas * 2 * kTile * row));
  x.first = reinterpret_cast<float*>(take(shared ? 2 * (size_t)p.B * p.Hkv * p.G * row : 0));
  x.line = reinterpret_cast<int64_t*>(take(shared ? ((size_t)p.n_groups + p.B + 2) * 8 : 0));
  if (w) *w = x;
  return at;
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// A bf16 tensor of `rank` dimensions (innermost 64-element boxes, 128-byte swizzle); strides in
// elements, for dimensions 1 ..; what has one entry may have any stride.
bool encode(CUtensorMap* m, const void* base, int rank, const int64_t* dims, const int64_t* strides,
            const int* box) {
  cuuint64_t d[4], st[3];
  cuuint32_t bx[4], one[4] = {1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = (cuuint64_t)dims[i];
    bx[i] = (cuuint32_t)box[i];
    if (i) st[i - 1] = dims[i] > 1 ? (cuuint64_t)strides[i - 1] * 2 : 16;
  }
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), d, st, bx,
                     one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool SHARED>
cudaError_t launch(const AttendParams& p, const Work& w, int ctas, cudaStream_t s) {
  const int tpt = kTile / p.G;
  CUtensorMap q, q1, k, v;
  const int64_t qd[3] = {D, (int64_t)p.Hkv * p.G, p.T}, qs[2] = {D, p.sq_t};
  const int qb[3] = {64, p.G, tpt}, qb1[3] = {64, p.G, kSmall / p.G};
  const int64_t kd[4] = {D, kPage, p.Hkv, p.kv.num_pages};
  const int64_t ks[3] = {p.kv.sk_t, p.kv.sk_h, p.kv.sk_p}, vs[3] = {p.kv.sv_t, p.kv.sv_h, p.kv.sv_p};
  const int kb[4] = {64, kPage, 1, 1};
  if (!encode_fn() || !encode(&q, p.q, 3, qd, qs, qb) || !encode(&q1, p.q, 3, qd, qs, qb1) ||
      !encode(&k, p.kv.k_pool, 4, kd, ks, kb) || !encode(&v, p.kv.v_pool, 4, kd, vs, kb))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(attend_kernel<D, SHARED>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  attend_kernel<D, SHARED><<<ctas, kThreads, Cfg<D>::SMEM, s>>>(p, w, q, q1, k, v);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (SHARED) {
    const int64_t rows = (int64_t)p.B * p.Hkv * p.G;
    join_rows_kernel<D><<<(unsigned)((rows + kJoinRows - 1) / kJoinRows), kJoinThreads, 0, s>>>(
        p, w, ctas);
  } else {
    join_items_kernel<D><<<dim3(ctas, 2 * kTile / kJoinRows), kJoinThreads, 0, s>>>(p, w);
  }
  return cudaGetLastError();
}

}  // namespace

size_t attend_workspace_bytes(const AttendParams& p, int sm_count) {
  return lay_out(p, sm_count, nullptr, nullptr);
}

cudaError_t launch_attend(const AttendParams& p, void* ws, int sm_count, cudaStream_t s) {
  Work w;
  lay_out(p, sm_count, ws, &w);
  const bool shared = p.prefix_pages != nullptr;
  if (p.D == 128)
    return shared ? launch<128, true>(p, w, sm_count, s) : launch<128, false>(p, w, sm_count, s);
  return shared ? launch<64, true>(p, w, sm_count, s) : launch<64, false>(p, w, sm_count, s);
}

}  // namespace vt
