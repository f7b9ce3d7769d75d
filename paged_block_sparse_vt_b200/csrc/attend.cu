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
//   p_j = 2^(c S_t[r, j] - ref), l = l + sum_j p_j      with c = scale log2 e
//   P_t = bf16(p)                (over the columns of S_t)
//   O_t = O_t + P_t V            (tcgen05, P_t read from tensor memory)
// The weights are rounded to bf16 because the tensor core wants P in V's type (one 16-bit kind for
// both operands; the 32-bit kind has half the rate and would need V widened on the way): half a
// step, 2^-8, of each weight at most, which brings the results' rms error from the output's own
// rounding, 0.0016-0.0017 of their size, to 0.0017-0.0022.  l sums the weights as they were before.
// A warpgroup has one tile, a thread one row, so no sum crosses lanes.  The reference need not be
// the largest score: out = O / l does not depend on it, and a weight of 2^50 keeps as many bits in
// bf16 and fp32 as one of 1.  So a step takes no maximum.  Its reference is that of the first
// tile's maximum, and where a tile's weights sum to 2^kLift or more, the next step first raises
// the reference by that sum's exponent and scales O_t and l.  Only a half whose weights sum to
// kFar or more is done again, with its maximum; and so is, from the start, a tile of which some
// keys are hidden.  The weights of a half of the keys are handed over as they are done, so that
// their product runs beside the other half's exponentials.
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
//
// What bounds it: a step of two row tiles takes ~3200 cycles, its products and its exponentials
// 2048 each; the rest is the chain scores - exponentials - values of a tile, and tensor memory has
// room for two tiles (512 columns: S and O of 128 each).  A prompt of 8192 tokens (32/8 heads of
// 128 dims) runs at 1160 TFLOP/s, its products alone at 1450.  Code size counts: the rare paths are
// loops that are not unrolled, which took a packed batch from 350 to 330 us.
#include <cuda.h>

#include <algorithm>

#include "attend_params.cuh"
#include "attend_plan.cuh"
#include "common.cuh"
#include "gqa_attend.cuh"
#include "umma.cuh"

namespace vt {

namespace {

// two softmax warpgroups, and one with the loading and the product warp
constexpr int kThreads = 384;
// Registers: a softmax thread holds 64 scores of its row (32 in flight behind 32 in use) and 32
// pairs of weights beside the rest; what the third warpgroup gives up goes to the other two
// (2 * 200 + 104 = 3 * 168, the launch's share).
constexpr int kRegsSoftmax = 200, kRegsOther = 104;
constexpr int kLoadWarp = 8, kMmaWarp = 9;
constexpr int kDescs = 4;       // items described ahead
constexpr int kBadRing = 16;    // key tiles whose page checks are kept (> tiles in flight)
constexpr int kPlan = 1024;     // entries of the cost table in shared memory
constexpr float kLazy = 8.0f;     // bits by which a known maximum may pass the reference
constexpr int kLift = 12;         // bits of a tile's sum from which on the reference moves
constexpr float kFar = 0x1p40f;   // a sum of weights that is not used any more (O has room for
                                  // values of 2^80 then)
constexpr int kPagesTile = kKeys / kPage;
constexpr int kSoftWarps = 8;
constexpr int kStage = 32 * 128;  // a softmax warp's staging: 128 bytes of each of its rows

template <int D>
struct Cfg {
  static constexpr int HALVES = D / 64;              // 64-dim boxes of a row
  static constexpr int BOX = kKeys * 128;            // bytes of one half of a tile
  static constexpr int TILE = HALVES * BOX;          // bytes of a Q, K or V tile
  static constexpr int STAGES = D == 128 ? 4 : 8;
  static constexpr int TILES_SMEM = 2 * TILE + STAGES * TILE + kSoftWarps * kStage;
  // a CTA of the second line: each warp's two pages in flight
  static constexpr int OWN_SMEM = kWarps * 2 * PageTile<D>::SLOT;
  static constexpr int SMEM = 1024 + (TILES_SMEM > OWN_SMEM ? TILES_SMEM : OWN_SMEM);
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
  float* own;          // shared prefixes: [ctas kWarps][8][D + 4], rows that a share continues
  int64_t* line;       // shared prefixes: [units] where each unit begins in its line
  Line* lines;         // shared prefixes: the two lines; lines[0].total -1: nothing was done
};

// A partial row: O, then m (scaled, base 2) and l; padded to 16 bytes.
template <int D>
constexpr int kRowF = D + 4;

struct Shared {
  Desc desc[kDescs];
  int bad[kBadRing];
  uint64_t q_full, q_empty, s_full[2], p_ready[2][2], a_done[2], o_full[2], desc_full[kDescs],
      desc_empty[kDescs], kv_full[8], kv_empty[8], drain;
  int64_t total[2];  // the lines' lengths (the tables themselves give way to q)
  uint32_t tmem;
  int abort;
};

// ---- the units ------------------------------------------------------------------------------

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
  if (pages < 0 || pages > p.max_pages) return -1;
  return p.start[g + 1] - p.start[g] >= 2 ? pages : 0;
}

template <bool SHARED>
__device__ Unit load_unit(const AttendParams& p, int u) {
  Unit x{};
  if (!SHARED) {
    const int len = p.seq_lens[u];
    x.tok0 = p.start[u];
    x.n = p.start[u + 1] - x.tok0;
    x.row = u;
    if (x.n == 0) return x;  // whatever its length
    x.bad = len < x.n || len > p.max_pages * kPage;
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
    x.bad = pages < 0 || len < 1 || len > p.max_pages * kPage ||
            len < p.prefix_pages[g] * kPage;
    x.page0 = max(pages, 0);
    x.kv_len = x.vis0 = x.bad ? 0 : len - x.page0 * kPage;
  }
  return x;
}

// ---- bounded waits --------------------------------------------------------------------------

// Whole warp, and one answer for all of it: what follows are shuffles, votes and tensor-memory
// instructions of the whole warp, so no lane may go on where another gives up.  Lanes that polled
// each for itself could part: one sees the phase complete, another the flag that a third set.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t phase, volatile int* abort_flag) {
  for (int i = 0; i < 64; ++i)
    if (__all_sync(kFull, umma::mbar_try_wait(bar, phase))) return true;
  const unsigned long long t0 = global_ns();
  while (!__all_sync(kFull, umma::mbar_try_wait(bar, phase))) {
    if (__any_sync(kFull, *abort_flag != 0 || global_ns() - t0 > kWaitNs)) {
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

// ---- a decode row's own pages ---------------------------------------------------------------

// Where a warp is in the second line: the item (request b, KV head h), its place and its pages.
struct OwnCursor {
  int b, h, pages;
  int64_t pos, cost;
  Unit un;

  __device__ __forceinline__ void take(const AttendParams& p, int b_) {
    b = b_;
    un = load_unit<true>(p, p.n_groups + b);
    pages = own_pages(un);
    cost = own_cost(un);
  }
  // The item that position x0 (below the line's end) is in.
  __device__ void seek(const AttendParams& p, const int64_t* table, int entries, int per,
                       int64_t x0) {
    int lo = 0, hi = entries - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (table[mid] <= x0) lo = mid; else hi = mid - 1;
    }
    pos = table[lo];
    take(p, max(0, lo * per - p.n_groups));
    while (pos + p.Hkv * cost <= x0) {
      pos += p.Hkv * cost;
      take(p, b + 1);
    }
    h = (int)((x0 - pos) / cost);
    pos += h * cost;
  }
  __device__ __forceinline__ void next(const AttendParams& p) {
    pos += cost;
    if (++h < p.Hkv) return;
    h = 0;
    do {
      if (b + 1 == p.B) {
        pos = INT64_MAX;  // behind every share
        return;
      }
      take(p, b + 1);
    } while (cost == 0);
  }
};

// One warp's share [x0, x1) of the second line: the pages one after the other, two of them in
// flight in its two slots of shared memory, across items too.  64 requests of 4096 tokens (128
// dims) are read at 5.6 TB/s (193 us) of the 6.5 a copy reaches.  Memory is not what bounds it: 200
// KB in flight per SM are more than it needs, and a warp waits for it in 28% of its time only.  It
// is each warp's own chain per page - products, softmax, products, refill of the slot just used -
// of which three warps on a scheduler issue in 47% of the cycles (ncu).  (Decode rows as tcgen05
// items, with six 32 KB stages in flight: the same rate for long rows, and ~9000 cycles for one of
// two key tiles, three times what the warps take.)
template <int D>
__device__ __forceinline__ void own_share(const AttendParams& p, const Work& w, OwnCursor cur,
                                          int64_t x0, int64_t x1, uint32_t smem, int ws, int lane) {
  using T = PageTile<D>;
  const int Hq = p.Hkv * p.G;
  const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(p.kv.k_pool);
  const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(p.kv.v_pool);
  struct Slot {
    int vr;  // valid tokens, -1: nothing staged
    bool first, last;
    const __nv_bfloat16* q;
    float* dst;
  };
  int i = 0, i0 = 0, i1 = 0, ids = -1, ids_next = -1;
  const int32_t* table = nullptr;
  float* dst = nullptr;
  auto id_at = [&](int k) { return k + lane < i1 ? table[k + lane] : -1; };
  auto find = [&]() {  // the next item with pages in this share
    while (cur.pos < x1) {
      i = i0 = own_cut(x0 - cur.pos, cur.pages);
      i1 = own_cut(x1 - cur.pos, cur.pages);
      if (i < i1) {
        table = p.page_table + (int64_t)cur.un.row * p.pt_stride + cur.un.page0;
        dst = i == 0 ? w.first + ((int64_t)p.B * Hq + (int64_t)cur.b * Hq + cur.h * p.G) * kRowF<D>
                     : w.own + (int64_t)ws * 8 * kRowF<D>;
        ids_next = id_at(i);
        return true;
      }
      cur.next(p);
    }
    return false;
  };
  bool more = find();
  auto stage = [&](Slot& s, uint32_t slot) {
    s.vr = -1;
    if (more) {
      if (((i - i0) & 31) == 0) {
        ids = ids_next;
        ids_next = id_at(i + 32);
      }
      const int id = __shfl_sync(kFull, ids, (i - i0) & 31);
      s.vr = min(kPage, cur.un.kv_len - kPage * i);
      s.first = i == i0;
      s.last = i + 1 == i1;
      s.q = p.q + cur.b * p.sq_t + (int64_t)cur.h * p.G * D;
      s.dst = dst;
      int page = id;
      if (id < 0 || id >= p.kv.num_pages) {
        if (lane == 0) flag(p.status, VT_DEV_BAD_PAGE);
        s.vr = page = 0;
      }
      stage_page<D>(slot, kp + page * p.kv.sk_p + cur.h * p.kv.sk_h,
                    vp + page * p.kv.sv_p + cur.h * p.kv.sv_h, p.kv.sk_t, p.kv.sv_t, s.vr, p.q,
                    lane);
      if (++i == i1) {
        cur.next(p);
        more = find();
      }
    }
    cp_async_commit();
  };
  WarpAttention<D, 8> wa;
  auto attend = [&](const Slot& s, uint32_t slot) {
    cp_async_wait<1>();
    __syncwarp();
    if (s.first) wa.init(s.q, lane, p.G);
    wa.template page<false>(slot, s.vr, p.qscale);
    if (s.last) {
      float l = wa.lrun;
      l += __shfl_xor_sync(kFull, l, 1);
      l += __shfl_xor_sync(kFull, l, 2);
      if (wa.g < p.G) {
        float* r = s.dst + wa.g * kRowF<D>;
#pragma unroll
        for (int t = 0; t < T::NT; ++t)
          *reinterpret_cast<float2*>(r + t * 8 + wa.qd) = make_float2(wa.o[t][0], wa.o[t][1]);
        if ((lane & 3) == 0) *reinterpret_cast<float2*>(r + D) = make_float2(wa.mrun, l);
      }
    }
    __syncwarp();
  };
  Slot s0, s1;
  stage(s0, smem);
  stage(s1, smem + T::SLOT);
  while (s0.vr >= 0) {
    attend(s0, smem);
    stage(s0, smem);
    if (s1.vr < 0) break;
    attend(s1, smem + T::SLOT);
    stage(s1, smem + T::SLOT);
  }
  cp_async_wait_all();
}

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
                  const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map) {
  using C = Cfg<D>;
  extern __shared__ unsigned char raw[];
  __shared__ Shared sh;
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t q_smem = base, kv_smem = base + 2 * C::TILE;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tpt = kTile / p.G;
  const int cta = blockIdx.x;
  volatile int* abort_flag = &sh.abort;
  let_next_launch();
  // the cost tables of both lines lie where q comes later
  int64_t* table0 = reinterpret_cast<int64_t*>(raw + (base - smem_u32(raw)));
  int64_t* table1 = table0 + kPlan + 1;

  // The starts, then the cost of every unit, summed up over entries of `per` units each.
  const int units = SHARED ? p.n_groups + p.B : p.B, tile_units = SHARED ? p.n_groups : p.B;
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
    umma::mbar_init(smem_u32(&sh.drain), 1);
    for (int t = 0; t < 2; ++t) {
      umma::mbar_init(smem_u32(&sh.s_full[t]), 1);
      umma::mbar_init(smem_u32(&sh.p_ready[t][0]), 4);
      umma::mbar_init(smem_u32(&sh.p_ready[t][1]), 4);
      umma::mbar_init(smem_u32(&sh.a_done[t]), 1);
      umma::mbar_init(smem_u32(&sh.o_full[t]), 1);
    }
    for (int i = 0; i < kDescs; ++i) {
      umma::mbar_init(smem_u32(&sh.desc_full[i]), 1);
      umma::mbar_init(smem_u32(&sh.desc_empty[i]), 9);
    }
    for (int i = 0; i < C::STAGES; ++i) {
      umma::mbar_init(smem_u32(&sh.kv_full[i]), 1);
      umma::mbar_init(smem_u32(&sh.kv_empty[i]), 1);
    }
    umma::mbar_fence_init();
  }
  // (costs are worked out before it is known that the starts are in order: no index depends on
  // them but `row` and `tok0`, which are not used here)
  const int per = (units + kPlan - 1) / kPlan, entries = (units + per - 1) / per;
  uint32_t bad_len = 0;
  for (int e = threadIdx.x; e < entries; e += kThreads) {
    int64_t c[2] = {0, 0};
    for (int u = e * per; u < min(units, (e + 1) * per); ++u) {
      const Unit x = load_unit<SHARED>(p, u);
      bad_len |= x.bad;
      if (SHARED && u >= p.n_groups) c[1] += p.Hkv * own_cost(x);
      else c[0] += p.Hkv * cost_before(x, tpt, unit_items(x, tpt));
    }
    table0[e + 1] = c[0];
    if (SHARED) table1[e + 1] = c[1];
  }
  umma::fence_before_sync();
  fine = __syncthreads_and(fine);
  umma::fence_after_sync();
  const uint32_t tm = sh.tmem;
  if (fine && bad_len && cta == 0) flag(p.status, VT_DEV_BAD_LEN);
  if (fine && warp < (SHARED ? 2 : 1)) {
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
    if (lane == 31) sh.total[warp] = before;
  }
  // Behind this barrier the loading warp may have q written over the tables at any time: of the
  // other warps only those read them that a further barrier holds back.
  __syncthreads();
  if (!fine && cta == 0 && threadIdx.x == 0) flag(p.status, VT_DEV_BAD_START);
  const int64_t total = fine ? sh.total[0] : 0, pages = SHARED && fine ? sh.total[1] : 0;
  const int split = SHARED ? first_own(total, pages, gridDim.x) : gridDim.x;
  const Line tiles_line = make_line(total, max(split, 1), kMinShare);

  // What the joining kernel needs to find the pieces: from a CTA without work, if there is one.
  if (SHARED && cta == (tiles_line.n < split ? tiles_line.n : (int)gridDim.x - 1)) {
    if (fine) {
      for (int e = threadIdx.x; e < entries; e += kThreads) {
        int64_t c[2] = {table0[e], table1[e]};
        for (int u = e * per; u < min(units, (e + 1) * per); ++u) {
          const Unit x = load_unit<SHARED>(p, u);
          w.line[u] = c[u >= p.n_groups];
          if (u >= p.n_groups) c[1] += p.Hkv * own_cost(x);
          else c[0] += p.Hkv * cost_before(x, tpt, unit_items(x, tpt));
        }
      }
    }
    if (threadIdx.x == 0) {
      w.lines[0] = tiles_line;
      if (!fine) w.lines[0].total = -1;
      w.lines[1] = make_line(pages, max(((int)gridDim.x - split) * kWarps, 1), kMinPages);
    }
    __syncthreads();  // (before what comes into shared memory overwrites the tables)
  }

  if (SHARED && cta >= split) {
    // ---- own pages: a warp, a share ------------------------------------------------------------
    const Line own_line = make_line(pages, (gridDim.x - split) * kWarps, kMinPages);
    const int ws = (cta - split) * kWarps + warp;
    const int64_t x0 = ws < own_line.n ? share_begin(own_line, ws) : 0;
    const int64_t x1 = ws < own_line.n ? share_begin(own_line, ws + 1) : 0;
    OwnCursor cur;
    if (x0 < x1) cur.seek(p, table1, entries, per, x0);
    __syncthreads();  // (before the pages overwrite the tables)
    if (x0 < x1) own_share<D>(p, w, cur, x0, x1, base + warp * 2 * PageTile<D>::SLOT, ws, lane);
    __syncthreads();
    if (warp == kMmaWarp) umma::tmem_dealloc(tm, 512);
    return;
  }

  const int64_t* line = table0;
  const bool work = total > 0 && cta < tiles_line.n;
  if (warp >= kLoadWarp) {
    regs_less<kRegsOther>();
    if (warp == kLoadWarp) {
      // ---- loading -----------------------------------------------------------------------------
      if (lane == 0 && !SHARED && w.head) {
        w.head[2 * cta].valid = 0;
        w.head[2 * cta + 1].valid = 0;
      }
      int n_desc = 0, n_item = 0, n_tile = 0;
      uint32_t filled = 0;  // stage uses, for the drain
      bool go = true;
      if (work) {
        const int64_t x0 = share_begin(tiles_line, cta), x1 = share_begin(tiles_line, cta + 1);
        int lo = 0, hi = entries - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (line[mid] <= x0) lo = mid; else hi = mid - 1;
        }
        int u = lo * per;
        int64_t pos = line[lo];
        Unit un = load_unit<SHARED>(p, u);
        int items = unit_items(un, tpt);
        int64_t head_cost = cost_before(un, tpt, items);
        while (pos + p.Hkv * head_cost <= x0) {  // x0 < total, so this ends at a unit with items
          pos += p.Hkv * head_cost;
          un = load_unit<SHARED>(p, ++u);
          items = unit_items(un, tpt);
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
          const int j0 = cut_tile(x0 - pos, cost, wt, tiles);
          const int j1 = cut_tile(x1 - pos, cost, wt, tiles);
          if (j0 < j1 || (tiles == 0 && pos >= x0)) {
            // describe it
            const int di = n_desc % kDescs;
            go = wait(smem_u32(&sh.desc_empty[di]), ((n_desc / kDescs) & 1) ^ 1, abort_flag);
            if (!go) break;
            const int first = t * 2 * tpt, n_tok = min(un.n - first, 2 * tpt);
            const bool whole = j0 == 0 && j1 == tiles;
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
                const int use = 2 * n_tile + kv, st = use % C::STAGES;
                const uint32_t full = smem_u32(&sh.kv_full[st]);
                go = go &&
                     wait(smem_u32(&sh.kv_empty[st]), ((use / C::STAGES) & 1) ^ 1, abort_flag);
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
                if (kv == 0 && j == j0) {
                  // q goes behind the first K tile: its buffer is free only when the last item's
                  // scores are done
                  go = wait(smem_u32(&sh.q_empty), (n_item & 1) ^ 1, abort_flag);
                  if (!go) break;
                  const int tiles_q = n_tok > tpt ? 2 : 1;
                  if (lane == 0) {
                    const uint32_t bar = smem_u32(&sh.q_full);
                    umma::mbar_expect_tx(bar, p.G * tpt * 128 * C::HALVES * tiles_q);
                    for (int tt = 0; tt < tiles_q; ++tt)
                      for (int half = 0; half < C::HALVES; ++half)
                        umma::tma_load_3d(q_smem + tt * C::TILE + half * C::BOX, &q_map, half * 64,
                                          h * p.G, un.tok0 + first + tt * tpt, bar);
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
                if (++u == tile_units) break;
                un = load_unit<SHARED>(p, u);
                items = unit_items(un, tpt);
              } while (items == 0);
              if (u == tile_units) break;
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
      // Copies in flight must land before the shared memory goes away, also where it is another
      // warp that gives up, later than this one is done.
      for (uint32_t i = 0; i < min(filled, (uint32_t)C::STAGES); ++i) {
        const uint32_t use = filled - 1 - i;
        const unsigned long long t0 = global_ns();
        while (!umma::mbar_try_wait(smem_u32(&sh.kv_full[use % C::STAGES]),
                                    (use / C::STAGES) & 1) &&
               global_ns() - t0 < kWaitNs) {
        }
      }
      const unsigned long long t0 = global_ns();
      while (n_item > 0 && !umma::mbar_try_wait(smem_u32(&sh.q_full), (n_item - 1) & 1) &&
             global_ns() - t0 < kWaitNs) {
      }
    } else if (warp == kMmaWarp) {
      // ---- products ----------------------------------------------------------------------------
      constexpr uint32_t kIdS = umma::idesc_bf16(kTile, kKeys, false, false);
      constexpr uint32_t kIdO = umma::idesc_bf16(kTile, D, false, true);
      int n_desc = 0, n_item = 0, n_tile = 0;
      uint32_t p_phase[2] = {0, 0};
      bool go = true;
      auto scores = [&](int t, int st) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k / 4) * C::BOX + (k % 4) * 32;
          umma::mma_bf16(tm + t * kKeys,
                         umma::sdesc_sw128(q_smem + t * C::TILE + off, 0, 1024),
                         umma::sdesc_sw128(kv_smem + st * C::TILE + off, 0, 1024), kIdS, k > 0);
        }
        umma::commit(smem_u32(&sh.s_full[t]));
      };
      auto values = [&](int t, int st, int half, bool more) {
#pragma unroll
        for (int k = half * (kKeys / 32); k < (half + 1) * (kKeys / 32); ++k)
          umma::mma_bf16_ta(tm + 2 * kKeys + t * D, tm + t * kKeys + k * 8,
                            umma::sdesc_sw128(kv_smem + st * C::TILE + k * 2048, C::BOX, 1024),
                            kIdO,
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
        const int nt = n_tok > tpt ? 2 : 1;
        for (int j = j0; go && j <= j1; ++j) {
          // step j: the values of tile j - 1, then the scores of tile j, row tile by row tile
          const int kst = 2 * n_tile % C::STAGES, vst = (2 * n_tile - 1) % C::STAGES;
          if (j == j0) go = wait(smem_u32(&sh.q_full), n_item & 1, abort_flag);
          if (go && j < j1)
            go = wait(smem_u32(&sh.kv_full[kst]), (2 * n_tile / C::STAGES) & 1, abort_flag);
          if (go && j > j0)
            go = wait(smem_u32(&sh.kv_full[vst]), ((2 * n_tile - 1) / C::STAGES) & 1, abort_flag);
          for (int t = 0; go && t < nt; ++t) {
            if (j > j0) {
              go = wait(smem_u32(&sh.p_ready[t][0]), p_phase[t], abort_flag);
              if (!go) break;
              umma::fence_after_sync();
              values(t, vst, 0, j > j0 + 1);
              umma::commit(smem_u32(&sh.a_done[t]));
              go = wait(smem_u32(&sh.p_ready[t][1]), p_phase[t], abort_flag);
              if (!go) break;
              umma::fence_after_sync();
              values(t, vst, 1, true);
              p_phase[t] ^= 1;
              if (j == j1) umma::commit(smem_u32(&sh.o_full[t]));
            } else {
              umma::fence_after_sync();
            }
            if (j < j1) scores(t, kst);
          }
          if (!go) break;
          if (j > j0) umma::commit(smem_u32(&sh.kv_empty[vst]));
          if (j < j1) {
            umma::commit(smem_u32(&sh.kv_empty[kst]));
            if (j == j1 - 1) umma::commit(smem_u32(&sh.q_empty));
            ++n_tile;
          }
        }
        if (!go) break;
        ++n_item;
      }
      // what was issued finishes before the tensor memory goes away
      if (n_tile > 0) {
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
    const float c = p.qscale;
    const int Hq = p.Hkv * p.G;
    const int tok_row = row / p.G, head_row = row - tok_row * p.G;
    uint32_t s_phase = 0, o_phase = 0, a_phase = 0;
    int n_tile = 0;
    for (int n_desc = 0;; ++n_desc) {
      const int di = n_desc % kDescs;
      if (!wait(smem_u32(&sh.desc_full[di]), (n_desc / kDescs) & 1, abort_flag)) break;
      const Desc d = sh.desc[di];
      __syncwarp();
      if (lane == 0) umma::mbar_arrive(smem_u32(&sh.desc_empty[di]));
      if (d.n_tok == 0) break;
      const int n_tok = min(tpt, d.n_tok - t * tpt);
      if (n_tok <= 0) {
        n_tile += d.j1 - d.j0;
        continue;
      }
      const bool active = (warp & 3) * 32 < n_tok * p.G, mine = row < n_tok * p.G;
      const int tok = t * tpt + min(tok_row, n_tok - 1);
      const int vis = d.vis0 + tok * d.step;
      const int vis_warp = d.vis0 + (t * tpt + min((warp & 3) * 32 / p.G, n_tok - 1)) * d.step;
      const int n_pages = (d.kv_len + kPage - 1) / kPage;
      const int gap = n_pages * kPage - d.kv_len;   // zero rows ahead of the last page's tokens
      // ref: the reference of this row's weights (base 2), l: their sum, lift: what the next tile
      // adds to the reference
      float ref = -INFINITY, l = 0.0f, lift = 0.0f;
      auto move = [&](float to, bool with_o) {
        const float f = ref == -INFINITY ? 0.0f : ex2(ref - to);
        ref = to;
        l *= f;
        if (with_o) {
#pragma unroll 1
          for (int i = 0; i < D / 16; ++i) {
            uint32_t o[16];
            umma::tmem_ld16(tm_o + 16 * i, o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            umma::tmem_st16_async(tm_o + 16 * i, o);
          }
        }
      };
      // half of the keys have their weights: the product with their values can start
      auto hand_over = [&](int h) {
        umma::tmem_wait_st();
        umma::fence_before_sync();
        __syncwarp();
        if (lane == 0) umma::mbar_arrive(smem_u32(&sh.p_ready[t][h]));
      };
      bool ok = true;
      for (int j = d.j0; j < d.j1; ++j, ++n_tile, a_phase ^= 1) {
        ok = wait(smem_u32(&sh.s_full[t]), s_phase, abort_flag);
        if (!ok) break;
        s_phase ^= 1;
        if (active) {
          umma::fence_after_sync();
          const uint32_t bad = (uint32_t)*(volatile int*)&sh.bad[n_tile % kBadRing];
          const int slot0 = j * kKeys;
          const bool masked = slot0 + kKeys > vis_warp || bad;
          // The usual tile: nothing to hide, and the reference serves as it is.
          int slow = 0;  // the first half that is still to be done: 0, 1, or 2 for none
          if (!masked && __all_sync(kFull, !mine || ref > -INFINITY)) {
            if (__any_sync(kFull, mine && lift > 0.0f)) move(ref + lift, true);
            lift = 0.0f;
            const uint64_t c2 = pair(c, c), ref2 = pair(-ref, -ref);
            uint32_t s[2][32];
            float tile_sum = 0.0f;
            umma::tmem_ld32_async(tm_s, s[0]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (slow < h) continue;
              uint64_t sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
              uint32_t pk[32];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                umma::tmem_wait_ld();
                umma::tmem_landed(s[i]);
                if (h + i < 2) umma::tmem_ld32_async(tm_s + 64 * h + 32 * (i + 1), s[i ^ 1]);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const uint64_t x = exp2_unit(fma2(
                      pair(__uint_as_float(s[i][2 * e]), __uint_as_float(s[i][2 * e + 1])), c2,
                      ref2));
                  sum[e & 1] = add2(sum[e & 1], x);
                  pk[16 * i + e] = pack2(x);
                }
              }
              const float half_sum = total2(sum[0], sum[1]);
              if (__any_sync(kFull, mine && !(half_sum < kFar))) {
                umma::tmem_wait_ld();  // (a load may be in flight into these registers)
                umma::tmem_landed(s[0]);
                continue;
              }
              umma::tmem_st32_async(tm_s + 32 * h, pk);  // (over scores that were read)
              l += half_sum;
              tile_sum += half_sum;
              hand_over(h);
              slow = h + 1;
            }
            // its exponent, from 2^kLift on
            if (tile_sum >= (float)(1 << kLift))
              lift = (float)((int)(__float_as_uint(tile_sum) >> 23) - 127);
            if (slow == 1) {  // the first half is in O, or about to be: it moves with the rest
              if (!wait(smem_u32(&sh.a_done[t]), a_phase, abort_flag)) {
                ok = false;
                break;
              }
              umma::fence_after_sync();
            }
          }
          if (slow < 2) {
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
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
            for (int i = slow; i < 2; ++i) {
              uint32_t s0[32], s1[32];
              umma::tmem_ld32_async(tm_s + 64 * i, s0);
              umma::tmem_ld32_async(tm_s + 64 * i + 32, s1);
              umma::tmem_wait_ld();
              umma::tmem_landed(s0);
              umma::tmem_landed(s1);
#pragma unroll
              for (int e = 0; e < 32; e += 4)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mx[k] =
                      fmaxf(mx[k], fmaxf(__uint_as_float(s0[e + k]), __uint_as_float(s1[e + k])));
            }
            const float top =
                fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c, ref + lift);
            lift = 0.0f;
            if (__any_sync(kFull, mine && (top > ref + kLazy || (ref == -INFINITY && top > ref))))
              move(fmaxf(ref, top), j > d.j0 || slow == 1);
            const float at = ref == -INFINITY ? 0.0f : ref;
            const uint64_t c2 = pair(c, c), ref2 = pair(-at, -at);
#pragma unroll 1
            for (int h = slow; h < 2; ++h) {
              uint64_t sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll 1
              for (int i = 0; i < 2; ++i) {
                uint32_t s[32], pk[16];
                umma::tmem_ld32_async(tm_s + 64 * h + 32 * i, s);
                umma::tmem_wait_ld();
                umma::tmem_landed(s);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const uint64_t x = exp2_unit(fma2(
                      pair(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), c2, ref2));
                  sum[e & 1] = add2(sum[e & 1], x);
                  pk[e] = pack2(x);
                }
                umma::tmem_st16_async(tm_s + 32 * h + 16 * i, pk);
              }
              l += total2(sum[0], sum[1]);
              hand_over(h);
            }
          }
        } else {
          // (no weights of its own, but it may just have read the last item's O, which the product
          // behind this arrival overwrites)
          umma::fence_before_sync();
          __syncwarp();
          if (lane == 0) {
            umma::mbar_arrive(smem_u32(&sh.p_ready[t][0]));
            umma::mbar_arrive(smem_u32(&sh.p_ready[t][1]));
          }
        }
      }
      if (!ok) break;
      if (d.j0 < d.j1) {
        if (!wait(smem_u32(&sh.o_full[t]), o_phase, abort_flag)) break;
        o_phase ^= 1;
        umma::fence_after_sync();
      }
      if (!active) continue;
      // Results leave through shared memory, 128 bytes of each row at a time (16-byte piece c of
      // row r at c ^ (r % 8)), so that a store covers whole lines: straight from a thread's own
      // row it would touch 32 of them.
      const bool whole = !SHARED && d.whole;
      const int64_t orow = (int64_t)(d.tok0 + tok) * Hq + d.h * p.G + head_row;
      const float inv = l != 0.0f ? 1.0f / l : 0.0f;
      const int rows = min(32, n_tok * p.G - (warp & 3) * 32);  // of this warp, the valid ones
      // each lane's eight rows r0, r0 + 4, .. in the stores: byte offsets from the result's base
      const int r0 = lane >> 3, piece = lane & 7;
      unsigned char* base_out =
          whole ? reinterpret_cast<unsigned char*>(p.out)
                : reinterpret_cast<unsigned char*>(
                      SHARED && d.j0 == 0
                          ? w.first
                          : w.part + ((int64_t)d.slot * 2 * kTile + t * kTile) * kRowF<D>);
      const int64_t row_at = whole ? orow * D * 2
                             : (SHARED && d.j0 == 0 ? orow : (int64_t)row) * kRowF<D> * 4;
      const uint32_t stage = kv_smem + C::STAGES * C::TILE + warp * kStage;
      const int passes = whole ? D / 64 : D / 32;
#pragma unroll 1
      for (int i = 0; i < passes; ++i) {
        uint32_t o[2][16];
        if (d.j0 < d.j1) {
          const uint32_t src = tm_o + (whole ? 64 : 32) * i;
          umma::tmem_ld16_async(src, o[0]);
          umma::tmem_ld16_async(src + 16, o[1]);
          umma::tmem_wait_ld();
          umma::tmem_landed(o[0]);
          umma::tmem_landed(o[1]);
        }
        if (l == 0.0f) {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e >> 4][e & 15] = 0u;
        }
        if (whole) {  // dims 64 i .. 64 i + 31, then the 32 behind them
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            if (part) {
              if (d.j0 < d.j1) {
                umma::tmem_ld16_async(tm_o + 64 * i + 32, o[0]);
                umma::tmem_ld16_async(tm_o + 64 * i + 48, o[1]);
                umma::tmem_wait_ld();
                umma::tmem_landed(o[0]);
                umma::tmem_landed(o[1]);
              }
              if (l == 0.0f) {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e >> 4][e & 15] = 0u;
              }
            }
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
#pragma unroll
          for (int q8 = 0; q8 < 8; ++q8)
            st_shared16(stage + lane * 128 + ((q8 ^ (lane & 7)) << 4),
                        o[q8 >> 2][4 * (q8 & 3)], o[q8 >> 2][4 * (q8 & 3) + 1],
                        o[q8 >> 2][4 * (q8 & 3) + 2], o[q8 >> 2][4 * (q8 & 3) + 3]);
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
          *reinterpret_cast<float2*>(base_out + row_at + D * 4) = make_float2(ref, l);
        else if (p.lse)
          p.lse[orow] = l != 0.0f ? ref * kLn2 + logf(l) : -INFINITY;
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
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    uint32_t* dst = reinterpret_cast<uint32_t*>(out + row * D) + lane * (E / 2);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) dst[e] = pack2(o[2 * e] * inv, o[2 * e + 1] * inv);
    if (lse && lane == 0) lse[row] = l != 0.0f ? m * kLn2 + logf(l) : -INFINITY;
  }
};

constexpr int kJoinThreads = 256;
constexpr int kJoinRows = kJoinThreads / 32;

// Prompts: block (c, y) joins rows y * 8 .. of the item that begins in CTA c and ends in another.
// At most one item per CTA, two or three pieces each, out of L2: ~10 us behind a packed batch.
template <int D>
__global__ void __launch_bounds__(kJoinThreads)
    join_items_kernel(const AttendParams p, const Work w) {
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  wait_for_previous();
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

// Shared prefixes: a warp joins one row, the pieces of its group's prefix and of its own pages.
// The time is a chain of trips to memory (11 us by itself for 32 samples of a prompt, a quarter of
// the call), so it has few links:
// which shares hold a piece is worked out a lane each, all their m and l are read at once, and the
// rows eight at a time.
template <int D>
__global__ void __launch_bounds__(kJoinThreads)
    join_rows_kernel(const AttendParams p, const Work w) {
  constexpr int E = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hq = p.Hkv * p.G, tpt = kTile / p.G;
  const int orow = blockIdx.x * kJoinRows + warp;  // (B Hq < 2^31, as api.cu checks)
  if (orow >= p.B * Hq) return;
  const int b = orow / Hq, hq = orow - b * Hq;
  const int h = hq / p.G, g_row = hq - h * p.G;
  const int g = group_of(p, b);
  Unit own{}, un{};
  if (g >= 0) {  // (inputs, which the kernel before does not write)
    own = load_unit<true>(p, p.n_groups + b);
    un = load_unit<true>(p, g);
  }
  const int t = (b - un.tok0) / (2 * tpt), i = (b - un.tok0) - t * 2 * tpt;
  const int r = i / tpt * kTile + i % tpt * p.G + g_row;  // the row within the prefix's item
  const int64_t a_in = h * cost_before(un, tpt, unit_items(un, tpt)) + cost_before(un, tpt, t);
  const int64_t a_cost = un.n > 0 ? item_cost(un, tpt, t) : 0, b_cost = own_cost(own);
  const int wt = un.n > 0 ? item_weight(un, tpt, t) : 1;
  const int tiles = un.n > 0 ? (item_keys(un, tpt, t) + kKeys - 1) / kKeys : 0;
  const int n_pages = own_pages(own);
  wait_for_previous();
  const Line tl = w.lines[0], ol = w.lines[1];
  const int64_t b_pos = w.line[p.n_groups + b] + h * b_cost;
  const int64_t a_pos = (g >= 0 ? w.line[g] : 0) + a_in;
  if (tl.total < 0 || g < 0) return;
  // the shares [a0, a1) and [b0, b1) may hold pieces
  int a0 = 0, a1 = 0, b0 = 0, b1 = 0;
  if (!own.bad && un.n > 0) {
    a0 = share_of(tl, a_pos);
    a1 = share_of(tl, a_pos + a_cost - 1) + 1;
  }
  if (!own.bad && own.kv_len > 0) {
    b0 = share_of(ol, b_pos);
    b1 = share_of(ol, b_pos + b_cost - 1) + 1;
  }
  float o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.0f;
#pragma unroll 1
  for (; a0 < a1 || b0 < b1; a0 += 32, b0 += 32) {
    // this lane's piece of either kind, NULL none
    const float *pa = nullptr, *pb = nullptr;
    if (a0 + lane < a1) {
      const int j0 = cut_tile(share_begin(tl, a0 + lane) - a_pos, a_cost, wt, tiles);
      const int j1 = cut_tile(share_begin(tl, a0 + lane + 1) - a_pos, a_cost, wt, tiles);
      if (j0 < j1)
        pa = j0 == 0 ? w.first + (int64_t)orow * kRowF<D>
                     : w.part + ((int64_t)(a0 + lane) * 2 * kTile + r) * kRowF<D>;
    }
    if (b0 + lane < b1) {
      const int i0 = own_cut(share_begin(ol, b0 + lane) - b_pos, n_pages);
      const int i1 = own_cut(share_begin(ol, b0 + lane + 1) - b_pos, n_pages);
      if (i0 < i1)
        pb = i0 == 0 ? w.first + ((int64_t)p.B * Hq + orow) * kRowF<D>
                     : w.own + ((int64_t)(b0 + lane) * 8 + g_row) * kRowF<D>;
    }
    const float2 none = make_float2(-INFINITY, 0.0f);
    const float2 ma = pa ? __ldcg(reinterpret_cast<const float2*>(pa + D)) : none;
    const float2 mb = pb ? __ldcg(reinterpret_cast<const float2*>(pb + D)) : none;
    float top = fmaxf(m, fmaxf(ma.x, mb.x));
#pragma unroll
    for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, x));
    const float keep = m == -INFINITY ? 0.0f : exp2f(m - top);
    const float fa = ma.x == -INFINITY ? 0.0f : exp2f(ma.x - top);
    const float fb = mb.x == -INFINITY ? 0.0f : exp2f(mb.x - top);
    float sum = ma.y * fa + mb.y * fb;
#pragma unroll
    for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(kFull, sum, x);
    l = l * keep + sum;
    m = top;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= keep;
    uint64_t left = __ballot_sync(kFull, pa != nullptr) |
                    (uint64_t)__ballot_sync(kFull, pb != nullptr) << 32;
    while (left) {
      constexpr int kAtOnce = 8;
      float x[kAtOnce][E], f[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const bool has = left != 0;
        const int src = has ? __ffsll((long long)left) - 1 : 0;
        left &= left - 1;
        const float* mine = src < 32 ? pa : pb;
        const float* row = reinterpret_cast<const float*>(
            __shfl_sync(kFull, reinterpret_cast<unsigned long long>(mine), src & 31));
        f[k] = __shfl_sync(kFull, src < 32 ? fa : fb, src & 31);
        if (!has) f[k] = 0.0f;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 v = has ? __ldcg(reinterpret_cast<const float2*>(row + lane * E + e))
                               : make_float2(0.0f, 0.0f);
          x[k][e] = v.x;
          x[k][e + 1] = v.y;
        }
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(x[k][e], f[k], o[e]);
    }
  }
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + (int64_t)orow * D) + lane * (E / 2);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) dst[e] = pack2(o[2 * e] * inv, o[2 * e + 1] * inv);
  if (p.lse && lane == 0) p.lse[orow] = l != 0.0f ? m * kLn2 + logf(l) : -INFINITY;
}

// ---- host -----------------------------------------------------------------------------------

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Whether prompts of these sizes can be more than one CTA's share, whatever their lengths: if
// not, no item is cut, and there is nothing to join and no workspace.
bool may_split(const AttendParams& p) {
  const int64_t tpt = kTile / p.G, items = p.Hkv * (p.T / (2 * tpt) + std::min<int64_t>(p.B, p.T));
  return items * kCostKey * (kCostItem + p.max_pages * kPage) >= 2 * kMinShare;
}

// Fills w from ws (NULL: only the size is wanted) and returns the bytes.
size_t lay_out(const AttendParams& p, int ctas, void* ws, Work* w) {
  const bool shared = p.prefix_pages != nullptr;
  if (!shared && !may_split(p)) {
    if (w) *w = Work{};
    return 0;
  }
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
  x.own = reinterpret_cast<float*>(take(shared ? (size_t)ctas * kWarps * 8 * row : 0));
  x.line = reinterpret_cast<int64_t*>(take(shared ? ((size_t)p.n_groups + p.B) * 8 : 0));
  x.lines = reinterpret_cast<Line*>(take(shared ? 2 * sizeof(Line) : 0));
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
  CUtensorMap q, k, v;
  const int64_t qd[3] = {D, (int64_t)p.Hkv * p.G, p.T}, qs[2] = {D, p.sq_t};
  const int qb[3] = {64, p.G, tpt};
  const int64_t kd[4] = {D, kPage, p.Hkv, p.kv.num_pages};
  const int64_t ks[3] = {p.kv.sk_t, p.kv.sk_h, p.kv.sk_p};
  const int64_t vs[3] = {p.kv.sv_t, p.kv.sv_h, p.kv.sv_p};
  const int kb[4] = {64, kPage, 1, 1};
  if (!encode_fn() || !encode(&q, p.q, 3, qd, qs, qb) ||
      !encode(&k, p.kv.k_pool, 4, kd, ks, kb) || !encode(&v, p.kv.v_pool, 4, kd, vs, kb))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(attend_kernel<D, SHARED>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  attend_kernel<D, SHARED><<<ctas, kThreads, Cfg<D>::SMEM, s>>>(p, w, q, k, v);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (SHARED) {
    const int64_t rows = (int64_t)p.B * p.Hkv * p.G;
    return launch_after(join_rows_kernel<D>, dim3((unsigned)((rows + kJoinRows - 1) / kJoinRows)),
                        kJoinThreads, s, p, w);
  }
  if (!w.head) return cudaSuccess;
  return launch_after(join_items_kernel<D>, dim3(ctas, 2 * kTile / kJoinRows), kJoinThreads, s, p,
                      w);
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
