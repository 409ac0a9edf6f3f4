// Attention weight that each key receives from the last queries of a
// sequence, without writing the probabilities:
//     weights[b, g, j] = sum_{h in group g} sum_{i in window, i >= j}
//                        2^(x_hij - lse_hi),   x = log2(e) scale q_hi . k_gj.
//
// Launch 1 (stats): lse_hi = log2 sum_{j <= i} 2^(x_hij).  An item is 128
// query rows of one KV head (two runs of 64: consecutive ones of a head, or
// two heads of the group, which share the keys); it walks 64-key tiles: S =
// Q K^T on the tensor cores, one running (max, sum) per row and group of
// warps.  With few row tiles the keys are split over items, and the CTA that
// finishes a row tile last joins the parts in split order.
// Launch 2 (sums): an item is 128 keys; it walks the 64-row runs of queries
// that see them, S^T = K Q^T: a thread owns a key and adds up 2^(x - lse) in
// fp32, one partial sum a run.  No atomics: the order of every sum is fixed.
//
// The scores are computed twice (2 D flops each) because keeping them would
// write and read 4 bytes per (query, key, head): at 2048 tokens x 32 heads
// 268 MB each way, 80 us.  Both launches are bound by the special-function
// unit, one exponential per score: 16 per clock and SM, 512 clocks for a 128 x
// 64 tile, which its products (N = 64 runs at half the tensor rate) take too
// at D = 128.
//
// Persistent CTAs, two per SM, so that one's waits are filled by the other (98
// KB of shared memory, 256 tensor-memory columns, 96 registers a thread): a
// TMA warp, an MMA warp, and two groups of four softmax warps that take the
// tiles in turn.  2048 tokens x 32 heads / the last 64 of 16000 tokens, 32
// heads, batch 2, both launches: both operands in shared memory and an item a
// CTA 78 / 87 us; the stationary one in tensor memory, packed arithmetic 63 /
// 74; persistent CTAs that load the next item's operand meanwhile 63 / 64;
// masked tiles in a body of their own, no second source for the scores 60.5 /
// 61; the second launch waiting for the statistics alone 59 / 59 (the
// exponentials alone: 30 / 29).  4096 tokens: 180 us (119).
//
// Not faster: one CTA per SM with 128 x 128 tiles and a quarter of the
// exponentials on the FMA pipe (201 us at 4096 tokens), 256 stationary rows
// (207: half the traffic from L2), 128 x 128 tiles in two CTAs with one S
// buffer (190), the same with the next item's operand in tensor memory ahead
// of time (191), and with the next tile's scores loaded ahead too (203).
// Without the exponentials 4096 tokens take 159 us, without seven eighths of
// the products 187, without both 120: the chain of waits, tensor-memory loads
// and hand-offs of a tile (900 clocks), the exponentials and the products each
// fill most of the time, and four warps per scheduler, all that registers
// allow, overlap them to 0.65 of the exponentials' rate.
// Every wait is bounded.
#include <cstring>

#include "kernels.h"
#include "tc.cuh"

namespace fsvd {
namespace {

constexpr int SU_THREADS = 320;  // TMA warp, MMA warp, 8 softmax warps
constexpr int SU_RUN = 64;       // query rows of a run
constexpr int SU_KEYS = 128;     // keys of a tile
constexpr int SU_MIN_TILES = 6;   // 64-key tiles of a split, at least

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (x0, x1) * (s, s) + (c0, c1) as one packed instruction.
__device__ __forceinline__ void fma2(float& x0, float& x1, float s, float c0, float c1) {
  asm("{\n\t.reg .b64 xx, ss, cc;\n\t"
      "mov.b64 xx, {%0, %1};\n\t"
      "mov.b64 ss, {%2, %2};\n\t"
      "mov.b64 cc, {%3, %4};\n\t"
      "fma.rn.f32x2 xx, xx, ss, cc;\n\t"
      "mov.b64 {%0, %1}, xx;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(s), "f"(c0), "f"(c1));
}
// (a0, a1) += (b0, b1) as one packed instruction.
__device__ __forceinline__ void add2(float& a0, float& a1, float b0, float b1) {
  asm("{\n\t.reg .b64 aa, bb;\n\t"
      "mov.b64 aa, {%0, %1};\n\t"
      "mov.b64 bb, {%2, %3};\n\t"
      "add.rn.f32x2 aa, aa, bb;\n\t"
      "mov.b64 {%0, %1}, aa;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <bool V>
struct SuBool {
  static constexpr bool value = V;
};

struct SuParams {
  const int* lens;
  float* weights;
  float* lse;        // [B][H][runs * 64]: -lse; -inf where there is no query
  float2* part;      // key splits: [B][G][row tiles][splits][128] (max, sum)
  int* counters;     // [B * G * row tiles], zero between launches
  int B, S, H, G, S_max, w_stride, window;
  int rep, runs;     // query heads per KV head; runs of the full window
  int row_tiles, splits;
  float scale_log2;
  int* status;
};

// One kernel's CTA: a tile of 128 rows (queries or keys) is the A operand and
// is moved into tensor memory once; runs of 64 rows of the other tensor pass
// through a ring of shared memory as B.  (With both operands in shared memory
// each 128 x 64 x 16 step reads 6 KB for 32 cycles of products, at 128 bytes a
// clock: two CTAs on an SM measured 800 cycles a tile instead of 256.)
template <int D>
struct SuLayout {
  static constexpr int KB = D / 64;
  static constexpr int RUN_B = SU_RUN * 128;    // one [64 x 64] bf16 block, 8 KB
  static constexpr int ROWS_B = 128 * 128;      // one [128 x 64] bf16 block, 16 KB
  static constexpr int NST = 4;
  static constexpr int RING = KB * ROWS_B;
  static constexpr int LSE = RING + NST * KB * RUN_B;      // the runs' -lse (sums)
  static constexpr int BAR = LSE + NST * SU_RUN * 4;
  static constexpr int XCH = BAR + 256;                    // exchange between the two threads of a row
  static constexpr int SMEM = 1024 + XCH + 2 * 128 * 8;
  static constexpr uint32_t TM_S = 64;          // tensor memory: A in [0, D / 2), S buffers of 64 from here
  static constexpr int NS = 3;
};

// Barriers of a CTA, in shared memory.
template <int D>
struct SuBars {
  uint64_t a_full, a_empty, a_tmem, a_free, full[SuLayout<D>::NST], empty[SuLayout<D>::NST];
  uint64_t s_full[SuLayout<D>::NS], s_empty[SuLayout<D>::NS], drain;
  uint32_t tmem;
  int abort_flag, last;
};

// Barrier set-up and tensor memory (held before dependents may start: a
// dependent kernel that took it first would wait for this one, and this one
// for it).  `readers`: arrivals that free a ring stage.
template <int D>
__device__ __forceinline__ uint32_t su_begin(SuBars<D>* bars, int readers, int warp) {
  if (threadIdx.x == 0) {
    tc::mbar_init(&bars->a_full, 1);
    tc::mbar_init(&bars->a_empty, 4);
    tc::mbar_init(&bars->a_tmem, 4);
    tc::mbar_init(&bars->a_free, 1);
    for (int i = 0; i < SuLayout<D>::NST; ++i) { tc::mbar_init(bars->full + i, 1); tc::mbar_init(bars->empty + i, readers); }
    for (int i = 0; i < SuLayout<D>::NS; ++i) { tc::mbar_init(bars->s_full + i, 1); tc::mbar_init(bars->s_empty + i, 4); }
    tc::mbar_init(&bars->drain, 1);
    bars->abort_flag = 0;
    tc::fence_barrier_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(&bars->tmem, 256);
    tc::tmem_relinquish();
    tc::fence_before_sync();
  }
  __syncthreads();
  tc::fence_after_sync();
  return bars->tmem;
}
template <int D>
__device__ __forceinline__ void su_end(SuBars<D>* bars, uint32_t tmem, int warp, int lane) {
  tc::fence_before_sync();
  __syncthreads();
  if (bars->abort_flag && warp == 0 && lane == 0) {
    // let copies still in flight land before shared memory is released
    const long long c0 = clock64();
    while (clock64() - c0 < 2000000) {}
  }
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 256);
  }
}

// The MMA warp's lane.  Item j (of those with work): `n` products A . run^T
// (runs through the ring) into the S buffers in turn; t counts the CTA's
// products so far.
template <int D>
__device__ __forceinline__ bool su_products(SuBars<D>* bars, uint8_t* smem, uint32_t tmem, int j, int t, int n,
                                            int* status) {
  using L = SuLayout<D>;
  constexpr uint32_t IDESC = tc::idesc_bf16(SU_RUN, false);
  volatile int* abort_flag = &bars->abort_flag;
  if (!tc::mbar_wait(&bars->a_tmem, (uint32_t)j & 1u, abort_flag, status)) return false;
  for (int k = t; k < t + n; ++k) {
    const int st = k % L::NST, sb = k % L::NS;
    if (!tc::mbar_wait(bars->full + st, (uint32_t)(k / L::NST) & 1u, abort_flag, status)) return false;
    if (!tc::mbar_wait(bars->s_empty + sb, ((uint32_t)(k / L::NS) & 1u) ^ 1u, abort_flag, status)) return false;
    tc::fence_after_sync();
    const uint32_t sq = tc::smem_u32(smem + L::RING + st * L::KB * L::RUN_B);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
      tc::mma_bf16_ts(tmem + L::TM_S + sb * SU_RUN, tmem + kk * 8,
                      tc::sdesc_sw128(sq + (kk >> 2) * L::RUN_B + (kk & 3) * 32, 16, 1024), IDESC, kk > 0 ? 1u : 0u);
    tc::mma_commit(bars->s_full + sb);
    tc::mma_commit(bars->empty + st);
  }
  tc::mma_commit(&bars->a_free);  // the item's products are done: A may be overwritten
  return true;
}
template <int D>
__device__ __forceinline__ void su_drain(SuBars<D>* bars) {
  tc::mma_commit(&bars->drain);
  const long long c0 = clock64();
  while (!tc::mbar_try_wait(&bars->drain, 0) && clock64() - c0 < tc::kWaitCycles) {}
}

// Four warps: item j's A tile from shared memory (128-byte swizzle) into
// tensor memory, row r in lane r, two bf16 per column.
template <int D>
__device__ __forceinline__ bool su_a_to_tmem(SuBars<D>* bars, const uint8_t* smem, uint32_t tmem, int j, int row, int lane,
                                             int* status) {
  using L = SuLayout<D>;
  volatile int* abort_flag = &bars->abort_flag;
  bool ok = tc::mbar_wait(&bars->a_full, (uint32_t)j & 1u, abort_flag, status);
  if (j > 0) ok = tc::mbar_wait(&bars->a_free, (uint32_t)(j - 1) & 1u, abort_flag, status) && ok;
  ok = __all_sync(0xffffffffu, ok);
  if (ok) {
    tc::fence_after_sync();
#pragma unroll
    for (int kb = 0; kb < L::KB; ++kb) {
      uint32_t r[32];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const uint4 v = *reinterpret_cast<const uint4*>(smem + kb * L::ROWS_B + row * 128 + ((u ^ (row & 7)) << 4));
        r[4 * u] = v.x; r[4 * u + 1] = v.y; r[4 * u + 2] = v.z; r[4 * u + 3] = v.w;
      }
      tc::tmem_st32(tmem + ((uint32_t)(row & ~31) << 16) + kb * 32, r);
    }
    tc::tmem_st_wait();
  }
  tc::fence_before_sync();
  __syncwarp();
  if (lane == 0) { tc::mbar_arrive(&bars->a_tmem); tc::mbar_arrive(&bars->a_empty); }
  return ok;
}

// A thread's 64 scores from tensor memory; its warp's loads are done on return.
// (After a failed wait too, whatever is there: a second source for the scores
// would cost a move for each.)
__device__ __forceinline__ void su_scores(float (&s)[64], uint32_t addr) {
  tc::fence_after_sync();
  tc::tmem_ld32(addr, reinterpret_cast<uint32_t*>(s));
  tc::tmem_ld32(addr + 32, reinterpret_cast<uint32_t*>(s + 32));
  tc::tmem_ld_wait();
  tc::reg_fence<64>(s);
  tc::fence_before_sync();
  __syncwarp();
}

// Persistent CTAs walk the items i G + c (odd rounds: i G + G - 1 - c) of a
// list that begins with the longest ones, so that long and short ones pair up.
// Every role walks the list by itself; an item with nothing to do is passed
// over by all of them.
struct SuItem {
  int pair, b, g, t;  // (batch row, KV head); row tile (stats) or key tile (sums)
  int sp;             // key split (stats)
  int len;            // tokens of the batch row, as read
};
__device__ __forceinline__ int su_index(int i) {
  const int G = gridDim.x, c = blockIdx.x;
  return i * G + ((i & 1) ? G - 1 - c : c);
}
__device__ __forceinline__ SuItem su_item(const SuParams& p, int k, bool stats) {
  SuItem it;
  const int pairs = p.B * p.G;
  int rest = k;
  it.sp = 0;
  if (stats) {
    rest = k / p.splits;
    it.sp = k - rest * p.splits;
  }
  it.t = rest / pairs;
  it.pair = rest - it.t * pairs;
  if (stats) it.t = p.row_tiles - 1 - it.t;  // the last rows see the most keys
  it.b = it.pair / p.G;
  it.g = it.pair - it.b * p.G;
  it.len = p.lens ? p.lens[it.b] : p.S;
  return it;
}
// The window of an item's sequence: tokens, first query, runs of 64 queries.
struct SuRow {
  int n, lo, runs;
  __device__ SuRow(const SuParams& p, int len) {
    n = len < 0 ? 0 : (len > p.S ? p.S : len);
    lo = n > p.window ? n - p.window : 0;
    runs = (n - lo + SU_RUN - 1) / SU_RUN;
  }
};
// Stats: the item's two (run, head) of the run-major list, and its 64-key
// tiles t0 .. t0 + n (those some row of it sees, one split's part).
struct SuStats {
  int run[2], head[2], two, t0, n;
  __device__ SuStats(const SuParams& p, const SuItem& it, const SuRow& R) {
    const int r0 = 2 * it.t, all = R.runs * p.rep;
    run[0] = r0 / p.rep; head[0] = r0 - run[0] * p.rep;
    run[1] = (r0 + 1) / p.rep; head[1] = r0 + 1 - run[1] * p.rep;
    two = r0 + 1 < all;
    const int last_q = min(R.n - 1, R.lo + ((two ? run[1] : run[0]) + 1) * SU_RUN - 1), nt = last_q / SU_RUN + 1;
    t0 = (int)((long long)it.sp * nt / p.splits);
    n = r0 < all ? (int)((long long)(it.sp + 1) * nt / p.splits) - t0 : 0;
  }
  __device__ bool live(const SuParams& p, const SuItem& it, const SuRow& R) const { return 2 * it.t < R.runs * p.rep; }
};
// Sums: first run that sees a key of the tile, and the (run, head) from it on.
struct SuSums {
  int key0, run0, n;
  __device__ SuSums(const SuParams& p, const SuItem& it, const SuRow& R) {
    key0 = it.t * SU_KEYS;
    run0 = key0 > R.lo ? (key0 - R.lo) / SU_RUN : 0;
    n = key0 < R.n ? (R.runs - run0) * p.rep : 0;
  }
};

template <int D>
__global__ void __launch_bounds__(SU_THREADS, 2)
attn_stats_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ SuParams p) {
  using L = SuLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  SuBars<D>* bars = reinterpret_cast<SuBars<D>*>(smem + L::BAR);
  float2* xch = reinterpret_cast<float2*>(smem + L::XCH);  // [2][128]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t tmem = su_begin<D>(bars, 1, warp);
  // q and k are there once this returns: the second launch, which can start
  // now, reads them without waiting, and waits for the statistics alone
  pdl_wait();
  pdl_launch_dependents();
  const int items = p.B * p.G * p.row_tiles * p.splits;

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      for (int i = 0, j = 0, t = 0; ok && su_index(i) < items; ++i) {
        const SuItem it = su_item(p, su_index(i), true);
        const SuRow R(p, it.len);
        const SuStats w(p, it, R);
        if (w.n == 0) continue;
        if (!(ok = tc::mbar_wait(&bars->a_empty, ((uint32_t)j & 1u) ^ 1u, &bars->abort_flag, p.status))) break;
        tc::mbar_expect_tx(&bars->a_full, (1 + w.two) * L::KB * L::RUN_B);
        for (int x = 0; x < 1 + w.two; ++x)
          for (int kb = 0; kb < L::KB; ++kb)
            tc::tma_load_2d(smem + kb * L::ROWS_B + x * L::RUN_B, &tmQ, &bars->a_full,
                            (it.g * p.rep + w.head[x]) * D + 64 * kb, it.b * p.S + R.lo + w.run[x] * SU_RUN);
        for (int k = t; k < t + w.n; ++k) {
          const int st = k % L::NST;
          if (!(ok = tc::mbar_wait(bars->empty + st, ((uint32_t)(k / L::NST) & 1u) ^ 1u, &bars->abort_flag, p.status))) break;
          tc::mbar_expect_tx(bars->full + st, L::KB * L::RUN_B);
          for (int kb = 0; kb < L::KB; ++kb)
            tc::tma_load_2d(smem + L::RING + (st * L::KB + kb) * L::RUN_B, &tmK, bars->full + st, it.g * D + 64 * kb,
                            it.b * p.S_max + (w.t0 + k - t) * SU_RUN);
        }
        t += w.n;
        ++j;
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      bool ok = true;
      for (int i = 0, j = 0, t = 0; ok && su_index(i) < items; ++i) {
        const SuItem it = su_item(p, su_index(i), true);
        const SuRow R(p, it.len);
        const SuStats w(p, it, R);
        if (w.n == 0) continue;
        ok = su_products<D>(bars, smem, tmem, j, t, w.n, p.status);
        t += w.n;
        ++j;
      }
      su_drain<D>(bars);
    }
  } else {
    // two groups of four warps take the tiles in turn, a thread a row
    const int quad = warp & 3, grp = (warp - 2) >> 2;
    const int row = quad * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const float sc = p.scale_log2;
    bool ok = true;
    int i = 0, j = 0, t = 0, done = 0;  // items: of the list, with products, finished
    SuItem next = su_item(p, min(su_index(0), items - 1), true);
    for (; su_index(i) < items; ++i) {
      const SuItem it = next;
      if (su_index(i + 1) < items) next = su_item(p, su_index(i + 1), true);  // (its length arrives meanwhile)
      const SuRow R(p, it.len);
      const SuStats w(p, it, R);
      if (!w.live(p, it, R)) continue;
      const int half = row >> 6;
      const int run = half ? w.run[1] : w.run[0], head = half ? w.head[1] : w.head[0];
      const bool mine = half == 0 || w.two;
      const int q = R.lo + run * SU_RUN + (row & 63);  // query position
      float* lse = p.lse + ((long long)(it.b * p.H + it.g * p.rep + head) * p.runs + run) * SU_RUN + (row & 63);
      float m = -INFINITY, l = 0.f;
      if (grp == 0 && w.n > 0) ok = su_a_to_tmem<D>(bars, smem, tmem, j, row, lane, p.status) && ok;
      for (int k = t + grp; k < t + w.n; k += 2) {
        const int sb = k % L::NS, key0 = (w.t0 + k - t) * SU_RUN;
        ok = ok && __all_sync(0xffffffffu, tc::mbar_wait(bars->s_full + sb, (uint32_t)(k / L::NS) & 1u, &bars->abort_flag,
                                                         p.status));
        // (two bodies, with the load in them: with one load and a branch around
        // the mask alone every tile paid for the mask's selects)
        auto tile = [&](auto diagonal) {
          float s[64];
          su_scores(s, tmem + lane_base + L::TM_S + sb * SU_RUN);
          if (lane == 0) tc::mbar_arrive(bars->s_empty + sb);
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  #pragma unroll
          for (int c = 0; c < 64; c += 2) {
            if (diagonal.value) {
              s[c] = key0 + c > q ? -INFINITY : s[c];
              s[c + 1] = key0 + c + 1 > q ? -INFINITY : s[c + 1];
            }
            m4[(c >> 1) & 3] = max3(m4[(c >> 1) & 3], s[c], s[c + 1]);
          }
          const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * sc;
          if (mx > m) {
            l *= ex2f(m - mx);
            m = mx;
          }
          const float e = m == -INFINITY ? 0.f : -m;
          float a4[4] = {0.f, 0.f, 0.f, 0.f};
  #pragma unroll
          for (int c = 0; c < 64; c += 2) {
            fma2(s[c], s[c + 1], sc, e, e);
            add2(a4[c & 2], a4[(c & 2) + 1], ex2f(s[c]), ex2f(s[c + 1]));
          }
          l += (a4[0] + a4[1]) + (a4[2] + a4[3]);
        };
        if (__any_sync(0xffffffffu, key0 + 63 > q))
          tile(SuBool<true>{});
        else
          tile(SuBool<false>{});
      }
      t += w.n;
      float2* x = xch + (done++ & 1) * 128 + row;  // (in turn: the last item's may still be read)
      if (grp == 1) *x = make_float2(m, l);
      asm volatile("bar.sync 1, 256;" ::: "memory");
      const int cell = it.pair * p.row_tiles + it.t;  // row tile of the pair
      if (grp == 0) {
        const float2 o = *x;
        const float M = fmaxf(m, o.x);
        const float e = M == -INFINITY ? 0.f : M;
        const float sum = l * ex2f(m - e) + o.y * ex2f(o.x - e);
        if (p.splits == 1) {
          if (mine) *lse = q < R.n ? -(M + log2f(sum)) : -INFINITY;
        } else {
          __stcg(p.part + ((long long)cell * p.splits + it.sp) * 128 + row, make_float2(M, sum));
        }
      }
      if (p.splits > 1) {
        __threadfence();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (threadIdx.x == 64) {
          const int old = atomicAdd(p.counters + cell, 1);
          bars->last = old == p.splits - 1;
          if (old == p.splits - 1) p.counters[cell] = 0;
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (bars->last && grp == 0 && mine) {
          __threadfence();
          const float2* src = p.part + (long long)cell * p.splits * 128 + row;
          float M = -INFINITY;
  #pragma unroll 8
          for (int z = 0; z < p.splits; ++z) M = fmaxf(M, __ldcg(src + z * 128).x);
          const float e = M == -INFINITY ? 0.f : M;
          float sum = 0.f;
  #pragma unroll 8
          for (int z = 0; z < p.splits; ++z) {
            const float2 o = __ldcg(src + z * 128);
            sum += o.y * ex2f(o.x - e);
          }
          *lse = q < R.n ? -(M + log2f(sum)) : -INFINITY;
        }
      }
      if (w.n > 0) ++j;
    }  // items
  }
  su_end<D>(bars, tmem, warp, lane);
}

template <int D>
__global__ void __launch_bounds__(SU_THREADS, 2)
attn_sums_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ SuParams p) {
  using L = SuLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  SuBars<D>* bars = reinterpret_cast<SuBars<D>*>(smem + L::BAR);
  float* xch = reinterpret_cast<float*>(smem + L::XCH);  // [2][128]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t tmem = su_begin<D>(bars, 5, warp);      // the MMA and the four warps that read the lse
  pdl_launch_dependents();

  const int items = p.B * p.G * ((p.S + SU_KEYS - 1) / SU_KEYS);

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      for (int i = 0, j = 0, t = 0; ok && su_index(i) < items; ++i) {
        const SuItem it = su_item(p, su_index(i), false);
        const SuRow R(p, it.len);
        const SuSums w(p, it, R);
        if (w.n == 0) continue;
        if (!(ok = tc::mbar_wait(&bars->a_empty, ((uint32_t)j & 1u) ^ 1u, &bars->abort_flag, p.status))) break;
        tc::mbar_expect_tx(&bars->a_full, L::KB * L::ROWS_B);
        for (int kb = 0; kb < L::KB; ++kb)
          for (int x = 0; x < 2; ++x)
            tc::tma_load_2d(smem + kb * L::ROWS_B + x * L::RUN_B, &tmK, &bars->a_full, it.g * D + 64 * kb,
                            it.b * p.S_max + w.key0 + x * SU_RUN);
        for (int k = t, run = w.run0, h = 0; k < t + w.n; ++k, ++h) {
          const int st = k % L::NST;
          if (h == p.rep) { h = 0; ++run; }
          if (!(ok = tc::mbar_wait(bars->empty + st, ((uint32_t)(k / L::NST) & 1u) ^ 1u, &bars->abort_flag, p.status))) break;
          tc::mbar_expect_tx(bars->full + st, L::KB * L::RUN_B + SU_RUN * 4);
          const int head = it.g * p.rep + h;
          for (int kb = 0; kb < L::KB; ++kb)
            tc::tma_load_2d(smem + L::RING + (st * L::KB + kb) * L::RUN_B, &tmQ, bars->full + st, head * D + 64 * kb,
                            it.b * p.S + R.lo + run * SU_RUN);
          if (k == 0) pdl_wait();  // for the statistics
          const float* src = p.lse + ((long long)(it.b * p.H + head) * p.runs + run) * SU_RUN;
          asm volatile(
              "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                  tc::smem_u32(smem + L::LSE + st * SU_RUN * 4)),
              "l"(src), "r"(SU_RUN * 4), "r"(tc::smem_u32(bars->full + st))
              : "memory");
        }
        t += w.n;
        ++j;
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      bool ok = true;
      for (int i = 0, j = 0, t = 0; ok && su_index(i) < items; ++i) {
        const SuItem it = su_item(p, su_index(i), false);
        const SuRow R(p, it.len);
        const SuSums w(p, it, R);
        if (w.n == 0) continue;
        ok = su_products<D>(bars, smem, tmem, j, t, w.n, p.status);
        t += w.n;
        ++j;
      }
      su_drain<D>(bars);
    }
  } else {
    // two groups of four warps take the runs in turn, a thread a key
    const int quad = warp & 3, grp = (warp - 2) >> 2;
    const int row = quad * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const float sc = p.scale_log2;
    bool ok = true;
    int i = 0, j = 0, t = 0;
    SuItem next = su_item(p, min(su_index(0), items - 1), false);
    for (; su_index(i) < items; ++i) {
      const SuItem it = next;
      if (su_index(i + 1) < items) next = su_item(p, su_index(i + 1), false);  // (its length arrives meanwhile)
      const SuRow R(p, it.len);
      const SuSums w(p, it, R);
      if (w.n == 0) continue;
      const int key0 = w.key0, key = key0 + row;
      float total = 0.f;
      if (grp == 0) ok = su_a_to_tmem<D>(bars, smem, tmem, j, row, lane, p.status) && ok;
      int q0 = R.lo + w.run0 * SU_RUN, h = grp;  // position of the run's first query
      for (int k = t + grp; k < t + w.n; k += 2, h += 2) {
        const int st = k % L::NST, sb = k % L::NS;
        while (h >= p.rep) { h -= p.rep; q0 += SU_RUN; }
        ok = ok && __all_sync(0xffffffffu, tc::mbar_wait(bars->full + st, (uint32_t)(k / L::NST) & 1u, &bars->abort_flag,
                                                         p.status));
        ok = ok && __all_sync(0xffffffffu, tc::mbar_wait(bars->s_full + sb, (uint32_t)(k / L::NS) & 1u, &bars->abort_flag,
                                                         p.status));
        const float4* ls = reinterpret_cast<const float4*>(smem + L::LSE + st * SU_RUN * 4);
        auto tile = [&](auto edge) {
          float s[64];
          su_scores(s, tmem + lane_base + L::TM_S + sb * SU_RUN);
          if (lane == 0) tc::mbar_arrive(bars->s_empty + sb);
          float a4[4] = {0.f, 0.f, 0.f, 0.f};
  #pragma unroll
          for (int c = 0; c < 64; c += 4) {
            const float4 e = ls[c >> 2];
            fma2(s[c], s[c + 1], sc, e.x, e.y);
            fma2(s[c + 2], s[c + 3], sc, e.z, e.w);
            float y[4];
  #pragma unroll
            for (int i = 0; i < 4; ++i) {
              y[i] = ex2f(s[c + i]);
              if (edge.value) y[i] = q0 + c + i < key || q0 + c + i >= R.n ? 0.f : y[i];
            }
            add2(a4[0], a4[1], y[0], y[1]);
            add2(a4[2], a4[3], y[2], y[3]);
          }
          total += (a4[0] + a4[1]) + (a4[2] + a4[3]);
        };
        // edge: queries before the key, and rows behind the sequence (whatever they hold)
        if (q0 < key0 + SU_KEYS || q0 + SU_RUN > R.n)
          tile(SuBool<true>{});
        else
          tile(SuBool<false>{});
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bars->empty + st);
      }
      t += w.n;
      ++j;
      float* x = xch + (j & 1) * 128 + row;  // (in turn: the last item's may still be read)
      if (grp == 1) *x = total;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (grp == 0 && ok && key < R.n) p.weights[(long long)it.pair * p.w_stride + key] = total + *x;
    }  // items
  }
  pdl_wait();  // (a CTA without items too: what follows this launch takes the one before it for done)
  su_end<D>(bars, tmem, warp, lane);
}

template <int D>
int launch_sums(const AttnSumsParams& a, int sm_count, cudaStream_t stream) {
  using L = SuLayout<D>;
  SuParams p;
  memset(&p, 0, sizeof(p));
  p.lens = a.lens; p.weights = a.weights;
  p.B = a.B; p.S = a.S; p.H = a.H; p.G = a.G; p.S_max = a.S_max; p.w_stride = a.w_stride;
  p.window = a.window < a.S ? a.window : a.S;
  p.rep = a.H / a.G;
  p.runs = ceil_div(p.window, SU_RUN);
  p.scale_log2 = a.scale_log2;
  p.status = a.status;
  const long long pairs = (long long)a.B * a.G, heads = (long long)a.B * a.H;
  p.row_tiles = ceil_div(p.runs * p.rep, 2);
  const int key_tiles = ceil_div(a.S, SU_KEYS);
  // With fewer row tiles than resident CTAs (two per SM) their keys are split,
  // SU_MIN_TILES 64-key tiles or more a part: joining parts costs about 4 us, as
  // much as six tiles (300 tokens x 8 heads: five parts 17.2 us, one 13.8; last
  // 64 of 4096 tokens, 8 heads, batch 2: parts of 2, 6 and 12 tiles 16.3, 17.5
  // and 21.3).
  const long long tiles = pairs * p.row_tiles, slots = 2LL * sm_count;
  const long long parts = ceil_div(2 * key_tiles, SU_MIN_TILES);
  long long splits = slots / tiles < parts ? slots / tiles : parts;
  if (splits < 1 || tiles > a.counters_cap) splits = 1;
  p.splits = (int)splits;
  const long long lse = heads * p.runs * SU_RUN;
  const long long part = splits > 1 ? tiles * splits * 128 * 2 : 0;
  if (lse + part > a.ws_cap || tiles * splits > 0x7fffffffLL || pairs * key_tiles > 0x7fffffffLL)
    return FLASHSVD_ERR_UNSUPPORTED_SHAPE;
  p.lse = a.ws;
  p.part = reinterpret_cast<float2*>(a.ws + lse);
  p.counters = a.counters;
  CUtensorMap mq, mk;
  const long long HD = (long long)a.H * D, GD = (long long)a.G * D;
  FSVD_TRY(encode_map(&mq, a.q, (long long)a.B * a.S, HD, HD, 64, SU_RUN, true));
  FSVD_TRY(encode_map(&mk, a.k, (long long)a.B * a.S_max, GD, GD, 64, SU_RUN, true));
  auto k1 = attn_stats_kernel<D>;
  auto k2 = attn_sums_kernel<D>;
  static SmemAttrOnce once1, once2;
  FSVD_TRY(set_smem_once(once1, k1, L::SMEM));
  FSVD_TRY(set_smem_once(once2, k2, L::SMEM));
  const double pq = (double)p.window * a.S - 0.5 * (double)p.window * p.window;  // visible pairs
  const double bytes = 2.0 * D * a.B * ((double)p.window * a.H + (double)a.S * a.G);
  const LaunchTag t1{"attn_stats", bytes + 4.0 * lse, 2.0 * D * heads * pq};
  const LaunchTag t2{"attn_sums", bytes + 4.0 * lse + 4.0 * pairs * a.S, 2.0 * D * heads * pq};
  FSVD_TRY(launch_pdl(t1, k1, dim3((unsigned)(tiles * splits < slots ? tiles * splits : slots)), dim3(SU_THREADS), (size_t)L::SMEM, stream, mq, mk, p));
  return launch_pdl(t2, k2, dim3((unsigned)(pairs * key_tiles < slots ? pairs * key_tiles : slots)), dim3(SU_THREADS), (size_t)L::SMEM, stream, mq, mk, p);
}

}  // namespace

int attn_sums_launch(const AttnSumsParams& a, int sm_count, cudaStream_t stream) {
  if (a.D == 128) return launch_sums<128>(a, sm_count, stream);
  if (a.D == 64) return launch_sums<64>(a, sm_count, stream);
  return FLASHSVD_ERR_UNSUPPORTED_SHAPE;
}

}  // namespace fsvd
