// Attention weight that each key receives from the last queries of a
// sequence, without writing the probabilities:
//     weights[b, g, j] = sum_{h in group g} sum_{i in window, i >= j}
//                        2^(x_hij - lse_hi),   x = log2(e) scale q_hi . k_gj.
//
// Launch 1 (stats): lse_hi = log2 sum_{j <= i} 2^(x_hij).  A CTA takes 128
// query rows of one KV head (two runs of 64: consecutive ones of a head, or
// two heads of the group, which share the keys) and walks 128-key tiles:
// S = Q K^T on the tensor cores, one running (max, sum) per row and half
// tile.  With few row tiles the keys are split over CTAs and the CTA that
// finishes a row tile last joins the parts in split order.
// Launch 2 (sums): a CTA keeps 128 keys and walks the 64-row runs of
// queries that see them, S^T = K Q^T: a thread owns a key (half of a run's
// queries each) and adds up 2^(x - lse) in fp32, one partial sum a run.  No
// atomics: the order of every sum is fixed.
//
// The scores are computed twice (2 D flops each) because keeping them would
// write and read 4 bytes per (query, key, head).  Both launches are bound by
// the special-function unit (one exponential per score; 16 per clock and SM
// against 4096 multiply-adds, that is D = 128 scores in half the time).
// 96 KB of shared memory and 256 tensor-memory columns per CTA let two CTAs
// share an SM, so that one's waits are filled by the other.  Every wait is
// bounded.
#include <cstring>

#include "kernels.h"
#include "tc.cuh"

namespace fsvd {
namespace {

constexpr int SU_THREADS = 320;  // TMA warp, MMA warp, 8 softmax warps
constexpr int SU_RUN = 64;       // query rows of a run
constexpr int SU_KEYS = 128;     // keys of a tile

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct SuParams {
  const int* lens;
  float* weights;
  float* lse;        // [B][H][runs * 64]; +inf where there is no query
  float2* part;      // key splits: [B][G][row tiles][splits][128] (max, sum)
  int* counters;     // [B * G * row tiles], zero between launches
  int B, S, H, G, S_max, w_stride, window;
  int rep, runs;     // query heads per KV head; runs of the full window
  int row_tiles, splits;
  float scale_log2;
  int* status;
};

template <int D>
struct SuLayout {
  static constexpr int KB = D / 64;
  static constexpr int RUN_B = SU_RUN * 128;    // one [64 x 64] bf16 block, 8 KB
  static constexpr int KEY_B = SU_KEYS * 128;   // one [128 x 64] bf16 block, 16 KB
  // stats: the row tile, then a ring of key tiles
  static constexpr int KST = 2;
  static constexpr int ST_K = KB * KEY_B;
  static constexpr int ST_BAR = ST_K + KST * KB * KEY_B;
  // sums: the key tile, then a ring of runs and their lse
  static constexpr int QST = 4;
  static constexpr int SM_Q = KB * KEY_B;
  static constexpr int SM_LSE = SM_Q + QST * KB * RUN_B;
  static constexpr int SM_BAR = SM_LSE + QST * SU_RUN * 4;
  static constexpr int X_BYTES = 2 * 128 * 8;   // exchange between the two threads of a row
  static constexpr int ST_SMEM = 1024 + ST_BAR + 256 + X_BYTES;
  static constexpr int SM_SMEM = 1024 + SM_BAR + 256 + X_BYTES;
};

// Sequence geometry of one batch row.
struct SuRow {
  int n, lo;  // tokens, first query of the window
  __device__ SuRow(const SuParams& p, int b) {
    n = p.lens ? p.lens[b] : p.S;
    n = n < 0 ? 0 : (n > p.S ? p.S : n);
    lo = n > p.window ? n - p.window : 0;
  }
  __device__ int runs() const { return (n - lo + SU_RUN - 1) / SU_RUN; }
};

template <int D>
__global__ void __launch_bounds__(SU_THREADS, 2)
attn_stats_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ SuParams p) {
  using L = SuLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + L::ST_BAR);
  uint64_t* k_full = q_full + 1;           // [KST]
  uint64_t* k_empty = k_full + L::KST;     // [KST]
  uint64_t* s_full = k_empty + L::KST;     // [2]
  uint64_t* s_empty = s_full + 2;          // [2]
  uint64_t* drain = s_empty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* s_last = reinterpret_cast<int*>(tmem_holder + 2);
  float2* xch = reinterpret_cast<float2*>(smem + L::ST_BAR + 256);  // [2][128]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    tc::mbar_init(q_full, 1);
    for (int i = 0; i < L::KST; ++i) { tc::mbar_init(k_full + i, 1); tc::mbar_init(k_empty + i, 1); }
    for (int i = 0; i < 2; ++i) { tc::mbar_init(s_full + i, 1); tc::mbar_init(s_empty + i, 8); }
    tc::mbar_init(drain, 1);
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_holder, 256);
    tc::tmem_relinquish();
    tc::fence_before_sync();
  }
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_holder;

  // (tensor memory is held before dependents may start: a dependent kernel
  // that took it first would wait for this one, and this one for it)
  pdl_launch_dependents();
  pdl_wait();

  // item: row tiles from the last (longest) to the first, then pairs, splits
  const int sp = blockIdx.x % p.splits;
  int rest = blockIdx.x / p.splits;
  const int pair = rest % (p.B * p.G);
  const int tile = p.row_tiles - 1 - rest / (p.B * p.G);
  const int b = pair / p.G, g = pair - b * p.G;
  const SuRow R(p, b);
  const int n_runs = R.runs() * p.rep;     // (run, head) in run-major order
  const int r0 = 2 * tile, r1 = 2 * tile + 1;
  float* lse_g = p.lse + (long long)(b * p.H + g * p.rep) * p.runs * SU_RUN;
  auto run_of = [&](int r) { return r / p.rep; };
  auto head_of = [&](int r) { return r % p.rep; };
  const bool active = r0 < n_runs;
  const bool two = r1 < n_runs;
  const int last_q = min(R.n - 1, R.lo + (run_of(two ? r1 : r0) + 1) * SU_RUN - 1);
  const int nt = last_q / SU_KEYS + 1;
  const int t0 = (int)((long long)sp * nt / p.splits);
  const int t1 = active ? (int)((long long)(sp + 1) * nt / p.splits) : t0;


  if (warp == 0) {
    if (lane == 0 && t1 > t0) {
      tc::mbar_expect_tx(q_full, (two ? 2 : 1) * L::KB * L::RUN_B);
      for (int i = 0; i < (two ? 2 : 1); ++i) {
        const int r = r0 + i;
        for (int kb = 0; kb < L::KB; ++kb)
          tc::tma_load_2d(smem + kb * L::KEY_B + i * L::RUN_B, &tmQ, q_full, (g * p.rep + head_of(r)) * D + 64 * kb,
                          b * p.S + R.lo + run_of(r) * SU_RUN);
      }
      for (int j = t0; j < t1; ++j) {
        const int k = j - t0, st = k % L::KST;
        if (!tc::mbar_wait(k_empty + st, ((uint32_t)(k / L::KST) & 1u) ^ 1u, abort_flag, p.status)) break;
        tc::mbar_expect_tx(k_full + st, L::KB * L::KEY_B);
        for (int kb = 0; kb < L::KB; ++kb)
          tc::tma_load_2d(smem + L::ST_K + (st * L::KB + kb) * L::KEY_B, &tmK, k_full + st, g * D + 64 * kb,
                          b * p.S_max + j * SU_KEYS);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && t1 > t0) {
      constexpr uint32_t IDESC = tc::idesc_bf16(SU_KEYS, false);
      const uint32_t sq = tc::smem_u32(smem);
      bool ok = tc::mbar_wait(q_full, 0, abort_flag, p.status);
      for (int k = 0; k < t1 - t0 && ok; ++k) {
        const int st = k % L::KST, sb = k & 1;
        if (!(ok = tc::mbar_wait(k_full + st, (uint32_t)(k / L::KST) & 1u, abort_flag, p.status))) break;
        if (!(ok = tc::mbar_wait(s_empty + sb, ((uint32_t)(k >> 1) & 1u) ^ 1u, abort_flag, p.status))) break;
        tc::fence_after_sync();
        const uint32_t sk = tc::smem_u32(smem + L::ST_K + st * L::KB * L::KEY_B);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t ad = tc::sdesc_sw128(sq + (kk >> 2) * L::KEY_B + (kk & 3) * 32, 16, 1024);
          const uint64_t bd = tc::sdesc_sw128(sk + (kk >> 2) * L::KEY_B + (kk & 3) * 32, 16, 1024);
          tc::mma_bf16(tmem + sb * SU_KEYS, ad, bd, IDESC, kk > 0 ? 1u : 0u);
        }
        tc::mma_commit(s_full + sb);
        tc::mma_commit(k_empty + st);
      }
      tc::mma_commit(drain);
      const long long c0 = clock64();
      while (!tc::mbar_try_wait(drain, 0) && clock64() - c0 < tc::kWaitCycles) {}
    }
  } else if (active) {
    const int quad = warp & 3, hf = (warp - 2) >> 2;
    const int row = quad * 32 + lane;
    const int r = r0 + (row >> 6);
    const int q = R.lo + run_of(r) * SU_RUN + (row & 63);  // query position
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const float sc = p.scale_log2;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int k = 0; k < t1 - t0; ++k) {
      const int sb = k & 1, key0 = (t0 + k) * SU_KEYS + hf * 64;
      ok = ok && __all_sync(0xffffffffu, tc::mbar_wait(s_full + sb, (uint32_t)(k >> 1) & 1u, abort_flag, p.status));
      float s[64];
      if (ok) {
        tc::fence_after_sync();
        tc::tmem_ld32(tmem + lane_base + sb * SU_KEYS + hf * 64, reinterpret_cast<uint32_t*>(s));
        tc::tmem_ld32(tmem + lane_base + sb * SU_KEYS + hf * 64 + 32, reinterpret_cast<uint32_t*>(s + 32));
        tc::tmem_ld_wait();
        tc::reg_fence<64>(s);
      } else {
#pragma unroll
        for (int c = 0; c < 64; ++c) s[c] = -INFINITY;
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(s_empty + sb);
      if (key0 + 63 > q) {
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (key0 + c > q) s[c] = -INFINITY;
      }
      float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 64; ++c) mx4[c & 3] = fmaxf(mx4[c & 3], s[c]);
      const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sc;
      if (mx > m) {
        l *= ex2f(m - mx);
        m = mx;
      }
      const float e = m == -INFINITY ? 0.f : -m;
      float a4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 64; ++c) a4[c & 3] += ex2f(fmaf(s[c], sc, e));
      l += (a4[0] + a4[1]) + (a4[2] + a4[3]);
    }
    xch[hf * 128 + row] = make_float2(m, l);
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (hf == 0) {
      const float2 o = xch[128 + row];
      const float M = fmaxf(m, o.x);
      const float e = M == -INFINITY ? 0.f : M;
      const float sum = l * ex2f(m - e) + o.y * ex2f(o.x - e);
      if (p.splits == 1) {
        if (r < n_runs)
          lse_g[(long long)head_of(r) * p.runs * SU_RUN + run_of(r) * SU_RUN + (row & 63)] =
              q < R.n ? M + log2f(sum) : INFINITY;
      } else {
        __stcg(p.part + (((long long)pair * p.row_tiles + tile) * p.splits + sp) * 128 + row, make_float2(M, sum));
      }
    }
    if (p.splits > 1) {
      __threadfence();
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (threadIdx.x == 64) {
        int* cnt = p.counters + (long long)pair * p.row_tiles + tile;
        const int old = atomicAdd(cnt, 1);
        *s_last = old == p.splits - 1;
        if (old == p.splits - 1) *cnt = 0;
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (*s_last && hf == 0 && r < n_runs) {
        __threadfence();
        const float2* src = p.part + ((long long)pair * p.row_tiles + tile) * p.splits * 128 + row;
        float M = -INFINITY;
        for (int i = 0; i < p.splits; ++i) M = fmaxf(M, __ldcg(src + i * 128).x);
        const float e = M == -INFINITY ? 0.f : M;
        float sum = 0.f;
        for (int i = 0; i < p.splits; ++i) {
          const float2 o = __ldcg(src + i * 128);
          sum += o.y * ex2f(o.x - e);
        }
        lse_g[(long long)head_of(r) * p.runs * SU_RUN + run_of(r) * SU_RUN + (row & 63)] =
            q < R.n ? M + log2f(sum) : INFINITY;
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (*abort_flag && warp == 0 && lane == 0) {
    // let copies still in flight land before shared memory is released
    const long long c0 = clock64();
    while (clock64() - c0 < 2000000) {}
  }
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 256);
  }
}

template <int D>
__global__ void __launch_bounds__(SU_THREADS, 2)
attn_sums_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ SuParams p) {
  using L = SuLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + L::SM_BAR);
  uint64_t* q_full = k_full + 1;           // [QST]
  uint64_t* q_empty = q_full + L::QST;     // [QST] the MMA and the 8 softmax warps
  uint64_t* s_full = q_empty + L::QST;     // [4]
  uint64_t* s_empty = s_full + 4;          // [4]
  uint64_t* drain = s_empty + 4;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  float* xch = reinterpret_cast<float*>(smem + L::SM_BAR + 256);  // [128]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    tc::mbar_init(k_full, 1);
    for (int i = 0; i < L::QST; ++i) { tc::mbar_init(q_full + i, 1); tc::mbar_init(q_empty + i, 9); }
    for (int i = 0; i < 4; ++i) { tc::mbar_init(s_full + i, 1); tc::mbar_init(s_empty + i, 8); }
    tc::mbar_init(drain, 1);
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_holder, 256);
    tc::tmem_relinquish();
    tc::fence_before_sync();
  }
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_holder;

  pdl_launch_dependents();  // tensor memory is held (see attn_stats_kernel)
  pdl_wait();

  const int pair = blockIdx.x % (p.B * p.G), kt = blockIdx.x / (p.B * p.G);
  const int b = pair / p.G, g = pair - b * p.G;
  const SuRow R(p, b);
  const int key0 = kt * SU_KEYS;
  const int run0 = key0 > R.lo ? (key0 - R.lo) / SU_RUN : 0;  // first run that sees a key
  const int items = key0 < R.n ? (R.runs() - run0) * p.rep : 0;  // (run, head), run-major
  const float* lse_g = p.lse + (long long)(b * p.H + g * p.rep) * p.runs * SU_RUN;


  if (warp == 0) {
    if (lane == 0 && items > 0) {
      tc::mbar_expect_tx(k_full, L::KB * L::KEY_B);
      for (int kb = 0; kb < L::KB; ++kb)
        tc::tma_load_2d(smem + kb * L::KEY_B, &tmK, k_full, g * D + 64 * kb, b * p.S_max + key0);
      for (int k = 0; k < items; ++k) {
        const int st = k % L::QST, run = run0 + k / p.rep, h = k % p.rep;
        if (!tc::mbar_wait(q_empty + st, ((uint32_t)(k / L::QST) & 1u) ^ 1u, abort_flag, p.status)) break;
        tc::mbar_expect_tx(q_full + st, L::KB * L::RUN_B + SU_RUN * 4);
        for (int kb = 0; kb < L::KB; ++kb)
          tc::tma_load_2d(smem + L::SM_Q + (st * L::KB + kb) * L::RUN_B, &tmQ, q_full + st,
                          (g * p.rep + h) * D + 64 * kb, b * p.S + R.lo + run * SU_RUN);
        const float* src = lse_g + (long long)h * p.runs * SU_RUN + run * SU_RUN;
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                tc::smem_u32(smem + L::SM_LSE + st * SU_RUN * 4)),
            "l"(src), "r"(SU_RUN * 4), "r"(tc::smem_u32(q_full + st))
            : "memory");
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && items > 0) {
      constexpr uint32_t IDESC = tc::idesc_bf16(SU_RUN, false);
      const uint32_t sk = tc::smem_u32(smem);
      bool ok = tc::mbar_wait(k_full, 0, abort_flag, p.status);
      for (int k = 0; k < items && ok; ++k) {
        const int st = k % L::QST, sb = k & 3;
        if (!(ok = tc::mbar_wait(q_full + st, (uint32_t)(k / L::QST) & 1u, abort_flag, p.status))) break;
        if (!(ok = tc::mbar_wait(s_empty + sb, ((uint32_t)(k >> 2) & 1u) ^ 1u, abort_flag, p.status))) break;
        tc::fence_after_sync();
        const uint32_t sq = tc::smem_u32(smem + L::SM_Q + st * L::KB * L::RUN_B);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t ad = tc::sdesc_sw128(sk + (kk >> 2) * L::KEY_B + (kk & 3) * 32, 16, 1024);
          const uint64_t bd = tc::sdesc_sw128(sq + (kk >> 2) * L::RUN_B + (kk & 3) * 32, 16, 1024);
          tc::mma_bf16(tmem + sb * SU_RUN, ad, bd, IDESC, kk > 0 ? 1u : 0u);
        }
        tc::mma_commit(s_full + sb);
        tc::mma_commit(q_empty + st);
      }
      tc::mma_commit(drain);
      const long long c0 = clock64();
      while (!tc::mbar_try_wait(drain, 0) && clock64() - c0 < tc::kWaitCycles) {}
    }
  } else {
    const int quad = warp & 3, hf = (warp - 2) >> 2;
    const int row = quad * 32 + lane, key = key0 + row;
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const float sc = p.scale_log2;
    float total = 0.f;
    bool ok = true;
    for (int k = 0; k < items; ++k) {
      const int st = k % L::QST, sb = k & 3;
      const int q0 = R.lo + (run0 + k / p.rep) * SU_RUN + hf * 32;  // position of column 0
      ok = ok && __all_sync(0xffffffffu, tc::mbar_wait(q_full + st, (uint32_t)(k / L::QST) & 1u, abort_flag, p.status));
      ok = ok && __all_sync(0xffffffffu, tc::mbar_wait(s_full + sb, (uint32_t)(k >> 2) & 1u, abort_flag, p.status));
      float s[32], e[32];
      if (ok) {
        tc::fence_after_sync();
        tc::tmem_ld32(tmem + lane_base + sb * SU_RUN + hf * 32, reinterpret_cast<uint32_t*>(s));
        const float4* ls = reinterpret_cast<const float4*>(smem + L::SM_LSE + st * SU_RUN * 4) + hf * 8;
#pragma unroll
        for (int c = 0; c < 8; ++c) *reinterpret_cast<float4*>(e + 4 * c) = ls[c];
        tc::tmem_ld_wait();
        tc::reg_fence<32>(s);
      } else {
#pragma unroll
        for (int c = 0; c < 32; ++c) s[c] = e[c] = 0.f;
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) { tc::mbar_arrive(s_empty + sb); tc::mbar_arrive(q_empty + st); }
      if (q0 < key0 + SU_KEYS || q0 + 32 > R.n) {
        // queries before the key, and rows behind the sequence (whatever they hold)
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (q0 + c < key || q0 + c >= R.n) { s[c] = -INFINITY; e[c] = 0.f; }
      }
      float a4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 32; ++c) a4[c & 3] += ex2f(fmaf(s[c], sc, -e[c]));
      total += (a4[0] + a4[1]) + (a4[2] + a4[3]);
    }
    if (hf == 1) xch[row] = total;
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (hf == 0 && ok && key < R.n) p.weights[(long long)pair * p.w_stride + key] = total + xch[row];
  }
  tc::fence_before_sync();
  __syncthreads();
  if (*abort_flag && warp == 0 && lane == 0) {
    const long long c0 = clock64();
    while (clock64() - c0 < 2000000) {}
  }
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 256);
  }
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
  // Split the keys of a row tile until there are about two CTAs per SM slot.
  const long long tiles = pairs * p.row_tiles;
  long long splits = tiles > 0 ? (4LL * sm_count) / tiles : 1;
  splits = splits < 1 ? 1 : (splits > key_tiles ? key_tiles : splits);
  if (tiles > a.counters_cap) splits = 1;
  p.splits = (int)splits;
  const long long lse = heads * p.runs * SU_RUN;
  const long long part = splits > 1 ? tiles * splits * 128 * 2 : 0;
  if (lse + part > a.ws_cap || tiles * splits > 0x7fffffffLL || pairs * key_tiles > 0x7fffffffLL)
    return FLASHSVD_ERR_UNSUPPORTED_SHAPE;
  p.lse = a.ws;
  p.part = reinterpret_cast<float2*>(a.ws + lse);
  p.counters = a.counters;
  CUtensorMap mq, mk_s, mk;
  const long long HD = (long long)a.H * D, GD = (long long)a.G * D;
  FSVD_TRY(encode_map(&mq, a.q, (long long)a.B * a.S, HD, HD, 64, SU_RUN, true));
  FSVD_TRY(encode_map(&mk, a.k, (long long)a.B * a.S_max, GD, GD, 64, SU_KEYS, true));
  mk_s = mk;
  auto k1 = attn_stats_kernel<D>;
  auto k2 = attn_sums_kernel<D>;
  static SmemAttrOnce once1, once2;
  FSVD_TRY(set_smem_once(once1, k1, L::ST_SMEM));
  FSVD_TRY(set_smem_once(once2, k2, L::SM_SMEM));
  const double pq = (double)p.window * a.S - 0.5 * (double)p.window * p.window;  // visible pairs
  const double bytes = 2.0 * D * a.B * ((double)p.window * a.H + (double)a.S * a.G);
  const LaunchTag t1{"attn_stats", bytes + 4.0 * lse, 2.0 * D * heads * pq};
  const LaunchTag t2{"attn_sums", bytes + 4.0 * lse + 4.0 * pairs * a.S, 2.0 * D * heads * pq};
  FSVD_TRY(launch_pdl(t1, k1, dim3((unsigned)(tiles * splits)), dim3(SU_THREADS), (size_t)L::ST_SMEM, stream, mq, mk_s, p));
  return launch_pdl(t2, k2, dim3((unsigned)(pairs * key_tiles)), dim3(SU_THREADS), (size_t)L::SM_SMEM, stream, mq, mk, p);
}

}  // namespace

int attn_sums_launch(const AttnSumsParams& a, int sm_count, cudaStream_t stream) {
  if (a.D == 128) return launch_sums<128>(a, sm_count, stream);
  if (a.D == 64) return launch_sums<64>(a, sm_count, stream);
  return FLASHSVD_ERR_UNSUPPORTED_SHAPE;
}

}  // namespace fsvd
