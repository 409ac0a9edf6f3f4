// Eviction from the 8-bit cache by accumulated attention weight.
//
// Launch 1 (select): per (batch row, KV head) with n > keep tokens, the
// keep - recent largest weights of the first n - recent tokens (ties to the
// lower index) by a radix selection on the weights' ordered bit patterns,
// then the kept indices in ascending order.  Launch 2 (move): one CTA per
// kept 64-token block gathers its rows into registers, finds their new
// scale and writes codes, scale, weights and, for the newest block, the tail.
//
// In place, a kept row moves to a lower or equal index, so a CTA may write
// block i only after the CTAs of lower blocks have loaded their rows from
// it: each CTA raises a flag when its rows are in registers, and the writer
// of block i waits for the flags of the blocks j < i whose rows reach into
// it.  CTAs take their blocks from a counter, so the ones waited for are
// always running already.  Every wait is bounded.
#include <cstring>

#include "kv8.cuh"
#include "tc.cuh"

namespace fsvd {
namespace {

constexpr int EV_SEL_THREADS = 1024;
constexpr int EV_THREADS = 256;

struct EvParams {
  Kv8 src, dst;
  const float* w_in; float* w_out;
  const int* n_in; int* n_out;
  int* kept;
  int keep, recent, in_place, nblk;  // nblk: blocks of `keep` tokens
  int* n_ws;                         // [B * G] token counts before eviction
  int* flags;                        // [B * G * nblk] rows loaded
  int* ticket;
  int* status;
};

// Bit pattern that orders as the weight does, NaN below everything and both
// zeros equal.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (isnan(w)) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(EV_SEL_THREADS)
kv8_select_kernel(const __grid_constant__ EvParams p) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t s_prefix, s_need;
  __shared__ uint32_t s_warp[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pair = blockIdx.x, b = pair / p.src.G;

  pdl_launch_dependents();
  pdl_wait();

  for (int i = tid; i < p.nblk; i += EV_SEL_THREADS) p.flags[(long long)pair * p.nblk + i] = 0;
  if (pair == 0 && tid == 0) *p.ticket = 0;
  int n = p.n_in[b];
  n = n < 0 ? 0 : (n > p.src.S_max ? p.src.S_max : n);
  if (tid == 0) p.n_ws[pair] = n;
  int* kept = p.kept + (long long)pair * p.keep;
  if (n <= p.keep) {
    for (int i = tid; i < p.keep; i += EV_SEL_THREADS) kept[i] = i < n ? i : -1;
    return;
  }
  const int c = n - p.recent, hk = p.keep - p.recent;
  for (int i = tid; i < p.recent; i += EV_SEL_THREADS) kept[hk + i] = c + i;
  if (hk == 0) return;
  const float* w = p.w_in + (long long)pair * p.src.S_max;

  // the hk-th largest key: one byte per pass, from the top
  uint32_t prefix = 0, need = hk;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < c; i += EV_SEL_THREADS) {
      const uint32_t k = order_key(w[i]);
      if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t above = 0;
      int d = 255;
      for (; d > 0 && above + hist[d] < need; --d) above += hist[d];
      s_prefix = (prefix << 8) | (uint32_t)d;
      s_need = need - above;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
    __syncthreads();
  }
  // in order: every key above it, and the first `need` equal to it
  uint32_t n_gt = 0, n_eq = 0;  // before this stretch
  for (int i0 = 0; i0 < c; i0 += EV_SEL_THREADS) {
    const int i = i0 + tid;
    const uint32_t k = i < c ? order_key(w[i]) : 0u;
    const bool gt = i < c && k > prefix, eq = i < c && k == prefix;
    const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) s_warp[warp] = (uint32_t)__popc(bg) | ((uint32_t)__popc(be) << 16);
    __syncthreads();
    uint32_t v = s_warp[lane], before = 0, total = 0;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    total = __shfl_sync(0xffffffffu, x, 31);
    before = __shfl_sync(0xffffffffu, x - v, warp);
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t g0 = n_gt + (before & 0xffffu) + __popc(bg & below);
    const uint32_t e0 = n_eq + (before >> 16) + __popc(be & below);
    if (gt || (eq && e0 < need)) kept[g0 + min(e0, need)] = i;
    n_gt += total & 0xffffu;
    n_eq += total >> 16;
    __syncthreads();
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(EV_THREADS)
kv8_move_kernel(const __grid_constant__ EvParams p) {
  constexpr int UPR = D / 16;                 // units of 16 elements per row
  constexpr int PER = KV8_BLOCK * UPR / 128;  // units per thread; 128 threads per tensor
  __shared__ int s_idx[KV8_BLOCK];
  __shared__ uint32_t s_max[EV_THREADS / 32];
  __shared__ int s_item, s_ok;
  const int tid = threadIdx.x, x = tid >> 7, t = tid & 127;

  pdl_launch_dependents();
  pdl_wait();

  if (tid == 0) { s_item = atomicAdd(p.ticket, 1); s_ok = 1; }
  __syncthreads();
  const int pair = s_item / p.nblk, i = s_item - pair * p.nblk;
  const int b = pair / p.src.G;
  const int n = p.n_ws[pair], m = min(n, p.keep);
  if (i == 0 && pair == b * p.src.G && tid == 0 && p.n_out) p.n_out[b] = m;
  const bool still = p.in_place && n <= p.keep;  // nothing moves
  const int row0 = i * KV8_BLOCK, rows = min(KV8_BLOCK, m - row0);
  if (still || rows <= 0) return;
  const int* kept = p.kept + (long long)pair * p.keep;
  if (tid < KV8_BLOCK) s_idx[tid] = tid < rows ? kept[row0 + tid] : -1;
  __syncthreads();

  // ---- load the rows as bf16 and the weights ----
  const int last = (n - 1) / KV8_BLOCK;  // the source's newest block: in its tail
  const uint8_t* codes = p.src.codes[x] + (long long)pair * p.src.S_max * D;
  const float* scale = p.src.scale[x] + (long long)pair * (p.src.S_max / KV8_BLOCK);
  const bf16* stail = p.src.tail[x] + (long long)pair * KV8_BLOCK * D;
  uint4 a[PER], c[PER];
  uint32_t mx = 0;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int u = t + 128 * k, r = s_idx[u / UPR], col = (u % UPR) * 16;
    a[k] = c[k] = make_uint4(0, 0, 0, 0);
    if (r >= 0) {
      if (r / KV8_BLOCK == last) {
        a[k] = ld_once(stail + (r % KV8_BLOCK) * D + col);
        c[k] = ld_once(stail + (r % KV8_BLOCK) * D + col + 8);
      } else {
        kv8_decode16<E4M3>(ld_once(codes + (long long)r * D + col), scale[r / KV8_BLOCK], a[k], c[k]);
      }
    }
  }
  float wv = 0.f;
  if (tid < rows) wv = p.w_in[(long long)pair * p.src.S_max + s_idx[tid]];
#pragma unroll
  for (int k = 0; k < PER; ++k) mx = max(mx, max(amax8(a[k]), amax8(c[k])));
  mx = __reduce_max_sync(0xffffffffu, mx);
  if ((tid & 31) == 0) s_max[tid >> 5] = mx;
  __syncthreads();

  if (p.in_place) {
    int* flags = p.flags + (long long)pair * p.nblk;
    if (tid == 0) {
      __threadfence();
      asm volatile("st.release.gpu.global.s32 [%0], 1;" ::"l"(flags + i) : "memory");
    }
    // blocks j < i whose last row lies in block i or beyond (the source's
    // newest block, whose rows the tail holds, is never below block i)
    if (tid < 32) {
      const long long t0 = clock64();
      for (int j = i - 1 - tid; j >= 0; j -= 32) {
        if (kept[j * KV8_BLOCK + KV8_BLOCK - 1] < row0) break;
        int v = 0;
        while (true) {
          asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(flags + j) : "memory");
          if (v) break;
          if (clock64() - t0 > tc::kWaitCycles) {
            atomicExch(p.status, DEV_STATUS_TIMEOUT);
            s_ok = 0;
            break;
          }
          __nanosleep(32);
        }
        if (!v) break;
      }
      __threadfence();
    }
    __syncthreads();
    if (!s_ok) return;
  }

  // ---- write ----
  if (tid < rows) p.w_out[(long long)pair * p.dst.S_max + row0 + tid] = wv;
  if (rows == KV8_BLOCK) {
    mx = max(max(s_max[4 * x], s_max[4 * x + 1]), max(s_max[4 * x + 2], s_max[4 * x + 3]));
    const int e = kv8_exponent<E4M3>(mx);
    const bool fin = kv8_finite(mx);
    uint8_t* dst = p.dst.codes[x] + ((long long)pair * p.dst.S_max + row0) * D;
#pragma unroll
    for (int k = 0; k < PER; ++k)
      *reinterpret_cast<uint4*>(dst + (t + 128 * k) * 16) = kv8_encode16<E4M3>(a[k], c[k], exp2i(-e), fin);
    if (t == 0) p.dst.scale[x][(long long)pair * (p.dst.S_max / KV8_BLOCK) + i] = kv8_scale(e, fin);
  }
  if (row0 + KV8_BLOCK >= m) {
    bf16* tail = p.dst.tail[x] + (long long)pair * KV8_BLOCK * D;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int u = t + 128 * k;
      if (u / UPR < rows) {
        *reinterpret_cast<uint4*>(tail + u * 16) = a[k];
        *reinterpret_cast<uint4*>(tail + u * 16 + 8) = c[k];
      }
    }
  }
}

}  // namespace

int kv8_evict_launch(const Kv8EvictParams& a, cudaStream_t stream) {
  EvParams p;
  memset(&p, 0, sizeof(p));
  p.src = a.src; p.dst = a.dst;
  p.w_in = a.w_in; p.w_out = a.w_out;
  p.n_in = a.n_in; p.n_out = a.n_out;
  p.kept = a.kept;
  p.keep = a.keep; p.recent = a.recent; p.in_place = a.in_place;
  p.nblk = ceil_div(a.keep, KV8_BLOCK);
  p.status = a.status;
  const long long pairs = (long long)a.src.B * a.src.G, items = pairs * p.nblk;
  if (items > 0x7fffffffLL || pairs + items + 4 > a.ws_cap) return FLASHSVD_ERR_UNSUPPORTED_SHAPE;
  p.ticket = a.ws;
  p.n_ws = a.ws + 4;
  p.flags = p.n_ws + pairs;
  const LaunchTag st{"kv8_select", 4.0 * pairs * ((double)a.src.S_max + a.keep), 0.0};
  FSVD_TRY(launch_pdl(st, kv8_select_kernel, dim3((unsigned)pairs), dim3(EV_SEL_THREADS), 0, stream, p));
  const LaunchTag mt{"kv8_move", pairs * (double)a.keep * (4.0 * a.src.D + 12.0), 0.0};
  const dim3 grid((unsigned)items), block(EV_THREADS);
  if (a.src.D == 128)
    return a.src.e4m3 ? launch_pdl(mt, kv8_move_kernel<128, true>, grid, block, 0, stream, p)
                      : launch_pdl(mt, kv8_move_kernel<128, false>, grid, block, 0, stream, p);
  if (a.src.D == 64)
    return a.src.e4m3 ? launch_pdl(mt, kv8_move_kernel<64, true>, grid, block, 0, stream, p)
                      : launch_pdl(mt, kv8_move_kernel<64, false>, grid, block, 0, stream, p);
  return FLASHSVD_ERR_UNSUPPORTED_SHAPE;
}

}  // namespace fsvd
