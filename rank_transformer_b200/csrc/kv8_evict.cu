// Eviction from the 8-bit cache by accumulated attention weight.
//
// Launch 1 (select): per (batch row, KV head) with n > keep tokens, the
// keep - recent largest weights of the first n - recent tokens (ties to the
// lower index) by a radix selection on the weights' ordered bit patterns,
// and the kept indices in ascending order.  The weights are read once, into
// registers; long rows are cut over a cluster.  Launch 2 (move): one CTA
// per kept 64-token block gathers its rows into registers, finds their new
// scale and writes codes, scale, weights and, for the newest block, the tail.
//
// 4 rows x 8 heads of 131072 tokens down to 32768 take 139 us against 86 for
// the bytes: about 30 for the selection (7 until the weights are there, 5 to 6
// for each of three rounds of counting, summing over the cluster and picking
// the digit, the rest counting again and writing the indices), 109 for the
// moves, whose rows of 128 bytes lie scattered: 4.9 TB/s.  With 2, 3, 4 and
// (spilling) 5 CTAs an SM the whole took 190, 160, 140 and 148 us; rows copied
// to shared memory an item ahead 138, with numbers and indices two items ahead
// 161; only codes held in registers, decoded twice, 5 CTAs 137; stores that
// leave the L2 first 135 to 138, and what reads the cache next would miss.
// 2048 tokens of 32 heads down to 1024: 12.4 us, two launches of a few us.
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

constexpr int EV_SEL_THREADS = 512;
constexpr int EV_SEL_STRETCH = 4096;  // weights per CTA of a selection,
constexpr int EV_SEL_CTAS = 8;        // up to so many CTAs a pair
constexpr int EV_BINS = 2048;
constexpr int EV_THREADS = 256;
constexpr int EV_CTAS = 4;              // CTAs per SM (64 registers a thread)

struct EvParams {
  Kv8 src, dst;
  const float* w_in; float* w_out;
  const int* n_in; int* n_out;
  int* kept;
  int keep, recent, in_place, nblk;  // nblk: blocks of `keep` tokens
  int sel_ctas;                      // CTAs per pair of the selection
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

// Exclusive sum over the threads of the block (by thread index, or from the
// last thread down) and the sum of all; s: one word a warp of shared memory.
template <bool FROM_TOP>
__device__ __forceinline__ uint32_t block_before(uint32_t v, uint32_t* s, int lane, int warp, uint32_t* total) {
  constexpr int WARPS = EV_SEL_THREADS / 32;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = FROM_TOP ? __shfl_down_sync(0xffffffffu, x, o) : __shfl_up_sync(0xffffffffu, x, o);
    if (FROM_TOP ? lane + o < 32 : lane >= o) x += y;
  }
  if (lane == (FROM_TOP ? 0 : 31)) s[warp] = x;
  __syncthreads();
  const uint32_t w = lane < WARPS ? s[lane] : 0u;
  *total = __reduce_add_sync(0xffffffffu, w);
  return __reduce_add_sync(0xffffffffu, (FROM_TOP ? lane > warp : lane < warp) ? w : 0u) + x - v;
}

__device__ __forceinline__ uint2 ld_cluster2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_cluster4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ void st_cluster4(uint32_t addr, uint4 v) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// A cluster of `ctas` CTAs per pair, each with one stretch of the weights;
// every thread keeps KPT consecutive ones in registers (a stretch longer than
// a CTA's threads hold is walked in tiles, read again each time).  Three
// passes over 11, 11 and 10 bits of the keys narrow down the hk-th largest
// key: every CTA counts its stretch's digits, and adds up the counts of all
// of them through distributed shared memory.  Then the kept indices are
// written in order, at the sum of the counts before them.
template <int KPT>
__global__ void __launch_bounds__(EV_SEL_THREADS, 2)
kv8_select_kernel(const __grid_constant__ EvParams p) {
  constexpr int TILE = EV_SEL_THREADS * KPT, BPT = EV_BINS / EV_SEL_THREADS;
  static_assert(BPT == 4, "four digits a thread");
  // the digits' counts of the stretch, a share of all, the sums; then kept offsets
  __shared__ uint4 s_buf[4 * EV_SEL_THREADS];
  static_assert(TILE * 2 <= sizeof(s_buf) && EV_BINS * 4 <= EV_SEL_THREADS * 16, "room of s_buf");
  uint32_t* hist = reinterpret_cast<uint32_t*>(s_buf);
  uint4* s_share = s_buf + EV_SEL_THREADS;
  uint4* s_all = s_buf + 2 * EV_SEL_THREADS;
  __shared__ uint32_t s_scan[EV_SEL_THREADS / 32], s_res[2];
  __shared__ __align__(8) uint32_t s_tot[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = p.sel_ctas, rank = blockIdx.x % ctas;
  const int pair = blockIdx.x / ctas, b = pair / p.src.G;

  pdl_launch_dependents();
  pdl_wait();

  const int t0 = rank * EV_SEL_THREADS + tid, step = ctas * EV_SEL_THREADS;
  for (int i = t0; i < p.nblk; i += step) p.flags[(long long)pair * p.nblk + i] = 0;
  if (blockIdx.x == 0 && tid == 0) *p.ticket = 0;
  int n = p.n_in[b];
  n = n < 0 ? 0 : (n > p.src.S_max ? p.src.S_max : n);
  if (rank == 0 && tid == 0) p.n_ws[pair] = n;
  int* kept = p.kept + (long long)pair * p.keep;
  if (n <= p.keep) {
    for (int i = t0; i < p.keep; i += step) kept[i] = i < n ? i : -1;
    return;
  }
  const int c = n - p.recent, hk = p.keep - p.recent;
  for (int i = t0; i < p.recent; i += step) kept[hk + i] = c + i;
  if (hk == 0) return;

  // this CTA's stretch [first, first + len), a multiple of four long but for the last
  const int chunk = ((c + ctas - 1) / ctas + 3) & ~3;
  const int first = rank * chunk, len = max(0, min(chunk, c - first));
  const int tiles = (chunk + TILE - 1) / TILE;
  const float* w = p.w_in + (long long)pair * p.src.S_max + first;
  uint32_t keys[KPT];
  int have = 0;  // keys of this thread
  auto load = [&](int tile) {
    const int i0 = tile * TILE + tid * KPT;
    have = max(0, min(KPT, len - i0));
#pragma unroll
    for (int k = 0; k < KPT; k += 4)
      if (k < have) {  // (rows are padded to 64 weights)
        const float4 v = *reinterpret_cast<const float4*>(w + i0 + k);
        keys[k] = order_key(v.x); keys[k + 1] = order_key(v.y);
        keys[k + 2] = order_key(v.z); keys[k + 3] = order_key(v.w);
      }
  };
  load(0);

  uint32_t prefix = 0, need = hk, total;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    *reinterpret_cast<uint4*>(hist + BPT * tid) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    for (int tile = 0; tile < tiles; ++tile) {
      if (tiles > 1) load(tile);
#pragma unroll
      for (int k = 0; k < KPT; ++k)
        if (k < have && (pass == 0 || (keys[k] >> (shift + bits)) == prefix))
          atomicAdd(&hist[(keys[k] >> shift) & ((1u << bits) - 1u)], 1u);
    }
    if (ctas > 1) tc::cluster_sync(); else __syncthreads();
    if (ctas > 1) {
      // Each CTA adds up its share of the digits (of four) and hands the sums
      // to all: one load and one store a thread, about a microsecond each
      // (every CTA reading all the counts took eight loads and 5 us).
      const int per = EV_SEL_THREADS / ctas, r = tid / per, q = tid - r * per;
      s_share[tid] = ld_cluster4(tc::mapa_shared(tc::smem_u32(hist) + 16 * (rank * per + q), r));
      __syncthreads();
      uint4 v = make_uint4(0, 0, 0, 0);
      for (int k = 0; k < ctas; ++k) {
        const uint4 o = s_share[k * per + q];
        v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
      }
      st_cluster4(tc::mapa_shared(tc::smem_u32(s_all) + 16 * (rank * per + q), r), v);
      tc::cluster_sync();
    }
    const uint4 counts = ctas > 1 ? s_all[tid] : *reinterpret_cast<const uint4*>(hist + BPT * tid);
    const uint32_t d[BPT] = {counts.x, counts.y, counts.z, counts.w};  // of digits 4 tid .. + 3
    const uint32_t sum = d[0] + d[1] + d[2] + d[3];
    uint32_t above = block_before<true>(sum, s_scan, lane, warp, &total);
    if (above < need && above + sum >= need) {
#pragma unroll
      for (int k = BPT - 1; k >= 0; --k) {
        if (above < need && above + d[k] >= need) {
          s_res[0] = (prefix << bits) | (uint32_t)(BPT * tid + k);
          s_res[1] = need - above;
        }
        above += d[k];
      }
    }
    __syncthreads();  // (the others' next sums come after the next cluster barrier)
    prefix = s_res[0];
    need = s_res[1];
  }

  // every key above `prefix`, and the first `need` equal to it
  uint32_t before = 0;
  auto count = [&]() {  // those of the tile in the threads before: above, and equal << 16 (a tile holds under 2^16 keys)
    uint32_t mine = 0;
#pragma unroll
    for (int k = 0; k < KPT; ++k)
      if (k < have) mine += keys[k] > prefix ? 1u : keys[k] == prefix ? 0x10000u : 0u;
    before = block_before<false>(mine, s_scan, lane, warp, &total);
  };
  uint32_t g = 0, e = 0;  // of those, in the stretches and tiles before
  if (ctas > 1) {
    uint32_t tg = 0, te = 0;
    for (int tile = 0; tile < tiles; ++tile) {
      if (tiles > 1) load(tile);
      count();
      __syncthreads();
      tg += total & 0xffffu; te += total >> 16;
    }
    if (tid == 0) { s_tot[0] = tg; s_tot[1] = te; }
    tc::cluster_sync();
    const uint2 t = lane < rank ? ld_cluster2(tc::mapa_shared(tc::smem_u32(s_tot), lane)) : make_uint2(0, 0);
    g = __reduce_add_sync(0xffffffffu, t.x);
    e = __reduce_add_sync(0xffffffffu, t.y);
    tc::cluster_sync();  // (no CTA leaves while its counts may be read)
  }
  // A tile's kept offsets go to shared memory first and from there in order
  // (written at once, each thread's to its own place, they took 10 us).
  uint16_t* s_off = reinterpret_cast<uint16_t*>(s_buf);
  for (int tile = 0; tile < tiles; ++tile) {
    if (tiles > 1) load(tile);
    if (tiles > 1 || ctas == 1) count();
    const uint32_t base = g + min(e, need);
    uint32_t gk = g + (before & 0xffffu), ek = e + (before >> 16);
#pragma unroll
    for (int k = 0; k < KPT; ++k)
      if (k < have) {
        const bool gt = keys[k] > prefix, eq = keys[k] == prefix;
        if (gt || (eq && ek < need)) s_off[gk + min(ek, need) - base] = (uint16_t)(tid * KPT + k);
        gk += gt;
        ek += eq;
      }
    g += total & 0xffffu;
    e += total >> 16;
    __syncthreads();
    const int at = first + tile * TILE, found = (int)(g + min(e, need) - base);
    for (int i = tid; i < found; i += EV_SEL_THREADS) kept[base + i] = at + s_off[i];
    __syncthreads();
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(EV_THREADS, EV_CTAS)
kv8_move_kernel(const __grid_constant__ EvParams p) {
  constexpr int UPR = D / 16;                 // units of 16 elements per row
  constexpr int PER = KV8_BLOCK * UPR / 128;  // units per thread; 128 threads per tensor
  __shared__ int s_idx[KV8_BLOCK];
  __shared__ uint32_t s_max[EV_THREADS / 32];
  __shared__ int s_next, s_ok;
  const int tid = threadIdx.x, x = tid >> 7, t = tid & 127;
  const int items = p.src.B * p.src.G * p.nblk;

  pdl_launch_dependents();
  pdl_wait();

  // Items come from a counter, each CTA one ahead: while an item's rows are
  // on their way, the next item's number and indices are fetched.
  if (tid == 0) { s_next = atomicAdd(p.ticket, 1); s_ok = 1; }
  __syncthreads();
  int item = s_next, idx = -1, n = 0;
  auto fetch = [&]() {
    if (item >= items) return;
    const int pair = item / p.nblk, row = (item - pair * p.nblk) * KV8_BLOCK + tid;
    n = p.n_ws[pair];
    if (tid < KV8_BLOCK) idx = row < p.keep ? p.kept[(long long)pair * p.keep + row] : -1;
  };
  fetch();
  while (item < items) {
    const int pair = item / p.nblk, i = item - pair * p.nblk;
    const int m = min(n, p.keep), row0 = i * KV8_BLOCK, rows = min(KV8_BLOCK, m - row0);
    const bool moves = rows > 0 && !(p.in_place && n <= p.keep);
    if (tid < KV8_BLOCK) s_idx[tid] = idx;
    __syncthreads();  // s_idx written; s_next read by all
    if (tid == 0) {
      s_next = atomicAdd(p.ticket, 1);
      if (i == 0 && pair % p.src.G == 0 && p.n_out) p.n_out[pair / p.src.G] = m;
    }

    // ---- load the rows and the weights ----
    // `codes_only`: every row comes from codes and goes to codes.  The rows
    // then stay half-precision codes: the new code is the old one times a
    // power of two, rounded, in one or two instructions a pair.  Otherwise
    // (the source's newest block, which is in its tail, or the destination's)
    // they become bf16.  (All of them as bf16 took 12 instructions an element
    // and bound the kernel: 132 us, then 111, for 32 x 32768 rows of 128.)
    const int last = (n - 1) / KV8_BLOCK;  // the source's newest block: in its tail
    const bool codes_only = row0 + KV8_BLOCK < m && s_idx[KV8_BLOCK - 1] / KV8_BLOCK < last;
    uint4 a[PER], c[PER];
    float sc[PER];
    float wv = 0.f;
    if (moves) {
      const uint8_t* codes = p.src.codes[x] + (long long)pair * p.src.S_max * D;
      const float* scale = p.src.scale[x] + (long long)pair * (p.src.S_max / KV8_BLOCK);
      const bf16* stail = p.src.tail[x] + (long long)pair * KV8_BLOCK * D;
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int u = t + 128 * k, r = s_idx[u / UPR], col = (u % UPR) * 16;
        a[k] = c[k] = make_uint4(0, 0, 0, 0);
        sc[k] = -1.f;  // bf16 already
        if (r >= 0 && (int)((uint32_t)r / KV8_BLOCK) == last) {
          a[k] = ld_once(stail + (r % KV8_BLOCK) * D + col);
          c[k] = ld_once(stail + (r % KV8_BLOCK) * D + col + 8);
        } else if (r >= 0) {
          a[k] = ld_once(codes + (long long)r * D + col);
          sc[k] = scale[(uint32_t)r / KV8_BLOCK];
        }
      }
      if (tid < rows) wv = p.w_in[(long long)pair * p.src.S_max + s_idx[tid]];
      uint32_t mx = 0;
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        if (codes_only) {
          __half2 h[8], most;
          kv8_decode16h<E4M3>(a[k], h);
          most = __habs2(h[0]);
#pragma unroll
          for (int i = 1; i < 8; ++i) most = __hmax2(most, __habs2(h[i]));
          const float top = fmaxf(__low2float(most), __high2float(most)) * sc[k];  // exact; NaN stays
          mx = max(mx, __float_as_uint(top) >> 16);
          memcpy(&a[k], h, 16);
          memcpy(&c[k], h + 4, 16);
        } else {
          if (!(sc[k] < 0.f)) kv8_decode16<E4M3>(a[k], sc[k], a[k], c[k]);  // (a NaN scale too)
          mx = max(mx, max(amax8(a[k]), amax8(c[k])));
        }
      }
      mx = __reduce_max_sync(0xffffffffu, mx);
      if ((tid & 31) == 0) s_max[tid >> 5] = mx;
    }
    __syncthreads();
    item = s_next;
    const int n_cur = n;
    fetch();
    if (!moves) continue;

    if (p.in_place) {
      int* flags = p.flags + (long long)pair * p.nblk;
      const int* kept = p.kept + (long long)pair * p.keep;
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
      const uint32_t mx = max(max(s_max[4 * x], s_max[4 * x + 1]), max(s_max[4 * x + 2], s_max[4 * x + 3]));
      const int e = kv8_exponent<E4M3>(mx);
      const bool fin = kv8_finite(mx);
      uint8_t* dst = p.dst.codes[x] + ((long long)pair * p.dst.S_max + row0) * D;
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        uint4 o;
        if (codes_only) {
          __half2 h[8];
          memcpy(h, &a[k], 16);
          memcpy(h + 4, &c[k], 16);
          o = fin ? kv8_rescale16<E4M3>(h, (int)(__float_as_uint(sc[k]) >> 23) - 127 - e) : make_uint4(0, 0, 0, 0);
        } else {
          o = kv8_encode16<E4M3>(a[k], c[k], exp2i(-e), fin);
        }
        *reinterpret_cast<uint4*>(dst + (t + 128 * k) * 16) = o;
      }
      if (t == 0) p.dst.scale[x][(long long)pair * (p.dst.S_max / KV8_BLOCK) + i] = kv8_scale(e, fin);
    }
    if (row0 + KV8_BLOCK >= min(n_cur, p.keep)) {
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
}

}  // namespace

int kv8_evict_launch(const Kv8EvictParams& a, int sm_count, cudaStream_t stream) {
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
  p.sel_ctas = 1;
  while (p.sel_ctas < EV_SEL_CTAS && p.sel_ctas * EV_SEL_STRETCH < a.src.S_max) p.sel_ctas *= 2;
  // eight weights a thread cover the stretch, or (up to 131072 tokens) 32 do
  const bool small = (long long)p.sel_ctas * EV_SEL_STRETCH >= a.src.S_max;
  FSVD_TRY(launch_pdl_cluster(st, p.sel_ctas, small ? kv8_select_kernel<8> : kv8_select_kernel<32>,
                              dim3((unsigned)(pairs * p.sel_ctas)), dim3(EV_SEL_THREADS), 0, stream, p));
  const LaunchTag mt{"kv8_move", pairs * (double)a.keep * (4.0 * a.src.D + 12.0), 0.0};
  const long long most = (long long)sm_count * EV_CTAS;
  const dim3 grid((unsigned)(items < most ? items : most)), block(EV_THREADS);
  if (a.src.D == 128)
    return a.src.e4m3 ? launch_pdl(mt, kv8_move_kernel<128, true>, grid, block, 0, stream, p)
                      : launch_pdl(mt, kv8_move_kernel<128, false>, grid, block, 0, stream, p);
  if (a.src.D == 64)
    return a.src.e4m3 ? launch_pdl(mt, kv8_move_kernel<64, true>, grid, block, 0, stream, p)
                      : launch_pdl(mt, kv8_move_kernel<64, false>, grid, block, 0, stream, p);
  return FLASHSVD_ERR_UNSUPPORTED_SHAPE;
}

}  // namespace fsvd
