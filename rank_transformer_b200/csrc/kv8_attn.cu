// One decode step of attention over the 8-bit key/value cache.
//
// For query head h of KV head g, x_j = log2(e) scale q_h . k_j over the
// tokens j = 0..pos, and out_h = sum_j 2^(x_j - M) v_j / sum_j 2^(x_j - M).
// The codes are read once, with a running maximum m and sum l: the products
// run on the codes themselves (exact halves), the block's key scale goes
// into x_j and its value scale into the block's contribution to the output.
//
// Work split.  The blocks of all (batch row, KV head) pairs form one line of
// units, cut evenly over the CTAs whatever the lengths; a pair that spans
// several CTAs leaves partial (m, l, O) in the workspace, and the CTA that
// finishes the pair last joins them in CTA order (deterministic).  Within a
// CTA, warp w takes the 16-token slices w, w + 8, ... of its run of blocks
// and the warps are joined through shared memory.  Each warp keeps a ring of
// its own: it issues the TMA loads of its next slices (2 KB of keys, 2 KB of
// values at D = 128) and waits for nobody else.  The 128-byte swizzle and the
// order kappa of a slice's tokens keep every shared-memory read free of bank
// conflicts.  The newest block comes from the bf16 tail, 16 tokens a warp,
// with bf16 products (probabilities as a sum of two bf16, 16 bits); the new
// rows are appended, and a block they complete is quantised, by the same CTA.
//
// Matrix instructions: S^T = K Q^T and O^T = V^T P^T (m16n8k16, fp32 sums),
// so that the tokens and the head's dimensions fill the 16 rows and the up
// to 8 query heads of a KV head the 8 columns (two column tiles for 9-16).
// Rounding to fewer bits: the codes are exact in half precision, and so is q,
// scaled by a power of two that brings its largest element to 2^14, but for
// elements below 2^-31 of that one: they lose bits, at most 2^-39 of the
// largest.  The probabilities are rounded to half after scaling by 2^15, so
// that they keep 11 bits down to 2^-29 and vanish only below 2^-40 of the
// largest; l is summed from the unrounded ones.  (Against 64 bits the outputs
// are off by 1.6306e-3, 2048 tokens x 32 heads of 128; with fp32 probabilities
// by 1.6297e-3: the rounding to bf16.)
//
// Range.  O / l is at most the largest |v|, but O alone is up to n times as
// large.  The output sums carry 2^-K, 2^(K - 1) >= S_max (one more bit than n
// needs: rounding may take a probability a little over 1), through the value
// scales, and its inverse at the end: values up to the last bf16 number do not
// overflow.  Each addition may then be off by 2^(K - 149), which is below half
// a step of a bf16 output unless that is itself near 2^-126.  (K by capacity,
// a launch's constant: one by the pair's length took a register and with it
// 246 us where this takes 242, 4 rows of 131071 tokens with weights.)
//
// Bound by HBM where histories are long: 32 rows of up to 8191 tokens, 8 KV
// heads of 128, take 55-59 us (46 for the bytes), 4 rows of 131071 tokens
// without weights 164 us (163).  What it took there: rings of TMA loads in
// place of loads by the threads, conflict-free reads, the split weighted by
// pair (KA_PAIR_COST), and codes that leave the L2 first (61 -> 55 us, and
// 108 -> 101 for two of the long rows with scores: the scores stay in the L2
// for the second launch).  With weights the long rows take 246 us: the scores
// are 134 MB, written and read (24 + 32 us), and the workspace holds two rows'
// at a time, so there are two pairs of launches.  (Token-major scores, half
// the store instructions: the attention took the same time and the second
// launch twice as long, 33 us.)  2048 tokens of one sequence (32 heads) take
// 13 us for 2.6 us of bytes: launch, first loads, the join of the warps and
// of the CTAs follow one another.
// CTAs with equal work do not end together (long rows: after 77 to 100 us, 87
// on average): memory serves some SMs better.  Handing out the work as they
// come would even that out, but either the order of the sums would change from
// call to call or every few blocks would leave a partial of 4 KB.
#include <cmath>

#include "kv8.cuh"
#include "tc.cuh"

namespace fsvd {
namespace {

constexpr int KA_WARPS = 8;
constexpr int KA_THREADS = 32 * KA_WARPS;
// What a pair costs beside its blocks, in blocks (work split): joins, the
// append and the first loads.  (64 rows of up to 600 tokens x 8 heads: 40 us
// with 0, 23.7 with 12; 32 rows of up to 8191: 58 and 52.)
constexpr int KA_PAIR_COST = 12;
// Least units worth a CTA of their own (4 heads x 1000 tokens / 32 x 500: 1, 2,
// 4 and 8 units 8.4, 8.8, 9.4, 10.9 / 10.4, 10.5, 11.5, 12.2 us; with 2 the two
// blocks of a 100-token history still stay together).
constexpr int KA_MIN_UNITS = 2;
constexpr int KA_PSHIFT = 15;  // probabilities and l carry a factor 2^15

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// One pair of the line of units: batch row, KV head, first block of this CTA's
// part, blocks of the pair (0: none), first unit of the pair.
struct KaPair {
  int b, g, j0, nblk, pair0;
};

struct KaParams {
  const bf16* q; const bf16* k_new; const bf16* v_new;
  Kv8 c;
  const int* seqlens;
  bf16* out;
  int H, rep;                  // query heads, query heads per KV head
  float scale_log2;
  float vdown, vup;            // 2^-(K + 15) on the values (15: KA_PSHIFT), its inverse on O / l
  float* part;                 // [2 * workers][KaLayout::SLOT] partials
  int* counters;               // [B * G] contributors done, zero between launches
  float* scores; float* ml;    // weights wanted: x_j [B * H][S_max]; (M, 1 / l) [B * H][2]
  int* status;
};

template <int D, int NT>
struct KaLayout {
  static constexpr int HP = 8 * NT;               // head columns
  static constexpr int OP = D + 4;                // row pitch of an O buffer (floats)
  static constexpr int SLOT = 2 * HP + HP * D;    // floats of one partial: m, l, O
  static constexpr int CTAS = NT == 1 ? 2 : 1;    // CTAs per SM (registers: 128 or 255 a thread)
  static constexpr int HALF = 16 * D;             // bytes of a slice's keys (or values)
  static constexpr int NST = (NT == 1 ? 2 : 4) * (128 / D);  // ring stages of a warp
  static constexpr int RING = KA_WARPS * NST * 2 * HALF;
  static constexpr int O_OFF = RING;              // [warps][HP][OP] floats
  // Workers whose partials of one pair the joining CTA has room for: a factor
  // per head each, beside four sums a thread, where the warps' O were.
  static constexpr int JOIN = (KA_WARPS * HP * OP - 4 * KA_THREADS) / HP;
  static_assert(148 * CTAS <= JOIN, "the CTAs of a B200");
  static constexpr int ML_OFF = O_OFF + KA_WARPS * HP * OP * 4;    // m, l, factor: [3][warps][HP] floats
  static constexpr int BAR_OFF = ML_OFF + 3 * KA_WARPS * HP * 4;
  static constexpr int SMEM = 1024 + BAR_OFF + KA_WARPS * NST * 8;
};

// Token (of the first eight of a slice) in row r of the matrix operands.
// D = 128: kappa(2i) and kappa(2i + 1) differ by 4 and the kappa(2t) lie in
// different pairs, so that with the 128-byte swizzle (16-byte unit u of row r
// at u ^ (r & 7)) the eight lanes of a read phase hit eight different units.
// D = 64 (two tokens a row): the natural order does.
template <int D>
__device__ __forceinline__ int kappa(int r) {
  return D == 128 ? (2 * (r >> 1) + (r >> 2)) ^ ((r & 1) << 2) : r;
}
// Byte offset of 16-byte unit u of token tok within a slice's half.
template <int D>
__device__ __forceinline__ int unit_at(int tok, int u) {
  if (D == 128) return tok * 128 + ((u ^ (tok & 7)) << 4);
  const int r = tok >> 1;
  return r * 128 + ((((tok & 1) * 4 + u) ^ (r & 7)) << 4);
}

__device__ __forceinline__ void mma_bf16_16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One column tile's softmax step over a slice: x (scaled scores; rows l4 and
// l4 + 8, heads 2t and 2t + 1) becomes 2^(x - m + 15); m, l and the output
// sums follow the running maximum.
template <int MT, int NT>
__device__ __forceinline__ void softmax_step(float* x, float* m, float* l, float (*acc)[NT][4], int nt) {
  float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
  }
  if (__any_sync(0xffffffffu, mx0 > m[0] || mx1 > m[1])) {
    const float n0 = fmaxf(m[0], mx0), n1 = fmaxf(m[1], mx1);
    const float c0 = m[0] == -INFINITY ? 0.f : ex2(m[0] - n0);
    const float c1 = m[1] == -INFINITY ? 0.f : ex2(m[1] - n1);
    m[0] = n0; m[1] = n1;
    l[0] *= c0; l[1] *= c1;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      acc[i][nt][0] *= c0; acc[i][nt][1] *= c1; acc[i][nt][2] *= c0; acc[i][nt][3] *= c1;
    }
  }
  // (no finite score so far: subtract nothing, so that 2^-inf stays 0)
  const float e0 = m[0] == -INFINITY ? 0.f : KA_PSHIFT - m[0];
  const float e1 = m[1] == -INFINITY ? 0.f : KA_PSHIFT - m[1];
  x[0] = ex2(x[0] + e0); x[1] = ex2(x[1] + e1);
  x[2] = ex2(x[2] + e0); x[3] = ex2(x[3] + e1);
  l[0] += x[0] + x[2];
  l[1] += x[1] + x[3];
}

template <int D, int NT, bool E4M3, bool SCORES>
__global__ void __launch_bounds__(KA_THREADS, KaLayout<D, NT>::CTAS)
kv8_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                const __grid_constant__ KaParams p) {
  using L = KaLayout<D, NT>;
  constexpr int HP = L::HP, KC = D / 64, MT = D / 16, NST = L::NST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ int s_prefix[KV8_MAX_BATCH + 1], s_pos[KV8_MAX_BATCH];
  __shared__ uint32_t s_amax[2][KA_WARPS];
  __shared__ KaPair s_join[2];  // pairs whose partials this CTA joins
  __shared__ int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int l4 = lane >> 2, t = lane & 3;
  const int B = p.c.B, G = p.c.G, S_max = p.c.S_max, rep = p.rep;
  uint8_t* ring = smem + warp * (NST * 2 * L::HALF);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF) + warp * NST;
  float* s_o = reinterpret_cast<float*>(smem + L::O_OFF);
  float* s_m = reinterpret_cast<float*>(smem + L::ML_OFF);  // [warps][HP]
  float* s_l = s_m + KA_WARPS * HP;
  float* s_f = s_l + KA_WARPS * HP;

  if (lane == 0)
    for (int i = 0; i < NST; ++i) tc::mbar_init(bar + i, 1);
  if (tid == 0) { s_abort = 0; s_join[0].nblk = s_join[1].nblk = 0; }
  tc::fence_barrier_init();
  pdl_launch_dependents();
  pdl_wait();

  // Units before each batch row: a pair is its blocks and KA_PAIR_COST more.
  if (warp == 0) {
    int base = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
      int x = 0;
      if (b0 + lane < B) {
        const int n = p.seqlens[b0 + lane];
        const int pos = n < 0 ? 0 : (n >= S_max ? S_max - 1 : n);
        s_pos[b0 + lane] = pos;
        x = pos / KV8_BLOCK + 1 + KA_PAIR_COST;
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b0 + lane < B) s_prefix[b0 + lane + 1] = base + x;
      base += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) s_prefix[0] = 0;
  }
  __syncthreads();
  // T units over W workers: the first `more` of them take one unit more
  // (all below 2^30: the host checks B G (S_max / 64 + KA_PAIR_COST))
  const int T = s_prefix[B] * G, me = blockIdx.x;
  const int W = min((T + KA_MIN_UNITS - 1) / KA_MIN_UNITS, (int)gridDim.x);
  if (me >= W) return;
  const int each = T / W, more = T - each * W;
  auto first_of = [&](int w) { return w * each + min(w, more); };
  auto worker_of = [&](int v) {
    return v < more * (each + 1) ? v / (each + 1) : more + (v - more * (each + 1)) / each;
  };
  const int u_begin = first_of(me), u_end = first_of(me + 1);

  // The part of a pair that starts at unit u or, where u is behind the
  // pair's blocks, at the next pair (nothing: nblk = 0).
  auto locate = [&](int u) {
    KaPair r;
    r.nblk = 0;
    while (u < u_end) {
      int lo = 0, hi = B - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_prefix[mid] * G <= u) lo = mid; else hi = mid - 1;
      }
      const int span = s_prefix[lo + 1] - s_prefix[lo], rel = u - s_prefix[lo] * G;
      const int g = rel / span, j = rel - g * span;
      if (j < span - KA_PAIR_COST) {
        r.b = lo; r.g = g; r.j0 = j;
        r.nblk = span - KA_PAIR_COST;
        r.pair0 = u - j;
        break;
      }
      u += span - j;
    }
    return r;
  };
  // A part's first load of each ring stage of this warp: slices run over the
  // tail's (which need no stage) and then the codes'; warp w takes w, w + 8, ...
  auto tail_slices = [&](const KaPair& r) {
    return r.nblk > 0 && r.pair0 + r.nblk <= u_end ? (s_pos[r.b] % KV8_BLOCK) / 16 + 1 : 0;
  };
  auto code_slices = [&](const KaPair& r) {
    const int end = r.pair0 + r.nblk <= u_end ? r.nblk - 1 : u_end - r.pair0;
    return r.nblk > 0 ? (end - r.j0) * (KV8_BLOCK / 16) : 0;
  };
  const uint64_t once = tc::policy_evict_first();
  auto issue = [&](const KaPair& r, int s, int use) {
    const int row = (int)((((long long)r.b * G + r.g) * S_max + (long long)r.j0 * KV8_BLOCK) * D / 128) + s * (L::HALF / 128);
    const int st = use % NST;
    uint8_t* dst = ring + st * 2 * L::HALF;
    tc::mbar_expect_tx(bar + st, 2 * L::HALF);
    tc::tma_load_2d_once(dst, &tmK, bar + st, 0, row, once);
    tc::tma_load_2d_once(dst + L::HALF, &tmV, bar + st, 0, row, once);
  };
  auto issue_first = [&](const KaPair& r, int use) {
    const int n_t = tail_slices(r), n_c = code_slices(r);
    int s = warp - n_t + (warp < n_t ? KA_WARPS : 0);
#pragma unroll 1
    for (int i = 0; i < NST && s < n_c; ++i, s += KA_WARPS) issue(r, s, use + i);
  };

  int uses = 0;     // ring uses of this warp so far
  bool ok = true;   // no wait has run out
  KaPair cur = locate(u_begin);
  if (lane == 0) issue_first(cur, uses);

  while (cur.nblk > 0) {
    const int b = cur.b, g = cur.g, j0 = cur.j0, nblk = cur.nblk, pair0 = cur.pair0;
    const int pos = s_pos[b], slot = pos % KV8_BLOCK;
    const bool tail = pair0 + nblk <= u_end;              // the newest block is ours
    const bool whole = j0 == 0 && tail;
    const int n_tail = tail_slices(cur), n_code = code_slices(cur);
    const int n_slices = n_tail + n_code;
    const long long pair = (long long)b * G + g;
    const int h0 = b * p.H + g * rep;                     // first query head (batch-global)

    // ---- q as the B operand: column l4 of tile nt is head 8 nt + l4 ----
    uint32_t qb[NT][KC][8];
    float fs[NT][2];  // score factors of heads 8 nt + 2t, + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = 8 * nt + l4;
      uint4 w[KC][2];
      uint32_t am = 0;
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          w[c][i] = h < rep ? *reinterpret_cast<const uint4*>(p.q + (long long)(h0 + h) * D + c * 64 + t * 16 + 8 * i)
                            : make_uint4(0, 0, 0, 0);
          am = max(am, amax8(w[c][i]));
        }
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
      // 2^k brings the largest |q| into [2^14, 2^15); k within float range
      int k = 141 - (int)(am >> 7);
      k = k > 100 ? 100 : k;
      const float up = exp2i(k);
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          qb[nt][c][4 * i] = pack_h2(bf_lo(w[c][i].x) * up, bf_hi(w[c][i].x) * up);
          qb[nt][c][4 * i + 1] = pack_h2(bf_lo(w[c][i].y) * up, bf_hi(w[c][i].y) * up);
          qb[nt][c][4 * i + 2] = pack_h2(bf_lo(w[c][i].z) * up, bf_hi(w[c][i].z) * up);
          qb[nt][c][4 * i + 3] = pack_h2(bf_lo(w[c][i].w) * up, bf_hi(w[c][i].w) * up);
        }
      const float f = p.scale_log2 * exp2i(-k);
      fs[nt][0] = __shfl_sync(0xffffffffu, f, 8 * t);
      fs[nt][1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
    }

    // ---- this warp's slices ----
    float m[NT][2], l[NT][2], acc[MT][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) { m[nt][i] = -INFINITY; l[nt][i] = 0.f; }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][nt][r] = 0.f;
    const float* ks = p.c.scale[0] + pair * (S_max / KV8_BLOCK) + j0;
    const float* vs = p.c.scale[1] + pair * (S_max / KV8_BLOCK) + j0;
    float* sc = SCORES ? p.scores + (long long)(h0 + 2 * t) * S_max + (long long)j0 * KV8_BLOCK + kappa<D>(l4) : nullptr;
    auto put_scores = [&](int tok, int nt, const float* x, bool v0, bool v1) {
      float* o = sc + (long long)(8 * nt) * S_max + tok;
      if (8 * nt + 2 * t < rep) { if (v0) o[0] = x[0]; if (v1) o[8] = x[2]; }
      if (8 * nt + 2 * t + 1 < rep) { if (v0) o[S_max] = x[1]; if (v1) o[S_max + 8] = x[3]; }
    };

    // ---- one slice of the newest block each for the first warps, from the tail
    // (while the first loads of the codes are on their way) ----
    const bf16* kt = p.c.tail[0] + pair * KV8_BLOCK * D;
    const bf16* vt = p.c.tail[1] + pair * KV8_BLOCK * D;
    const bf16* kn = p.k_new ? p.k_new + pair * D : kt + slot * D;
    const bf16* vn = p.v_new ? p.v_new + pair * D : vt + slot * D;
    if (warp < n_tail) {
      const int tok0 = warp * 16;                 // first token of the slice within the block
      const int ta = tok0 + kappa<D>(l4), tb = ta + 8;    // tokens of rows l4, l4 + 8
      const bf16* ra = ta >= slot ? kn : kt + ta * D;     // (rows behind the newest are masked below)
      const bf16* rb = tb >= slot ? kn : kt + tb * D;
      float x[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 4; ++r) x[nt][r] = 0.f;
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 ka = *reinterpret_cast<const uint4*>(ra + c * 64 + t * 16 + 8 * i);
          const uint4 kb = *reinterpret_cast<const uint4*>(rb + c * 64 + t * 16 + 8 * i);
          const uint32_t a0[4] = {ka.x, kb.x, ka.y, kb.y}, a1[4] = {ka.z, kb.z, ka.w, kb.w};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int h = 8 * nt + l4;
            const uint4 w = h < rep ? *reinterpret_cast<const uint4*>(p.q + (long long)(h0 + h) * D + c * 64 + t * 16 + 8 * i)
                                    : make_uint4(0, 0, 0, 0);
            mma_bf16_16816(x[nt], a0, w.x, w.y);
            mma_bf16_16816(x[nt], a1, w.z, w.w);
          }
        }
      uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int r = 0; r < 4; ++r) x[nt][r] = (r < 2 ? ta : tb) > slot ? -INFINITY : x[nt][r] * p.scale_log2;
        if (SCORES) put_scores((nblk - 1 - j0) * KV8_BLOCK + tok0, nt, x[nt], ta <= slot, tb <= slot);
        softmax_step<MT, NT>(x[nt], m[nt], l[nt], acc, nt);
        float r4[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[nt][r] *= p.vdown;
          r4[r] = x[nt][r] - bf2f(f2bf(x[nt][r]));
        }
        ph[nt][0] = transpose8x8(pack_bf2(x[nt][0], x[nt][1]));
        ph[nt][1] = transpose8x8(pack_bf2(x[nt][2], x[nt][3]));
        pl[nt][0] = transpose8x8(pack_bf2(r4[0], r4[1]));
        pl[nt][1] = transpose8x8(pack_bf2(r4[2], r4[3]));
      }
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint4 v[4];  // eight dimensions of the thread's four tokens
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = tok0 + kappa<D>(2 * t + (i & 1)) + 8 * (i >> 1);
          const bf16* r = tok >= slot ? vn : vt + tok * D;
          v[i] = tok > slot ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4*>(r + l4 * (D / 8) + 8 * c);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w0 = i == 0 ? v[0].x : i == 1 ? v[0].y : i == 2 ? v[0].z : v[0].w;
          const uint32_t w1 = i == 0 ? v[1].x : i == 1 ? v[1].y : i == 2 ? v[1].z : v[1].w;
          const uint32_t w2 = i == 0 ? v[2].x : i == 1 ? v[2].y : i == 2 ? v[2].z : v[2].w;
          const uint32_t w3 = i == 0 ? v[3].x : i == 1 ? v[3].y : i == 2 ? v[3].z : v[3].w;
          const uint32_t a[4] = {__byte_perm(w0, w1, 0x5410), __byte_perm(w0, w1, 0x7632),
                                 __byte_perm(w2, w3, 0x5410), __byte_perm(w2, w3, 0x7632)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_bf16_16816(acc[4 * c + i][nt], a, ph[nt][0], ph[nt][1]);
            mma_bf16_16816(acc[4 * c + i][nt], a, pl[nt][0], pl[nt][1]);
          }
        }
      }
    }

    int s = warp - n_tail + (warp < n_tail ? KA_WARPS : 0);
    float sk = 0.f, sv = 0.f, sk_next = 0.f, sv_next = 0.f;  // the scales, loaded a slice ahead
    if (s < n_code) { sk_next = ks[s >> 2]; sv_next = vs[s >> 2]; }
#pragma unroll 1
    for (; s < n_code; s += KA_WARPS, ++uses) {
      const int st = uses % NST;
      const uint8_t* kh = ring + st * 2 * L::HALF;
      const uint8_t* vh = kh + L::HALF;
      sk = sk_next; sv = sv_next * p.vdown;
      if (s + KA_WARPS < n_code) { sk_next = ks[(s + KA_WARPS) >> 2]; sv_next = vs[(s + KA_WARPS) >> 2]; }
      if (!tc::mbar_wait(bar + st, (uint32_t)(uses / NST) & 1u, &s_abort, p.status)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      // S^T = K Q^T: rows l4, l4 + 8 are tokens kappa(l4), kappa(l4) + 8
      float x[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 4; ++r) x[nt][r] = 0.f;
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const uint4 ka = *reinterpret_cast<const uint4*>(kh + unit_at<D>(kappa<D>(l4), 4 * c + t));
        const uint4 kb = *reinterpret_cast<const uint4*>(kh + unit_at<D>(kappa<D>(l4) + 8, 4 * c + t));
        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a[4];  // (row l4, dims +0 +1), (row l4 + 8, same), (row l4, dims +2 +3), (row l4 + 8, same)
          kv8_decode4<E4M3>(wa[i], a[0], a[2]);
          kv8_decode4<E4M3>(wb[i], a[1], a[3]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(x[nt], a, qb[nt][c][2 * i], qb[nt][c][2 * i + 1]);
        }
      }
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float f0 = fs[nt][0] * sk, f1 = fs[nt][1] * sk;
        x[nt][0] *= f0; x[nt][1] *= f1; x[nt][2] *= f0; x[nt][3] *= f1;
        if (SCORES) put_scores(s * 16, nt, x[nt], true, true);
        softmax_step<MT, NT>(x[nt], m[nt], l[nt], acc, nt);
        pb[nt][0] = transpose8x8(pack_h2(x[nt][0], x[nt][1]));
        pb[nt][1] = transpose8x8(pack_h2(x[nt][2], x[nt][3]));
      }
      // O^T += sv V^T P^T: this thread's tokens are rows 2t, 2t + 1 and 8 on;
      // its dimensions the D / 8 from l4 D / 8 on
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tok = kappa<D>(2 * t + (i & 1)) + 8 * (i >> 1);
        if (D == 128) {
          v[i] = *reinterpret_cast<const uint4*>(vh + unit_at<D>(tok, l4));
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(vh + unit_at<D>(tok, l4 >> 1) + 8 * (l4 & 1));
          v[i] = make_uint4(w.x, w.y, 0, 0);
        }
      }
#pragma unroll
      for (int i = 0; i < MT / 2; ++i) {
        const uint32_t w0 = i == 0 ? v[0].x : i == 1 ? v[0].y : i == 2 ? v[0].z : v[0].w;
        const uint32_t w1 = i == 0 ? v[1].x : i == 1 ? v[1].y : i == 2 ? v[1].z : v[1].w;
        const uint32_t w2 = i == 0 ? v[2].x : i == 1 ? v[2].y : i == 2 ? v[2].z : v[2].w;
        const uint32_t w3 = i == 0 ? v[3].x : i == 1 ? v[3].y : i == 2 ? v[3].z : v[3].w;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // bytes (row 2t, row 2t + 1) of two dimensions, then of rows 2t + 8, 2t + 9
          const uint32_t sel = half ? 0x7362u : 0x5140u;
          uint32_t a[4];
          kv8_decode4<E4M3>(__byte_perm(w0, w1, sel), a[0], a[1]);
          kv8_decode4<E4M3>(__byte_perm(w2, w3, sel), a[2], a[3]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float o[4] = {0.f, 0.f, 0.f, 0.f};
            mma_f16(o, a, pb[nt][0], pb[nt][1]);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[2 * i + half][nt][r] = fmaf(o[r], sv, acc[2 * i + half][nt][r]);
          }
        }
      }
      __syncwarp();
      if (lane == 0 && s + NST * KA_WARPS < n_code) issue(cur, s + NST * KA_WARPS, uses + NST);
    }

    // the next pair's first loads run under this one's join
    const KaPair next = locate(pair0 + nblk);
    if (lane == 0 && ok) issue_first(next, uses);

    // ---- join the warps ----
    const int n_warps = min(KA_WARPS, n_slices);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v = l[nt][i];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (l4 == 0) {
          s_m[warp * HP + 8 * nt + 2 * t + i] = m[nt][i];
          s_l[warp * HP + 8 * nt + 2 * t + i] = v;
        }
      }
      if (warp < n_warps) {
        float* o = s_o + (warp * HP + 8 * nt + 2 * t) * L::OP + l4 * (D / 8);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          *reinterpret_cast<float2*>(o + 2 * i) = make_float2(acc[i][nt][0], acc[i][nt][2]);
          *reinterpret_cast<float2*>(o + L::OP + 2 * i) = make_float2(acc[i][nt][1], acc[i][nt][3]);
        }
      }
    }
    __syncthreads();
    ok = ok && s_abort == 0;
    // a worker's first pair uses its slot 0, its last pair slot 1
    float* part = p.part + (long long)(2 * me + (u_begin < pair0 ? 1 : 0)) * L::SLOT;
    if (tid < HP) {
      float M = -INFINITY, ls = 0.f;
      for (int w = 0; w < n_warps; ++w) M = fmaxf(M, s_m[w * HP + tid]);
      for (int w = 0; w < n_warps; ++w) {
        // a warp whose scores are all NaN has m = -inf and l = NaN
        const float mw = s_m[w * HP + tid];
        const float f = mw == -INFINITY ? 1.f : ex2(mw - M);
        ls = fmaf(s_l[w * HP + tid], f, ls);
        s_f[w * HP + tid] = f;
      }
      s_l[tid] = ls;  // (column tid of every warp is this thread's alone)
      if (whole) {
        if (SCORES && tid < rep) {
          p.ml[2 * (h0 + tid)] = M;
          p.ml[2 * (h0 + tid) + 1] = exp2f(KA_PSHIFT) / ls;
        }
      } else {
        __stcg(part + tid, M);
        __stcg(part + HP + tid, ls);
      }
    }
    __syncthreads();
    for (int i = tid * 4; i < rep * D; i += KA_THREADS * 4) {
      const int h = i / D, dim = i - h * D;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < n_warps; ++w) {
        const float f = s_f[w * HP + h];
        const float4 v = *reinterpret_cast<const float4*>(s_o + (w * HP + h) * L::OP + dim);
        o.x = fmaf(v.x, f, o.x); o.y = fmaf(v.y, f, o.y); o.z = fmaf(v.z, f, o.z); o.w = fmaf(v.w, f, o.w);
      }
      if (whole) {
        const float r = p.vup / s_l[h];
        *reinterpret_cast<uint2*>(p.out + (long long)h0 * D + i) =
            make_uint2(pack_bf2(o.x * r, o.y * r), pack_bf2(o.z * r, o.w * r));
      } else {
        __stcg(reinterpret_cast<float4*>(part + 2 * HP + i), o);
      }
    }

    if (!whole) {
      // the CTA that is last to leave a partial will join them, after its own
      // work (a CTA leaves at most two)
      const int nc = worker_of(pair0 + nblk - 1) - worker_of(pair0) + 1;
      // (the barrier orders the other threads' stores before thread 0's fence)
      __syncthreads();
      if (tid == 0) {
        __threadfence();
        if (atomicAdd(p.counters + pair, 1) == nc - 1) {
          __threadfence();
          s_join[u_begin < pair0 ? 1 : 0] = cur;
        }
      }
    }

    // ---- append: the new rows into the tail, a completed block into the codes ----
    if (tail && p.k_new) {
      if (tid < 2 * (D / 8)) {
        const int x = tid / (D / 8), c = (tid % (D / 8)) * 8;
        *reinterpret_cast<uint4*>(p.c.tail[x] + (pair * KV8_BLOCK + slot) * D + c) =
            *reinterpret_cast<const uint4*>((x ? vn : kn) + c);
      }
      if (slot == KV8_BLOCK - 1) {
        constexpr int UPR = D / 16, PER = KV8_BLOCK * UPR / KA_THREADS;
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
          uint4 a[PER], c[PER];
          uint32_t am = 0;
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const int un = tid + KA_THREADS * i, r = un / UPR, col = (un % UPR) * 16;
            const bf16* src = (r == slot ? (x ? vn : kn) : (x ? vt : kt) + r * D) + col;
            a[i] = *reinterpret_cast<const uint4*>(src);
            c[i] = *reinterpret_cast<const uint4*>(src + 8);
            am = max(am, max(amax8(a[i]), amax8(c[i])));
          }
          am = __reduce_max_sync(0xffffffffu, am);
          if (lane == 0) s_amax[x][warp] = am;
          __syncthreads();
#pragma unroll
          for (int w = 0; w < KA_WARPS; ++w) am = max(am, s_amax[x][w]);
          const int e = kv8_exponent<E4M3>(am);
          const bool fin = kv8_finite(am);
          uint8_t* dst = p.c.codes[x] + (pair * S_max + (long long)(nblk - 1) * KV8_BLOCK) * D;
#pragma unroll
          for (int i = 0; i < PER; ++i)
            *reinterpret_cast<uint4*>(dst + (tid + KA_THREADS * i) * 16) =
                kv8_encode16<E4M3>(a[i], c[i], exp2i(-e), fin);
          if (tid == 0) p.c.scale[x][pair * (S_max / KV8_BLOCK) + nblk - 1] = kv8_scale(e, fin);
        }
      }
    }
    cur = next;
    __syncthreads();
  }

  // ---- join the partials of a pair, in CTA order ----
  for (int x = 0; x < 2; ++x) {
    const int nblk = s_join[x].nblk, pair0 = s_join[x].pair0;
    if (nblk == 0) continue;
    const int h0 = s_join[x].b * p.H + s_join[x].g * rep;
    const int w0 = worker_of(pair0), nc = worker_of(pair0 + nblk - 1) - w0 + 1;
    const int late = first_of(w0) < pair0 ? 1 : 0;  // the pair is the last one of its first worker
    auto slot_of = [&](int k) { return p.part + (long long)(2 * (w0 + k) + (k == 0 ? late : 0)) * L::SLOT; };
    float* fac = s_o;                         // [nc][HP] factors
    float* red = s_o + nc * HP;               // [groups][rep * D] sums
    // vectors of four sums; with few of them, groups of threads share the
    // partials.  A batch of loads is in flight while the factors are formed.
    constexpr int BATCH = 16;
    const int nv = rep * D / 4, groups = max(1, KA_THREADS / nv), grp = tid / nv;
    float4 v[BATCH];
    auto fetch = [&](int i, int k0) {
#pragma unroll
      for (int k = 0; k < BATCH; ++k)
        if (k0 + k * groups < nc) v[k] = __ldcg(reinterpret_cast<const float4*>(slot_of(k0 + k * groups) + 2 * HP) + i);
    };
    const bool mine = tid < nv || grp < groups;
    if (mine) fetch(tid - grp * nv, grp);
    for (int h = warp; h < rep; h += KA_WARPS) {
      // (two partials a lane in registers: more than 64 of one pair are reloaded)
      float mv[2], lv[2], M = -INFINITY, ls = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = lane + 32 * i;
        mv[i] = k < nc ? __ldcg(slot_of(k) + h) : -INFINITY;
        lv[i] = k < nc ? __ldcg(slot_of(k) + HP + h) : 0.f;
        M = fmaxf(M, mv[i]);
      }
      for (int k = lane + 64; k < nc; k += 32) M = fmaxf(M, __ldcg(slot_of(k) + h));
      M = warp_max(M);
      auto take = [&](int k, float mw, float lw) {
        const float f = mw == -INFINITY ? 1.f : ex2(mw - M);
        fac[k * HP + h] = f;
        ls = fmaf(lw, f, ls);
      };
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (lane + 32 * i < nc) take(lane + 32 * i, mv[i], lv[i]);
      for (int k = lane + 64; k < nc; k += 32) take(k, __ldcg(slot_of(k) + h), __ldcg(slot_of(k) + HP + h));
      ls = warp_sum(ls);
      if (lane == 0) {
        s_l[h] = ls;
        if (SCORES) {
          p.ml[2 * (h0 + h)] = M;
          p.ml[2 * (h0 + h) + 1] = exp2f(KA_PSHIFT) / ls;
        }
      }
    }
    __syncthreads();
    if (mine) {
      for (int i = tid - grp * nv; i < nv; i += KA_THREADS) {
        const int h = 4 * i / D;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = grp; k0 < nc; k0 += BATCH * groups) {
          if (k0 != grp || i >= KA_THREADS) fetch(i, k0);
#pragma unroll
          for (int k = 0; k < BATCH; ++k)
            if (k0 + k * groups < nc) {
              const float f = fac[(k0 + k * groups) * HP + h];
              o.x = fmaf(v[k].x, f, o.x); o.y = fmaf(v[k].y, f, o.y);
              o.z = fmaf(v[k].z, f, o.z); o.w = fmaf(v[k].w, f, o.w);
            }
        }
        if (groups > 1) {
          *reinterpret_cast<float4*>(red + 4 * (grp * nv + i)) = o;
        } else {
          const float r = p.vup / s_l[h];
          *reinterpret_cast<uint2*>(p.out + (long long)h0 * D + 4 * i) =
              make_uint2(pack_bf2(o.x * r, o.y * r), pack_bf2(o.z * r, o.w * r));
        }
      }
    }
    if (groups > 1) {
      __syncthreads();
      if (tid < nv) {
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < groups; ++k) {
          const float4 w = *reinterpret_cast<const float4*>(red + 4 * (k * nv + tid));
          o.x += w.x; o.y += w.y; o.z += w.z; o.w += w.w;
        }
        const float r = p.vup / s_l[4 * tid / D];
        *reinterpret_cast<uint2*>(p.out + (long long)h0 * D + 4 * tid) =
            make_uint2(pack_bf2(o.x * r, o.y * r), pack_bf2(o.z * r, o.w * r));
      }
    }
    if (tid == 0) p.counters[(long long)s_join[x].b * G + s_join[x].g] = 0;
    __syncthreads();
  }
  if (!ok && lane == 0) {
    // let copies still in flight land before shared memory is released
    const long long c0 = clock64();
    while (clock64() - c0 < 2000000) {}
  }
}

// weights[b, g, j] (+)= sum over the group's heads of 2^(x_j - M) / l, for
// j = 0..pos; with `fresh` the entry of the token just appended is set.  A
// launch of its own, because M and l are known only once every CTA of a pair
// is done; bound by memory (two rows of 131071 tokens, 64 heads: 84 MB, partly
// from the L2, in 16 us).
struct KwParams {
  const float* scores; const float* ml;
  const int* seqlens;
  float* weights;
  int G, H, rep, S_max, accumulate, fresh;
};
constexpr int KW_THREADS = 256;

__global__ void __launch_bounds__(KW_THREADS)
kv8_weights_kernel(const __grid_constant__ KwParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int pair = blockIdx.y, b = pair / p.G, g = pair - b * p.G;
  int pos = p.seqlens[b];
  pos = pos < 0 ? 0 : (pos >= p.S_max ? p.S_max - 1 : pos);
  const int j = (blockIdx.x * KW_THREADS + threadIdx.x) * 4;  // S_max is a multiple of 64
  if (j > pos) return;
  const long long h0 = (long long)b * p.H + (long long)g * p.rep;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int h = 0; h < p.rep; ++h) {
    const float4 x = __ldcg(reinterpret_cast<const float4*>(p.scores + (h0 + h) * p.S_max + j));
    const float M = p.ml[2 * (h0 + h)], r = p.ml[2 * (h0 + h) + 1];
    a.x = fmaf(ex2(x.x - M), r, a.x);
    a.y = fmaf(ex2(x.y - M), r, a.y);
    a.z = fmaf(ex2(x.z - M), r, a.z);
    a.w = fmaf(ex2(x.w - M), r, a.w);
  }
  float* w = p.weights + (long long)pair * p.S_max + j;
  const float v[4] = {a.x, a.y, a.z, a.w};
  if (j + 3 < pos && p.accumulate) {
    float4 o = *reinterpret_cast<const float4*>(w);
    o.x += a.x; o.y += a.y; o.z += a.z; o.w += a.w;
    *reinterpret_cast<float4*>(w) = o;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (j + i <= pos) w[i] = (p.accumulate && !(p.fresh && j + i == pos)) ? w[i] + v[i] : v[i];
}

template <int D, int NT>
int launch_ka(const KaParams& p, bool scores, int workers, const LaunchTag& tag, cudaStream_t s) {
  using L = KaLayout<D, NT>;
  if (workers > L::JOIN) return FLASHSVD_ERR_UNSUPPORTED_SHAPE;
  CUtensorMap mk, mv;
  const long long rows = (long long)p.c.B * p.c.G * p.c.S_max * D / 128;
  if (rows > 0x7fffffffLL) return FLASHSVD_ERR_UNSUPPORTED_SHAPE;
  FSVD_TRY(encode_map_bytes(&mk, p.c.codes[0], rows, L::HALF / 128));
  FSVD_TRY(encode_map_bytes(&mv, p.c.codes[1], rows, L::HALF / 128));
#define FSVD_KA(E4M3, SC)                                                                  \
  {                                                                                        \
    auto kern = kv8_attn_kernel<D, NT, E4M3, SC>;                                          \
    static SmemAttrOnce once;                                                              \
    FSVD_TRY(set_smem_once(once, kern, L::SMEM));                                          \
    return launch_pdl(tag, kern, dim3(workers), dim3(KA_THREADS), (size_t)L::SMEM, s, mk, mv, p);  \
  }
  if (p.c.e4m3) {
    if (scores) FSVD_KA(true, true)
    FSVD_KA(true, false)
  }
  if (scores) FSVD_KA(false, true)
  FSVD_KA(false, false)
#undef FSVD_KA
}

}  // namespace

int kv8_attn_launch(const Kv8AttnParams& a, int sm_count, cudaStream_t stream) {
  const int rep = a.H / a.c.G, NT = rep <= 8 ? 1 : 2;
  if (rep > 16 || a.c.B > KV8_MAX_BATCH) return FLASHSVD_ERR_UNSUPPORTED_SHAPE;
  const int workers = sm_count * (NT == 1 ? 2 : 1);
  if ((long long)a.c.B * a.c.G * (a.c.S_max / KV8_BLOCK + KA_PAIR_COST) > 0x3fffffffLL)
    return FLASHSVD_ERR_UNSUPPORTED_SHAPE;
  const long long slot = 2 * 8 * NT + 8LL * NT * a.c.D;
  const long long part = 2LL * workers * slot;
  if (part + 2LL * a.c.B * a.H > a.part_cap || (long long)a.c.B * a.c.G > a.counters_cap)
    return FLASHSVD_ERR_UNSUPPORTED_SHAPE;
  // With weights: the scores of as many batch rows as the workspace holds per
  // pair of launches, the rows spread evenly over the pairs; where one row's
  // do not fit, its KV heads are cut in the same way.
  int step = a.c.B, heads = a.c.G;
  if (a.weights) {
    const long long fit = a.scores_cap / ((long long)rep * a.c.S_max);  // (batch row, KV head) pairs
    if (fit < 1) return FLASHSVD_ERR_UNSUPPORTED_SHAPE;
    if (fit < a.c.G) {
      step = 1;
      heads = ceil_div(a.c.G, ceil_div(a.c.G, (int)fit));
    } else if (fit / a.c.G < step) {
      step = ceil_div(a.c.B, ceil_div(a.c.B, (int)(fit / a.c.G)));
    }
  }
  int K = 1;
  while ((1LL << (K - 1)) < a.c.S_max) ++K;
  const int cuts = ceil_div(a.c.G, heads);
  for (int i = 0; i < ceil_div(a.c.B, step) * cuts; ++i) {
    const int b0 = i / cuts * step, g0 = i % cuts * heads;
    const int nb = a.c.B - b0 < step ? a.c.B - b0 : step, ng = a.c.G - g0 < heads ? a.c.G - g0 : heads;
    KaParams p;
    p.c = a.c;
    p.c.B = nb; p.c.G = ng;  // (fewer heads than G: one row, whose heads are contiguous)
    const long long pr = (long long)b0 * a.c.G + g0;
    for (int x = 0; x < 2; ++x) {
      p.c.codes[x] += pr * a.c.S_max * a.c.D;
      p.c.scale[x] += pr * (a.c.S_max / KV8_BLOCK);
      p.c.tail[x] += pr * KV8_BLOCK * a.c.D;
    }
    p.q = a.q + pr * rep * a.c.D;
    p.k_new = a.k_new ? a.k_new + pr * a.c.D : nullptr;
    p.v_new = a.v_new ? a.v_new + pr * a.c.D : nullptr;
    p.out = a.out + pr * rep * a.c.D;
    p.seqlens = a.seqlens + b0;
    p.H = ng * rep; p.rep = rep;
    p.scale_log2 = a.scale_log2;
    p.vup = std::ldexp(1.f, KA_PSHIFT + K);
    p.vdown = 1.f / p.vup;
    p.part = a.part;
    p.counters = a.counters;
    p.status = a.status;
    p.ml = a.part + part;
    p.scores = a.scores;
    // the cache length is only known on the device: the tag counts the capacity
    const double kv = 2.0 * nb * ng * (double)a.c.S_max * a.c.D;
    const LaunchTag tag{"kv8_decode_attn", kv, 2.0 * kv * rep};
    int st;
    if (a.c.D == 128)
      st = NT == 1 ? launch_ka<128, 1>(p, a.weights != nullptr, workers, tag, stream)
                   : launch_ka<128, 2>(p, a.weights != nullptr, workers, tag, stream);
    else
      st = NT == 1 ? launch_ka<64, 1>(p, a.weights != nullptr, workers, tag, stream)
                   : launch_ka<64, 2>(p, a.weights != nullptr, workers, tag, stream);
    FSVD_TRY(st);
    if (a.weights) {
      KwParams w;
      w.scores = p.scores; w.ml = p.ml; w.seqlens = p.seqlens;
      w.weights = a.weights + pr * a.c.S_max;
      w.G = ng; w.H = p.H; w.rep = rep; w.S_max = a.c.S_max;
      w.accumulate = a.accumulate; w.fresh = a.k_new != nullptr;
      const LaunchTag wt{"kv8_weights", 4.0 * nb * (p.H + 2.0 * ng) * a.c.S_max, 0.0};
      const int pairs = nb * ng;
      if (pairs > 65535) return FLASHSVD_ERR_UNSUPPORTED_SHAPE;
      FSVD_TRY(launch_pdl(wt, kv8_weights_kernel, dim3(ceil_div(a.c.S_max, KW_THREADS * 4), pairs), dim3(KW_THREADS), 0,
                          stream, w));
    }
  }
  return FLASHSVD_OK;
}

}  // namespace fsvd
