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
// and the warps are joined through shared memory.  The newest block comes
// from the bf16 tail and is computed in fp32 by the whole CTA, which also
// appends the new rows and, when they complete the block, quantises it.
//
// Matrix instructions: S^T = K Q^T and O^T = V^T P^T (m16n8k16, fp32 sums),
// so that the tokens and the head's dimensions fill the 16 rows and the up
// to 8 query heads of a KV head the 8 columns (two column tiles for 9-16).
// Rounding to fewer bits: q and the codes are exact in half precision (q
// scaled by a power of two), the probabilities are rounded to half after
// scaling by 2^15, so that they keep 11 bits down to 2^-29 and vanish only
// below 2^-40 of the largest; l is summed from the unrounded ones.
#include "kv8.cuh"

namespace fsvd {
namespace {

constexpr int KA_WARPS = 8;
constexpr int KA_THREADS = 32 * KA_WARPS;
constexpr float KA_PSHIFT = 15.f;  // probabilities carry a factor 2^15 (it cancels in O / l)

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

struct KaParams {
  const bf16* q; const bf16* k_new; const bf16* v_new;
  Kv8 c;
  const int* seqlens;
  bf16* out;
  int H, rep;                  // query heads, query heads per KV head
  float scale_log2;
  float* part;                 // [2 * workers][KaLayout::SLOT] partials
  int* counters;               // [B * G] contributors done, zero between launches
  float* scores; float* ml;    // weights wanted: x_j [B * H][S_max]; (M, 1 / l) [B * H][2]
};

template <int D, int NT>
struct KaLayout {
  static constexpr int HP = 8 * NT;              // head columns
  static constexpr int OP = D + 4;               // row pitch of an O buffer (floats)
  static constexpr int SLOT = 2 * HP + HP * D;   // floats of one partial: m, l, O
  // shared memory (floats): O of the warps and of the tail, m and l of each
  static constexpr int O_OFF = 0;
  static constexpr int ML_OFF = (KA_WARPS + 1) * HP * OP;
  static constexpr int Q_OFF = ML_OFF + 2 * (KA_WARPS + 1) * HP;  // q [HP][D] fp32, scaled
  static constexpr int P_OFF = Q_OFF + HP * D;   // tail probabilities [HP][64]
  static constexpr int SMEM = (P_OFF + HP * 64) * 4;
};

// One 16-token slice of a head's codes: keys l4 and l4 + 8 (16 bytes of each
// 64 dimensions), and of the values of tokens 2t, 2t + 1, 2t + 8, 2t + 9 the
// D / 8 dimensions from l4 D / 8 on.
template <int D>
struct Slice {
  uint4 k[2][D / 64];
  uint4 v[4];  // D = 64: .x and .y only
};

template <int D>
__device__ __forceinline__ void load_slice(Slice<D>& s, const uint8_t* k, const uint8_t* v, int l4, int t) {
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int c = 0; c < D / 64; ++c) s.k[r][c] = ld_once(k + (l4 + 8 * r) * D + c * 64 + t * 16);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint8_t* p = v + (2 * t + (i & 1) + 8 * (i >> 1)) * D + l4 * (D / 8);
    if (D == 128) {
      s.v[i] = ld_once(p);
    } else {
      const uint2 w = ld_once8(p);
      s.v[i] = make_uint4(w.x, w.y, 0, 0);
    }
  }
}

template <int D, int NT, bool E4M3, bool SCORES>
__global__ void __launch_bounds__(KA_THREADS)
kv8_attn_kernel(const __grid_constant__ KaParams p) {
  using L = KaLayout<D, NT>;
  constexpr int HP = L::HP, KC = D / 64, MT = D / 16;
  extern __shared__ __align__(16) float sm[];
  __shared__ int s_prefix[KV8_MAX_BATCH + 1];
  __shared__ uint32_t s_amax[2][KA_WARPS];
  __shared__ int s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int l4 = lane >> 2, t = lane & 3;
  const int B = p.c.B, G = p.c.G, S_max = p.c.S_max, rep = p.rep;

  pdl_launch_dependents();
  pdl_wait();

  auto pos_of = [&](int b) {
    const int n = p.seqlens[b];
    return n < 0 ? 0 : (n >= S_max ? S_max - 1 : n);
  };
  // blocks before each batch row
  if (warp == 0) {
    int base = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
      const int nb = b0 + lane < B ? pos_of(b0 + lane) / KV8_BLOCK + 1 : 0;
      int x = nb;
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
  const long long T = (long long)s_prefix[B] * G;
  const long long W = T < gridDim.x ? T : gridDim.x;  // workers with work
  const long long me = blockIdx.x;
  if (me >= W) return;
  long long u = me * T / W;
  const long long u_end = (me + 1) * T / W;
  auto first_of = [&](long long w) { return w * T / W; };

  while (u < u_end) {
    // ---- the pair that unit u belongs to, and this CTA's part of it ----
    int lo = 0, hi = B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((long long)s_prefix[mid] * G <= u) lo = mid; else hi = mid - 1;
    }
    const int b = lo;
    const int pos = pos_of(b), nblk = pos / KV8_BLOCK + 1;
    const long long rel = u - (long long)s_prefix[b] * G;
    const int g = (int)(rel / nblk), j0 = (int)(rel % nblk);
    const long long pair0 = u - j0;                       // first unit of the pair
    const int j1 = (int)min((long long)nblk, j0 + (u_end - u));
    const bool whole = j0 == 0 && j1 == nblk;
    const bool tail = j1 == nblk;                         // the newest block is ours
    const int jc = tail ? nblk - 1 : j1;                  // blocks j0..jc-1 from codes
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

    // ---- this warp's slices of the coded blocks ----
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

    const uint8_t* kc = p.c.codes[0] + (pair * S_max + (long long)j0 * KV8_BLOCK) * D;
    const uint8_t* vc = p.c.codes[1] + (pair * S_max + (long long)j0 * KV8_BLOCK) * D;
    const float* ks = p.c.scale[0] + pair * (S_max / KV8_BLOCK) + j0;
    const float* vs = p.c.scale[1] + pair * (S_max / KV8_BLOCK) + j0;
    const int n_slices = (jc - j0) * (KV8_BLOCK / 16);
    Slice<D> cur, nxt;
    float sk = 0.f, sv = 0.f, skn = 0.f, svn = 0.f;
    if (warp < n_slices) {
      load_slice<D>(cur, kc + (long long)warp * 16 * D, vc + (long long)warp * 16 * D, l4, t);
      sk = ks[warp >> 2]; sv = vs[warp >> 2];
    }
    for (int s = warp; s < n_slices; s += KA_WARPS) {
      const int sn = s + KA_WARPS;
      if (sn < n_slices) {
        load_slice<D>(nxt, kc + (long long)sn * 16 * D, vc + (long long)sn * 16 * D, l4, t);
        skn = ks[sn >> 2]; svn = vs[sn >> 2];
      }
      // S^T = K Q^T
      float x[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 4; ++r) x[nt][r] = 0.f;
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const uint32_t wa[4] = {cur.k[0][c].x, cur.k[0][c].y, cur.k[0][c].z, cur.k[0][c].w};
        const uint32_t wb[4] = {cur.k[1][c].x, cur.k[1][c].y, cur.k[1][c].z, cur.k[1][c].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a[4];  // (key l4, dims +0 +1), (key l4 + 8, same), (key l4, dims +2 +3), (key l4 + 8, same)
          kv8_decode4<E4M3>(wa[i], a[0], a[2]);
          kv8_decode4<E4M3>(wb[i], a[1], a[3]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(x[nt], a, qb[nt][c][2 * i], qb[nt][c][2 * i + 1]);
        }
      }
      // softmax over the slice's 16 tokens (rows l4 and l4 + 8 of a column)
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float f0 = fs[nt][0] * sk, f1 = fs[nt][1] * sk;
        x[nt][0] *= f0; x[nt][1] *= f1; x[nt][2] *= f0; x[nt][3] *= f1;
        if (SCORES) {
          float* sc = p.scores + (long long)(h0 + 8 * nt + 2 * t) * S_max + (long long)j0 * KV8_BLOCK + s * 16 + l4;
          if (8 * nt + 2 * t < rep) { sc[0] = x[nt][0]; sc[8] = x[nt][2]; }
          if (8 * nt + 2 * t + 1 < rep) { sc[S_max] = x[nt][1]; sc[S_max + 8] = x[nt][3]; }
        }
        float mx0 = fmaxf(x[nt][0], x[nt][2]), mx1 = fmaxf(x[nt][1], x[nt][3]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
        }
        if (__any_sync(0xffffffffu, mx0 > m[nt][0] || mx1 > m[nt][1])) {
          const float n0 = fmaxf(m[nt][0], mx0), n1 = fmaxf(m[nt][1], mx1);
          const float c0 = m[nt][0] == -INFINITY ? 0.f : ex2(m[nt][0] - n0);
          const float c1 = m[nt][1] == -INFINITY ? 0.f : ex2(m[nt][1] - n1);
          m[nt][0] = n0; m[nt][1] = n1;
          l[nt][0] *= c0; l[nt][1] *= c1;
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            acc[i][nt][0] *= c0; acc[i][nt][1] *= c1; acc[i][nt][2] *= c0; acc[i][nt][3] *= c1;
          }
        }
        // (no finite score so far: subtract nothing, so that 2^-inf stays 0)
        const float e0 = m[nt][0] == -INFINITY ? 0.f : KA_PSHIFT - m[nt][0];
        const float e1 = m[nt][1] == -INFINITY ? 0.f : KA_PSHIFT - m[nt][1];
#pragma unroll
        for (int r = 0; r < 4; ++r) x[nt][r] = ex2(x[nt][r] + ((r & 1) ? e1 : e0));
        l[nt][0] += x[nt][0] + x[nt][2];
        l[nt][1] += x[nt][1] + x[nt][3];
        pb[nt][0] = transpose8x8(pack_h2(x[nt][0], x[nt][1]));
        pb[nt][1] = transpose8x8(pack_h2(x[nt][2], x[nt][3]));
      }
      // O^T += sv V^T P^T
#pragma unroll
      for (int i = 0; i < MT / 2; ++i) {
        const uint32_t w0 = i == 0 ? cur.v[0].x : i == 1 ? cur.v[0].y : i == 2 ? cur.v[0].z : cur.v[0].w;
        const uint32_t w1 = i == 0 ? cur.v[1].x : i == 1 ? cur.v[1].y : i == 2 ? cur.v[1].z : cur.v[1].w;
        const uint32_t w2 = i == 0 ? cur.v[2].x : i == 1 ? cur.v[2].y : i == 2 ? cur.v[2].z : cur.v[2].w;
        const uint32_t w3 = i == 0 ? cur.v[3].x : i == 1 ? cur.v[3].y : i == 2 ? cur.v[3].z : cur.v[3].w;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // bytes (token 2t, token 2t + 1) of two dimensions, then of tokens 2t + 8, 2t + 9
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
      cur = nxt;
      sk = skn; sv = svn;
    }

    // ---- (m, l, O) of this warp into shared memory ----
    float* s_o = sm + L::O_OFF;
    float* s_m = sm + L::ML_OFF;                       // [warps + 1][HP]
    float* s_l = s_m + (KA_WARPS + 1) * HP;
    float* s_q = sm + L::Q_OFF;
    float* s_p = sm + L::P_OFF;
    __syncthreads();  // the previous pair's readers are done
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
      if (warp < n_slices) {
        float* o = s_o + (warp * HP + 8 * nt + 2 * t) * L::OP + l4 * (D / 8);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          *reinterpret_cast<float2*>(o + 2 * i) = make_float2(acc[i][nt][0], acc[i][nt][2]);
          *reinterpret_cast<float2*>(o + L::OP + 2 * i) = make_float2(acc[i][nt][1], acc[i][nt][3]);
        }
      }
    }

    // ---- the newest block, from the bf16 tail, in fp32 ----
    const int slot = pos % KV8_BLOCK, n_tail = slot + 1;
    if (tail) {
      for (int i = tid; i < HP * D; i += KA_THREADS) {
        const int h = i / D;
        s_q[i] = h < rep ? bf2f(p.q[(long long)h0 * D + i]) * p.scale_log2 : 0.f;
      }
      __syncthreads();
      const bf16* kt = p.c.tail[0] + pair * KV8_BLOCK * D;
      const bf16* vt = p.c.tail[1] + pair * KV8_BLOCK * D;
      const bf16* kn = p.k_new ? p.k_new + pair * D : kt + slot * D;
      const bf16* vn = p.v_new ? p.v_new + pair * D : vt + slot * D;
      {
        const int j = tid & 63, hq = tid >> 6;  // token, first head
        if (j < n_tail) {
          const bf16* kr = j == slot ? kn : kt + j * D;
          float d[HP / 4];
#pragma unroll
          for (int i = 0; i < HP / 4; ++i) d[i] = 0.f;
#pragma unroll 4
          for (int c = 0; c < D; c += 8) {
            const uint4 w = *reinterpret_cast<const uint4*>(kr + c);
            const float kf[8] = {bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y),
                                 bf_lo(w.z), bf_hi(w.z), bf_lo(w.w), bf_hi(w.w)};
#pragma unroll
            for (int i = 0; i < HP / 4; ++i)
#pragma unroll
              for (int e = 0; e < 8; ++e) d[i] = fmaf(kf[e], s_q[(hq + 4 * i) * D + c + e], d[i]);
          }
#pragma unroll
          for (int i = 0; i < HP / 4; ++i) {
            const int h = hq + 4 * i;
            s_p[h * 64 + j] = d[i];
            if (SCORES && h < rep)
              p.scores[(long long)(h0 + h) * S_max + (long long)(nblk - 1) * KV8_BLOCK + j] = d[i];
          }
        }
      }
      __syncthreads();
      for (int h = warp; h < HP; h += KA_WARPS) {
        const float x0 = lane < n_tail ? s_p[h * 64 + lane] : -INFINITY;
        const float x1 = lane + 32 < n_tail ? s_p[h * 64 + lane + 32] : -INFINITY;
        const float mx = warp_max(fmaxf(x0, x1));
        const float e = mx == -INFINITY ? 0.f : KA_PSHIFT - mx;
        const float p0 = lane < n_tail ? ex2(x0 + e) : 0.f;
        const float p1 = lane + 32 < n_tail ? ex2(x1 + e) : 0.f;
        s_p[h * 64 + lane] = p0;
        s_p[h * 64 + lane + 32] = p1;
        const float sum = warp_sum(p0 + p1);
        if (lane == 0) { s_m[KA_WARPS * HP + h] = mx; s_l[KA_WARPS * HP + h] = sum; }
      }
      __syncthreads();
      {
        constexpr int GROUPS = KA_THREADS / D;   // 2 or 4 groups of heads
        constexpr int PER = HP / GROUPS;
        const int dim = tid % D, hg = (tid / D) * PER;
        float o[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) o[i] = 0.f;
#pragma unroll 4
        for (int j = 0; j < n_tail; ++j) {
          const float v = bf2f(j == slot ? vn[dim] : vt[j * D + dim]);
#pragma unroll
          for (int i = 0; i < PER; ++i) o[i] = fmaf(s_p[(hg + i) * 64 + j], v, o[i]);
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) s_o[(KA_WARPS * HP + hg + i) * L::OP + dim] = o[i];
      }
      if (p.k_new) {
        // the new rows into the tail; a completed block into the codes
        if (tid < 2 * (D / 8)) {
          const int x = tid / (D / 8), c = (tid % (D / 8)) * 8;
          *reinterpret_cast<uint4*>(p.c.tail[x] + (pair * KV8_BLOCK + slot) * D + c) =
              *reinterpret_cast<const uint4*>((x ? vn : kn) + c);
        }
        if (n_tail == KV8_BLOCK) {
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
    } else if (tid < HP) {
      s_m[KA_WARPS * HP + tid] = -INFINITY;
      s_l[KA_WARPS * HP + tid] = 0.f;
    }
    __syncthreads();

    // ---- join the warps and the tail ----
    const long long slot_id = 2 * me + (first_of(me) < pair0 ? 1 : 0);
    float* part = p.part + slot_id * L::SLOT;
    for (int i = tid; i < rep * D; i += KA_THREADS) {
      const int h = i / D, dim = i - h * D;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w <= KA_WARPS; ++w) M = fmaxf(M, s_m[w * HP + h]);
      float ls = 0.f, o = 0.f;
#pragma unroll
      for (int w = 0; w <= KA_WARPS; ++w) {
        const bool used = w == KA_WARPS ? tail : w < n_slices;
        const float mw = s_m[w * HP + h];
        // a part whose scores are all NaN has mw = -inf and l = NaN
        const float f = mw == -INFINITY ? (used ? 1.f : 0.f) : ex2(mw - M);
        if (used) {
          ls = fmaf(s_l[w * HP + h], f, ls);
          o = fmaf(s_o[(w * HP + h) * L::OP + dim], f, o);
        }
      }
      if (whole) {
        p.out[(long long)(h0 + h) * D + dim] = f2bf(o / ls);
        if (SCORES && dim == 0) {
          p.ml[2 * (h0 + h)] = M;
          p.ml[2 * (h0 + h) + 1] = 1.f / ls * exp2f(KA_PSHIFT);
        }
      } else {
        __stcg(part + 2 * HP + h * D + dim, o);
        if (dim == 0) { __stcg(part + h, M); __stcg(part + HP + h, ls); }
      }
    }

    if (!whole) {
      // ---- the last CTA of the pair joins the partials in CTA order ----
      const long long w0 = ((pair0 + 1) * W - 1) / T;
      const long long w1 = ((pair0 + nblk) * W - 1) / T;
      const int nc = (int)(w1 - w0 + 1);
      __threadfence();
      __syncthreads();
      if (tid == 0) s_last = atomicAdd(p.counters + pair, 1) == nc - 1;
      __syncthreads();
      if (s_last) {
        __threadfence();
        for (int i = tid; i < rep * D; i += KA_THREADS) {
          const int h = i / D;
          float M = -INFINITY, ls = 0.f, o = 0.f;
          for (int k = 0; k < nc; ++k) {
            const long long w = w0 + k;
            const float* q = p.part + (2 * w + (first_of(w) < pair0 ? 1 : 0)) * L::SLOT;
            const float mw = __ldcg(q + h), lw = __ldcg(q + HP + h), ow = __ldcg(q + 2 * HP + i);
            const float Mn = fmaxf(M, mw);
            const float c = M == -INFINITY ? 1.f : ex2(M - Mn);
            const float f = mw == -INFINITY ? 1.f : ex2(mw - Mn);
            ls = fmaf(ls, c, lw * f);
            o = fmaf(o, c, ow * f);
            M = Mn;
          }
          p.out[(long long)h0 * D + i] = f2bf(o / ls);
          if (SCORES && i % D == 0) {
            p.ml[2 * (h0 + h)] = M;
            p.ml[2 * (h0 + h) + 1] = 1.f / ls * exp2f(KA_PSHIFT);
          }
        }
        if (tid == 0) p.counters[pair] = 0;
      }
    }
    u += j1 - j0;
    __syncthreads();
  }
}

// weights[b, g, j] (+)= sum over the group's heads of 2^(x_j - M) / l, for
// j = 0..pos; with `fresh` the entry of the token just appended is set.
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
#define FSVD_KA(E4M3, SC)                                                                  \
  {                                                                                        \
    auto kern = kv8_attn_kernel<D, NT, E4M3, SC>;                                          \
    static SmemAttrOnce once;                                                              \
    FSVD_TRY(set_smem_once(once, kern, L::SMEM));                                          \
    return launch_pdl(tag, kern, dim3(workers), dim3(KA_THREADS), (size_t)L::SMEM, s, p);  \
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
  const int workers = sm_count;
  const long long slot = 2 * 8 * NT + 8LL * NT * a.c.D;
  const long long part = 2LL * workers * slot;
  // With weights, the scores of as many batch rows as the workspace holds
  // per pair of launches.
  const long long row = (long long)a.H * a.c.S_max + 2LL * a.H;
  const long long room = a.part_cap - part - 4;
  if (room < 0 || (long long)a.c.B * a.c.G > a.counters_cap) return FLASHSVD_ERR_UNSUPPORTED_SHAPE;
  int step = a.c.B;
  if (a.weights) {
    if (row > room) return FLASHSVD_ERR_UNSUPPORTED_SHAPE;
    step = (int)(room / row < step ? room / row : step);
  }
  for (int b0 = 0; b0 < a.c.B; b0 += step) {
    const int nb = a.c.B - b0 < step ? a.c.B - b0 : step;
    KaParams p;
    p.c = a.c;
    p.c.B = nb;
    const long long pr = (long long)b0 * a.c.G;
    for (int x = 0; x < 2; ++x) {
      p.c.codes[x] += pr * a.c.S_max * a.c.D;
      p.c.scale[x] += pr * (a.c.S_max / KV8_BLOCK);
      p.c.tail[x] += pr * KV8_BLOCK * a.c.D;
    }
    p.q = a.q + (long long)b0 * a.H * a.c.D;
    p.k_new = a.k_new ? a.k_new + pr * a.c.D : nullptr;
    p.v_new = a.v_new ? a.v_new + pr * a.c.D : nullptr;
    p.out = a.out + (long long)b0 * a.H * a.c.D;
    p.seqlens = a.seqlens + b0;
    p.H = a.H; p.rep = rep;
    p.scale_log2 = a.scale_log2;
    p.part = a.part;
    p.counters = a.counters;
    p.ml = a.part + part;
    p.scores = p.ml + round_up(2 * nb * a.H, 4);
    // the cache length is only known on the device: the tag counts the capacity
    const double kv = 2.0 * nb * a.c.G * (double)a.c.S_max * a.c.D;
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
      w.G = a.c.G; w.H = a.H; w.rep = rep; w.S_max = a.c.S_max;
      w.accumulate = a.accumulate; w.fresh = a.k_new != nullptr;
      const LaunchTag wt{"kv8_weights", 4.0 * nb * (a.H + 2.0 * a.c.G) * a.c.S_max, 0.0};
      const int pairs = nb * a.c.G;
      if (pairs > 65535) return FLASHSVD_ERR_UNSUPPORTED_SHAPE;
      FSVD_TRY(launch_pdl(wt, kv8_weights_kernel, dim3(ceil_div(a.c.S_max, KW_THREADS * 4), pairs), dim3(KW_THREADS), 0,
                          stream, w));
    }
  }
  return FLASHSVD_OK;
}

}  // namespace fsvd
