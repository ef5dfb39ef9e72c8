// kv8_attend.hip — attention over the 8-bit paged cache (helm_kv8_attend) and
// the weight it gives each cached token (helm_kv8_weigh).
//
// Matrix products are v_mfma_f32_16x16x32_bf16 with both codes taken to bf16
// (exact: e4m3 has fewer bits) and q as it is; a block's scale multiplies the
// scores of its tokens (K) and, as log2 added to the exponent, their
// probabilities (V) instead of the codes: a token far below the maximum whose
// values are large does not underflow on the way.
// Scores are formed transposed, S^T = K Q^T: in the result a lane holds four
// tokens of one query row, which is where the second product, O^T = V^T P^T,
// takes its right operand from — P never leaves the registers.  The order of
// the contracted index is free as long as both operands agree, so
//   - lane (g, m) of a wave (g = lane / 16, m = lane % 16) loads the D/4
//     consecutive codes d = g*D/4.. of token m of a 16-token tile for S^T, and
//   - codes d = m*D/16.. of tokens 4g..4g+3 of two tiles for O^T, whose 4x4
//     byte blocks it transposes in registers (v_perm): output row m of the
//     j-th product is d = m*D/16 + j.
// Both loads cover whole 128-byte tokens; nothing is staged in LDS.
//
// The softmax runs over the tokens in one pass: per query row a reference
// mref (a recent maximum), l = sum 2^(x - mref) and O, with x in units of
// log2.  A wave rescales only where some x exceeds its row's mref by more than
// 8: sums then hold values up to 2^8 times larger, which costs fp32 and bf16
// no precision, and the steady state has no exchange between lanes.
//
// A row of the products is a (query, head of the group) pair: single tokens of
// a group of up to 16 heads share each key read.
#include <math.h>

#include "serve.hpp"

namespace helm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.0f;       // log2 of how far sums may outgrow mref
constexpr int kStep = 32;           // tokens a wave takes at a time: the second product's depth

__device__ __forceinline__ bf16x2 cvt_pair(uint32_t w, bool high) {
  return high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, 1.0f, true)
              : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, 1.0f, false);
}
// 8 codes in two words to bf16.
__device__ __forceinline__ bf16x8 cvt8(uint32_t lo, uint32_t hi) {
  const bf16x2 a = cvt_pair(lo, false), b = cvt_pair(lo, true), c = cvt_pair(hi, false), d = cvt_pair(hi, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Bytes of four words transposed: w[j] = byte j of t0, t1, t2, t3.
__device__ __forceinline__ void transpose4(uint32_t t0, uint32_t t1, uint32_t t2, uint32_t t3, uint32_t* w) {
  const uint32_t a = __builtin_amdgcn_perm(t1, t0, 0x05010400u), b = __builtin_amdgcn_perm(t1, t0, 0x07030602u);
  const uint32_t c = __builtin_amdgcn_perm(t3, t2, 0x05010400u), d = __builtin_amdgcn_perm(t3, t2, 0x07030602u);
  w[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
  w[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
  w[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
  w[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

__device__ __forceinline__ f32x4 mfma(const bf16x8& a, const bf16x8& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// One request's queries and context, uniform over the wave.
struct Request {
  int r, n;          // its index, its queries
  int64_t c0;        // packed index of its first query
  int len;           // tokens present in its context
  int pos0;          // position of its first query
};
__device__ __forceinline__ Request request_at(const Kv8AttendArgs& a, int r) {
  Request q;
  q.r = r;
  q.c0 = cu_at(a.cu, r, a.n_tok);
  q.n = (int)max((int64_t)0, cu_at(a.cu, r + 1, a.n_tok) - q.c0);
  const int kv = max(a.kv_len[r], 0);
  q.len = (int)min(min((int64_t)kv, (int64_t)a.c.max_len), (int64_t)a.c.max_blocks * a.c.B);
  q.pos0 = kv - q.n;
  return q;
}

// A 16-token tile of a request's context: where its codes are.
struct Tile {
  int64_t slab;      // (block, head)
  int off;           // first slot
  bool ok;           // inside the context, in a block of the pool
};
__device__ __forceinline__ Tile tile_at(const Kv8Cache& c, const int32_t* row, int h, int t, int len) {
  Tile x;
  const int page = c.page_magic ? (int)__umulhi((uint32_t)t >> 4, c.page_magic) : t >> 4;
  x.ok = t < len;
  int blk = 0;
  if (x.ok) blk = row[page];
  x.ok = x.ok && (uint32_t)blk < (uint32_t)c.n_blocks;
  blk = __builtin_amdgcn_readfirstlane(x.ok ? blk : 0);
  x.slab = (int64_t)blk * c.H + h;
  x.off = t - page * c.B;
  if (!x.ok) x.off = 0;
  return x;
}

// Keys of a tile: this lane's D/4 codes.
template <int D>
__device__ __forceinline__ void load_k(const Kv8Cache& c, const Tile& x, int g, int m, u32x4 (&w)[D / 64]) {
  const uint8_t* p = c.k_pool + (x.slab * c.B + x.off) * D + m * D + g * (D / 4);
#pragma unroll
  for (int i = 0; i < D / 64; ++i) w[i] = *(const u32x4*)(p + 16 * i);
}

// 16 queries as the right operand of S^T: this lane's row, d = g*D/4 + 8s.
template <int D>
__device__ __forceinline__ void load_q(const Kv8AttendArgs& a, const Request& q, int h, int row, int g,
                                       bf16x8 (&v)[D / 32]) {
  const int i = row / a.G;
  const uint16_t* p = a.q + (q.c0 + i) * a.q_tok + (int64_t)(h * a.G + row - i * a.G) * a.q_head + g * (D / 4);
#pragma unroll
  for (int s = 0; s < D / 32; ++s) __builtin_memcpy(&v[s], p + 8 * s, 16);
}

template <int D>
__device__ __forceinline__ f32x4 scores(const u32x4 (&k)[D / 64], const bf16x8 (&q)[D / 32]) {
  f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    s = mfma(cvt8(k[i][0], k[i][1]), q[2 * i], s);
    s = mfma(cvt8(k[i][2], k[i][3]), q[2 * i + 1], s);
  }
  return s;
}

// Tokens [lo, hi) that a query row sees.
struct Seen {
  int lo, hi;
};
__device__ __forceinline__ Seen seen_by(const Kv8AttendArgs& a, const Request& q, int i) {
  Seen s = {0, q.len};
  if (a.causal) {
    const int p1 = q.pos0 + i + 1;
    s.hi = min(q.len, p1);
    if (a.window) s.lo = max(0, p1 - a.window);
  }
  return s;
}

// ---- attention ------------------------------------------------------------
// One workgroup: 16*MT rows of one request and KV head over one piece of its
// context; its waves take 32 tokens in turn and join at the end.
template <int D, int MT>
__global__ void __launch_bounds__(kThreads) kv8_attend_kernel(Kv8AttendArgs a) {
  constexpr int TR = 16 * MT, NJ = D / 16, PAD = D + 4;
  __shared__ float lds_o[kWaves][TR][PAD];
  __shared__ float lds_m[kWaves][TR], lds_l[kWaves][TR];
  const Kv8Cache& c = a.c;
  const int split = blockIdx.x % a.splits;
  const int th = blockIdx.x / a.splits;
  const int h = th % c.H;
  int64_t base;
  const int r = owner_of(a.cu, c.R, a.n_tok, a.G, TR, 1, th / c.H, base);
  const Request q = request_at(a, r);
  const int M = q.n * a.G;
  const int64_t first = (th / c.H - base) * TR;
  if (first >= M) return;
  const int row0 = (int)first;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;

  bf16x8 qv[MT][D / 32];
  Seen see[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int row = min(row0 + 16 * t + m, M - 1);
    load_q<D>(a, q, h, row, g, qv[t]);
    see[t] = seen_by(a, q, row / a.G);
  }
  const Seen s_first = seen_by(a, q, row0 / a.G), s_last = seen_by(a, q, (min(row0 + TR, M) - 1) / a.G);
  const int begin = (s_first.lo & ~15) + split * a.chunk;
  const int end = min(s_last.hi, begin + a.chunk);

  f32x4 o[MT][NJ];
  float mref[MT], l[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    mref[t] = -3.402823466e38f;
    l[t] = 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) o[t][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  const int32_t* table = c.table + (int64_t)q.r * c.max_blocks;
  for (int t0 = begin + wave * kStep; t0 < end; t0 += kWaves * kStep) {
    Tile x[2];
    u32x4 kw[2][D / 64];
    uint32_t vw[2][4][D / 64];
    float ks[2], vs[2];
    bool odd = t0 + kStep > q.len;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      x[u] = tile_at(c, table, h, t0 + 16 * u, q.len);
      load_k<D>(c, x[u], g, m, kw[u]);
      const uint8_t* p = c.v_pool + (x[u].slab * c.B + x[u].off + 4 * g) * D + m * (D / 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (D == 128) {
          const u32x2 v = *(const u32x2*)(p + i * D);
          vw[u][i][0] = v[0];
          vw[u][i][1] = v[1];
        } else {
          vw[u][i][0] = *(const uint32_t*)(p + i * D);
        }
      }
      ks[u] = c.k_scale[x[u].slab] * a.scale_log2;
      vs[u] = c.v_scale[x[u].slab];
      odd |= !x[u].ok || !(vs[u] > 0.0f);
    }
    // tokens past the context are not read as numbers: their codes may be anything
    if (odd) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bool none = !x[u].ok || !(vs[u] > 0.0f);
        if (none) vs[u] = 1.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (none || t0 + 16 * u + 4 * g + i >= q.len) {
#pragma unroll
            for (int b = 0; b < D / 64; ++b) vw[u][i][b] = 0u;
          }
      }
    }
    float lv[2], inv[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      lv[u] = __builtin_amdgcn_logf(vs[u]);
      inv[u] = __builtin_amdgcn_rcpf(vs[u]);
    }
    const bool all_seen = t0 >= s_last.lo && t0 + kStep <= s_first.hi && x[0].ok && x[1].ok;

    bf16x8 pv[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      float y[8];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const f32x4 s = scores<D>(kw[u], qv[t]);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[4 * u + i] = fmaf(s[i], ks[u], lv[u]);
      }
      if (!all_seen) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tok = t0 + 16 * u + 4 * g + i;
            if (!x[u].ok || tok < see[t].lo || tok >= see[t].hi) y[4 * u + i] = -INFINITY;
          }
      }
      const float top0 = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])) - lv[0];
      const float top1 = fmaxf(fmaxf(y[4], y[5]), fmaxf(y[6], y[7])) - lv[1];
      float top = fmaxf(top0, top1);
      if (__any(top > mref[t] + kLazy)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        top = fmaxf(top, mref[t]);
        const float shrink = exp2f(mref[t] - top);
        mref[t] = top;
        l[t] *= shrink;
#pragma unroll
        for (int j = 0; j < NJ; ++j) o[t][j] *= shrink;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = __builtin_amdgcn_exp2f(y[i] - mref[t]);   // probability times the value's scale
        l[t] = fmaf(p, inv[i >> 2], l[t]);
        pv[t][i] = (__bf16)p;
      }
    }
#pragma unroll
    for (int b = 0; b < D / 64; ++b) {
      uint32_t w0[4], w1[4];
      transpose4(vw[0][0][b], vw[0][1][b], vw[0][2][b], vw[0][3][b], w0);
      transpose4(vw[1][0][b], vw[1][1][b], vw[1][2][b], vw[1][3][b], w1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bf16x8 v = cvt8(w0[j], w1[j]);
#pragma unroll
        for (int t = 0; t < MT; ++t) o[t][4 * b + j] = mfma(v, pv[t], o[t][4 * b + j]);
      }
    }
  }

  // join the waves: lane (g, m) has row m, d = g*D/4 + (D/16)*i + j
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    l[t] += __shfl_xor(l[t], 16);
    l[t] += __shfl_xor(l[t], 32);
    if (g == 0) {
      lds_m[wave][16 * t + m] = mref[t];
      lds_l[wave][16 * t + m] = l[t];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int b = 0; b < D / 64; ++b)
        *(f32x4*)&lds_o[wave][16 * t + m][g * (D / 4) + (D / 16) * i + 4 * b] =
            f32x4{o[t][4 * b][i], o[t][4 * b + 1][i], o[t][4 * b + 2][i], o[t][4 * b + 3][i]};
  }
  __syncthreads();
  const int64_t rows = a.n_tok * a.Hq;
  for (int e = threadIdx.x; e < TR * (D / 4); e += kThreads) {
    const int t = e / (D / 4), d = e % (D / 4) * 4, row = row0 + t;
    if (row >= M) break;
    float top = lds_m[0][t];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) top = fmaxf(top, lds_m[w][t]);
    float sum = 0.0f;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float f = exp2f(lds_m[w][t] - top);
      sum += f * lds_l[w][t];
      v += f * *(const f32x4*)&lds_o[w][t][d];
    }
    const int i = row / a.G;
    const int64_t at = (q.c0 + i) * a.Hq + h * a.G + (row - i * a.G);
    if (a.splits == 1) {
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;   // a row that sees nothing: 0
      const bf16x2 lo = {(__bf16)(v[0] * inv), (__bf16)(v[1] * inv)}, hi = {(__bf16)(v[2] * inv), (__bf16)(v[3] * inv)};
      const u32x2 w = {__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
      *(u32x2*)(a.out + at * D + d) = w;
      if (d == 0) a.lse[at] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
    } else {
      float* ml = a.part + ((int64_t)split * rows + at) * 2;
      if (d == 0) *(f32x2*)ml = f32x2{top, sum};
      if (sum != 0.0f)
        *(f32x4*)(a.part + 2 * (int64_t)a.splits * rows + ((int64_t)split * rows + at) * D + d) = v;
    }
  }
}

// Joins the pieces of a split context: one workgroup per (query, head), its
// threads side by side over the D values and, in kThreads * 4 / D groups, over
// the pieces.
template <int D>
__global__ void __launch_bounds__(kThreads) kv8_join_kernel(Kv8AttendArgs a) {
  constexpr int NG = kThreads * 4 / D;
  __shared__ float red_m[kWaves], red_l[NG];
  __shared__ f32x4 red_o[NG][D / 4];
  const int64_t rows = a.n_tok * a.Hq, at = blockIdx.x;
  const f32x2* ml = (const f32x2*)a.part + at;
  const float* part = a.part + 2 * (int64_t)a.splits * rows;
  float top = -3.402823466e38f;
  for (int s = threadIdx.x; s < a.splits; s += kThreads) top = fmaxf(top, ml[s * rows][0]);
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
  if ((threadIdx.x & 63) == 0) red_m[threadIdx.x >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) top = fmaxf(top, red_m[w]);
  const int d = threadIdx.x % (D / 4), grp = threadIdx.x / (D / 4);
  float sum = 0.0f;
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int s = grp; s < a.splits; s += NG) {
    const f32x2 x = ml[s * rows];
    if (x[1] == 0.0f) continue;      // nothing seen there: no sums were written
    const float f = exp2f(x[0] - top);
    sum += f * x[1];
    v += f * *(const f32x4*)(part + (s * rows + at) * D + 4 * d);
  }
  red_o[grp][d] = v;
  if (d == 0) red_l[grp] = sum;
  __syncthreads();
  if (grp != 0) return;
#pragma unroll
  for (int i = 1; i < NG; ++i) {
    sum += red_l[i];
    v += red_o[i][d];
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const bf16x2 lo = {(__bf16)(v[0] * inv), (__bf16)(v[1] * inv)}, hi = {(__bf16)(v[2] * inv), (__bf16)(v[3] * inv)};
  *(u32x2*)(a.out + at * D + 4 * d) = u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
  if (d == 0) a.lse[at] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// ---- accumulated weight ---------------------------------------------------
// The scores again, with 2^(x - lse) summed over the rows.  Each weight is
// summed by one workgroup.  ROWS: the waves share 64 tokens and take row tiles
// in turn (prompts); else each wave has 32 tokens of its own (few rows).
template <int D, bool ROWS>
__global__ void __launch_bounds__(kThreads) kv8_weigh_kernel(Kv8AttendArgs a) {
  constexpr int SUB = ROWS ? 4 : 2;
  __shared__ float red[ROWS ? kWaves : 1][64];
  const Kv8Cache& c = a.c;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
  const int h = blockIdx.y;
  const Request q = request_at(a, blockIdx.z);
  const int t0 = blockIdx.x * (ROWS ? 64 : 128) + (ROWS ? 0 : wave * 32);
  if (blockIdx.x * (ROWS ? 64 : 128) >= q.len) return;

  const int32_t* table = c.table + (int64_t)q.r * c.max_blocks;
  Tile x[SUB];
  u32x4 kw[SUB][D / 64];
  float ks[SUB];
  f32x4 acc[SUB];
#pragma unroll
  for (int u = 0; u < SUB; ++u) {
    x[u] = tile_at(c, table, h, t0 + 16 * u, q.len);
    load_k<D>(c, x[u], g, m, kw[u]);
    ks[u] = c.k_scale[x[u].slab] * a.scale_log2;
    acc[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  const int M = q.n * a.G;
  for (int row0 = ROWS ? 16 * wave : 0; row0 < M; row0 += ROWS ? 16 * kWaves : 16) {
    const Seen s_first = seen_by(a, q, row0 / a.G), s_last = seen_by(a, q, (min(row0 + 16, M) - 1) / a.G);
    if (s_last.hi <= t0 || s_first.lo >= t0 + 16 * SUB) continue;
    const int row = min(row0 + m, M - 1), i = row / a.G;
    bf16x8 qv[D / 32];
    load_q<D>(a, q, h, row, g, qv);
    const Seen see = seen_by(a, q, i);
    float lse = a.lse[(q.c0 + i) * a.Hq + h * a.G + (row - i * a.G)] * kLog2e;
    if (row0 + m >= M || !(fabsf(lse) <= 3.402823466e38f)) lse = INFINITY;   // adds nothing
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      const f32x4 s = scores<D>(kw[u], qv);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int tok = t0 + 16 * u + 4 * g + e;
        const float p = __builtin_amdgcn_exp2f(fmaf(s[e], ks[u], -lse));
        acc[u][e] += x[u].ok && tok >= see.lo && tok < see.hi ? p : 0.0f;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < SUB; ++u) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) acc[u][e] += __shfl_xor(acc[u][e], o);
    }
    if constexpr (ROWS) {
      if (m == 0) *(f32x4*)&red[wave][16 * u + 4 * g] = acc[u];
    } else if (m == 0 && x[u].ok) {
      float* w = a.weights + x[u].slab * c.B + x[u].off + 4 * g;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (t0 + 16 * u + 4 * g + e < q.len) w[e] += acc[u][e];
    }
  }
  if constexpr (ROWS) {
    __syncthreads();
    if (wave == 0) {
      float sum = red[0][lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) sum += red[w][lane];
#pragma unroll
      for (int u = 0; u < SUB; ++u)
        if (g == u && x[u].ok && t0 + lane < q.len) a.weights[x[u].slab * c.B + x[u].off + m] += sum;
    }
  }
}

template <int D>
hipError_t attend(const Kv8AttendArgs& a, hipStream_t stream) {
  const bool two = a.n_tok * a.G > 16 * (int64_t)a.c.R;
  const int64_t tiles = a.n_tok * a.G / (two ? 32 : 16) + a.c.R;
  const int64_t grid = tiles * a.c.H * a.splits;
  if (two)
    kv8_attend_kernel<D, 2><<<dim3((unsigned)grid), kThreads, 0, stream>>>(a);
  else
    kv8_attend_kernel<D, 1><<<dim3((unsigned)grid), kThreads, 0, stream>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t rows = a.n_tok * a.Hq;
  kv8_join_kernel<D><<<dim3((unsigned)rows), kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

template <int D>
hipError_t weigh(const Kv8AttendArgs& a, hipStream_t stream) {
  const bool rows = a.n_tok * a.G > 32 * (int64_t)a.c.R;
  const int per = rows ? 64 : 128;
  const dim3 grid((unsigned)((a.c.max_len + per - 1) / per), (unsigned)a.c.H, (unsigned)a.c.R);
  if (rows)
    kv8_weigh_kernel<D, true><<<grid, kThreads, 0, stream>>>(a);
  else
    kv8_weigh_kernel<D, false><<<grid, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

void kv8_attend_split(Kv8AttendArgs& a) {
  const int TR = a.n_tok * a.G > 16 * (int64_t)a.c.R ? 32 : 16;
  int64_t tiles = (a.n_tok * a.G + TR - 1) / TR;
  if (tiles < a.c.R) tiles = a.c.R < a.n_tok ? a.c.R : a.n_tok;
  int64_t span = a.c.max_len;   // tokens that one row tile looks at, at most
  if (a.causal && a.window && (int64_t)a.window + TR + 16 < span) span = (int64_t)a.window + TR + 16;
  const int64_t base = tiles * a.c.H;
  int64_t splits = base > 0 ? 1536 / base : 1;
  const int64_t most = span / 256;
  if (splits > most) splits = most;
  if (splits < 1) splits = 1;
  const int64_t chunk = (span + splits - 1) / splits;
  a.chunk = (int32_t)((chunk + kWaves * kStep - 1) / (kWaves * kStep) * (kWaves * kStep));
  a.splits = (int32_t)((span + a.chunk - 1) / a.chunk);
  if (a.splits < 1) a.splits = 1;
}

size_t kv8_attend_workspace(const Kv8AttendArgs& a) {
  return a.splits == 1 ? 0 : (size_t)a.splits * a.n_tok * a.Hq * (2 + a.c.D) * sizeof(float);
}

hipError_t launch_kv8_attend(const Kv8AttendArgs& a, hipStream_t stream) {
  return a.c.D == 128 ? attend<128>(a, stream) : attend<64>(a, stream);
}
hipError_t launch_kv8_weigh(const Kv8AttendArgs& a, hipStream_t stream) {
  return a.c.D == 128 ? weigh<128>(a, stream) : weigh<64>(a, stream);
}

}  // namespace helm
