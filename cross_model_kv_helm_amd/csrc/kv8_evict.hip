// kv8_evict.hip — eviction by accumulated weight (helm_kv8_evict).
//
// Selection, one workgroup per (request, KV head): the weights become 32-bit
// keys in the same order (NaN lowest), a radix selection of four 8-bit digits
// finds the key of the last token that stays and how many equal ones stay with
// it, and one ordered pass writes the kept indices ascending (the first of the
// equal ones, so ties go to the lowest index).  Each pass reads the request's
// weights again, from L2.
//
// Copy, one workgroup per (block written, head, K or V): the kept tokens'
// codes, whose blocks have scales of their own, are taken to one new scale.
// The blocks written are disjoint from the blocks read, so the copies need no
// order.  Bound by memory: 2 bytes moved per kept value, 8 per token looked at.
#include "serve.hpp"

namespace helm {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;
constexpr int kThreads = 256;

// Larger weight, larger key; -0 equals +0; NaN below -inf.
__device__ __forceinline__ uint32_t key_of(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ int clamped_len(const Kv8Cache& c, int len) {
  const int64_t room = (int64_t)c.max_blocks * c.B;
  return (int)max((int64_t)0, min(min((int64_t)len, (int64_t)c.max_len), room));
}

// Weight of token t of request r, head h; a token of an absent block: NaN (goes first).
__device__ __forceinline__ float weight_at(const Kv8EvictArgs& a, const int32_t* row, int h, int t) {
  const Kv8Cache& c = a.c;
  const int page = c.page_magic ? (int)__umulhi((uint32_t)t >> 4, c.page_magic) : t >> 4;
  const int blk = row[page];
  if ((uint32_t)blk >= (uint32_t)c.n_blocks) return __builtin_nanf("");
  return a.weights[((int64_t)blk * c.H + h) * c.B + (t - page * c.B)];
}

__global__ void __launch_bounds__(kSelThreads) kv8_select_kernel(Kv8EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int found[2];                 // digit, how many of the tokens above stay
  __shared__ int above[2][kSelWaves], equal[2][kSelWaves];
  const Kv8Cache& c = a.c;
  const int r = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int n = clamped_len(c, a.kv_len[r]);
  const int keep = min(n, a.budget);
  int32_t* kept = a.kept + ((int64_t)r * c.H + h) * a.budget;
  if (h == 0 && tid == 0) a.new_len[r] = keep;
  for (int j = keep + tid; j < a.budget; j += kSelThreads) kept[j] = -1;
  if (n <= a.budget) {
    for (int j = tid; j < keep; j += kSelThreads) kept[j] = j;
    return;
  }
  const int32_t* row = c.table + (int64_t)r * c.max_blocks;
  const int cand = n - a.recent;           // tokens that compete
  int need = a.budget - a.recent;          // how many of them stay: 0 <= need < cand

  uint32_t prefix = 0, mask = 0;           // the digits found so far
  for (int shift = 24; need > 0 && shift >= 0; shift -= 8) {
    for (int j = tid; j < 256; j += kSelThreads) hist[j] = 0;
    __syncthreads();
    for (int t = tid; t < cand; t += kSelThreads) {
      const uint32_t k = key_of(weight_at(a, row, h, t));
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (wave == 0) {   // from the largest digit down: lane l looks at digits 255-4l .. 252-4l
      int own = 0;
      for (int j = 0; j < 4; ++j) own += hist[255 - 4 * lane - j];
      int before = own;
      for (int o = 1; o < 64; o <<= 1) {
        const int x = __shfl_up(before, o);
        if (lane >= o) before += x;
      }
      before -= own;
      if (before < need && before + own >= need) {
        int d = 255 - 4 * lane;
        while (before + hist[d] < need) before += hist[d--];
        found[0] = d;
        found[1] = before;
      }
    }
    __syncthreads();
    prefix |= (uint32_t)found[0] << shift;
    mask |= 255u << shift;
    need -= found[1];
    __syncthreads();
  }
  // need: how many tokens of key `prefix` stay (0 only where none competes)

  int written = 0, same = 0;               // kept so far, equal ones seen so far
  for (int t0 = 0, buf = 0; t0 < n; t0 += kSelThreads, buf ^= 1) {
    const int t = t0 + tid;
    const uint32_t k = t < cand ? key_of(weight_at(a, row, h, t)) : 0u;
    const bool over = t < n && (t >= cand || (need > 0 && k > prefix));
    const bool tie = t < cand && need > 0 && k == prefix;
    const uint64_t bo = __ballot(over), be = __ballot(tie);
    if (lane == 0) {
      above[buf][wave] = __popcll(bo);
      equal[buf][wave] = __popcll(be);
    }
    __syncthreads();
    int o_before = 0, e_before = 0, o_all = 0, e_all = 0;
    for (int w = 0; w < kSelWaves; ++w) {
      const int o = above[buf][w], e = equal[buf][w];
      if (w < wave) { o_before += o; e_before += e; }
      o_all += o;
      e_all += e;
    }
    const uint64_t low = (uint64_t(1) << lane) - 1;
    const int e_rank = same + e_before + __popcll(be & low);       // equal tokens before this one
    const int at = written + o_before + __popcll(bo & low) + (min(e_rank, need) - min(same, need));
    if (over || (tie && e_rank < need)) kept[at] = t;
    written += o_all + (min(same + e_all, need) - min(same, need));
    same += e_all;
  }
}

__global__ void __launch_bounds__(kThreads) kv8_copy_kernel(Kv8EvictArgs a) {
  __shared__ float red[kThreads / 64];
  const Kv8Cache& c = a.c;
  const int page = blockIdx.x, h = blockIdx.y, r = blockIdx.z >> 1;
  const bool is_v = blockIdx.z & 1;
  const int keep = min(clamped_len(c, a.kv_len[r]), a.budget);
  const int j0 = page * c.B;
  if (j0 >= keep) return;
  const int blk = a.dst[(int64_t)r * a.max_dst + page];
  if ((uint32_t)blk >= (uint32_t)c.n_blocks) return;
  const int cnt = min(c.B, keep - j0);
  const int32_t* kept = a.kept + ((int64_t)r * c.H + h) * a.budget + j0;
  const int32_t* row = c.table + (int64_t)r * c.max_blocks;
  const uint8_t* pool = is_v ? c.v_pool : c.k_pool;
  const float* scales = is_v ? c.v_scale : c.k_scale;
  const int per = c.D / 16, shift = 31 - __clz(per);   // 16-byte pieces of a token

  const int64_t dst = (int64_t)blk * c.H + h;
  float amax = 0.0f;
  // first the size of what is kept, then (from the caches) its codes
  for (int phase = 0; phase < 2; ++phase) {
    float inv = 0.0f;
    if (phase) {
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
      if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = amax;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kThreads / 64; ++w) amax = fmaxf(amax, red[w]);
      const float now = kv8_scale_of(amax);
      inv = 1.0f / now;
      if (threadIdx.x == 0) (is_v ? c.v_scale : c.k_scale)[dst] = now;
    }
    for (int u = threadIdx.x; u < c.B * per; u += kThreads) {
      const int j = u >> shift, part = u & (per - 1);
      u32x4 w = {0, 0, 0, 0};
      float s = 0.0f;
      if (j < cnt) {
        const int t = kept[j];
        const int sp = c.page_magic ? (int)__umulhi((uint32_t)t >> 4, c.page_magic) : t >> 4;
        const int sb = row[sp];
        if ((uint32_t)sb < (uint32_t)c.n_blocks) {
          const int64_t from = (int64_t)sb * c.H + h;
          s = scales[from];
          w = *(const u32x4*)(pool + (from * c.B + (t - sp * c.B)) * c.D + part * 16);
          if (phase && !is_v && part == 0) a.weights[dst * c.B + j] = a.weights[from * c.B + (t - sp * c.B)];
        } else if (phase && !is_v && part == 0) {
          a.weights[dst * c.B + j] = 0.0f;
        }
      } else if (phase && !is_v && part == 0) {
        a.weights[dst * c.B + j] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f32x4 x = kv8_decode4(w[i]);
        if (!phase) {
#pragma unroll
          for (int e = 0; e < 4; ++e) amax = fmaxf(amax, kv8_size(x[e] * s));
        } else {
          const float f = s * inv;
          w[i] = kv8_encode4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
        }
      }
      if (phase) *(u32x4*)((is_v ? c.v_pool : c.k_pool) + (dst * c.B + j) * c.D + part * 16) = w;
    }
  }
}

}  // namespace

hipError_t launch_kv8_evict(const Kv8EvictArgs& a, hipStream_t stream) {
  const Kv8Cache& c = a.c;
  kv8_select_kernel<<<dim3((unsigned)c.R, (unsigned)c.H), kSelThreads, 0, stream>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((a.budget + c.B - 1) / c.B), (unsigned)c.H, (unsigned)c.R * 2);
  kv8_copy_kernel<<<grid, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace helm
