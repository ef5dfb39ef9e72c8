// kv8_store.hip — new tokens into the 8-bit paged cache (helm_kv8_store).
//
// Per (block, head, K or V): amax = max |x| over the block's new tokens,
// scale = the smallest power of two 2^e with amax <= 448 * 2^e (at least the
// block's own where it held tokens before), code = e4m3(x / scale), and where
// the scale grew the codes held before are taken to it.  Each value is read
// once from HBM (the second reading below comes from the caches) and one byte
// is written for it: bound by memory.
//
// One workgroup owns one block of one head, so the scale needs no atomics and
// nothing is read that another workgroup writes.  The host does not know which
// blocks the ragged requests touch: request r gets floor(n / B) + 2 items,
// enough for n new tokens at any offset, and the surplus ones leave at once.
#include "serve.hpp"

namespace helm {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void load8(const float* p, float* x) { __builtin_memcpy(x, p, 32); }
__device__ __forceinline__ void load8(const __bf16* p, float* x) {
  u32x4 w;
  __builtin_memcpy(&w, p, 16);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) kv8_store_kernel(Kv8StoreArgs a) {
  __shared__ float red[kThreads / 64];
  const Kv8Cache& c = a.c;
  const int h = blockIdx.y;
  const bool is_v = blockIdx.z;
  int64_t base;
  const int r = owner_of(a.cu, c.R, a.n_tok, 1, c.B, 2, blockIdx.x, base);
  const int64_t c0 = cu_at(a.cu, r, a.n_tok), n = cu_at(a.cu, r + 1, a.n_tok) - c0;
  const int64_t start = max(a.start[r], 0);
  const int64_t page = start / c.B + (blockIdx.x - base);
  // tokens [t0, t1) of the request are the new ones of this page
  const int64_t t0 = max(start, page * c.B), t1 = min(min(start + n, (page + 1) * c.B), (int64_t)c.max_len);
  if (n <= 0 || t0 >= t1 || page >= c.max_blocks) return;
  const int blk = c.table[(int64_t)r * c.max_blocks + page];
  if ((uint32_t)blk >= (uint32_t)c.n_blocks) return;
  const int o0 = (int)(t0 - page * c.B), cnt = (int)(t1 - t0);   // slots [o0, o0 + cnt)

  const int64_t tok = is_v ? a.v_tok : a.k_tok;
  const T* src = (is_v ? (const T*)a.v + h * a.v_head : (const T*)a.k + h * a.k_head) + (c0 + (t0 - start)) * tok;
  const int64_t slab = (int64_t)blk * c.H + h;
  uint8_t* pool = (is_v ? c.v_pool : c.k_pool) + slab * c.B * c.D;
  float* scale = (is_v ? c.v_scale : c.k_scale) + slab;

  const int per = c.D / 8;   // pieces of 8 values a token: a power of two
  const int shift = 31 - __clz(per);
  float amax = 0.0f;
  for (int u = threadIdx.x; u < cnt * per; u += kThreads) {
    float x[8];
    load8(src + (u >> shift) * tok + (u & (per - 1)) * 8, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, kv8_size(x[j]));
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = amax;
  const float was = o0 > 0 ? *scale : 0.0f;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) amax = fmaxf(amax, red[w]);
  const float now = fmaxf(kv8_scale_of(amax), was);   // fmaxf: a NaN scale counts as none
  const float inv = 1.0f / now;                       // exact: a power of two (or the caller's own scale)
  if (threadIdx.x == 0) *scale = now;                 // every wave has read it before the barrier

  if (o0 > 0 && was != now) {
    const float ratio = was * inv;
    for (int u = threadIdx.x; u < o0 * (c.D / 4); u += kThreads) {
      uint32_t* p = (uint32_t*)pool + u;
      const f32x4 x = kv8_decode4(*p);
      *p = kv8_encode4(x[0] * ratio, x[1] * ratio, x[2] * ratio, x[3] * ratio);
    }
  }
  for (int u = threadIdx.x; u < cnt * per; u += kThreads) {
    float x[8];
    load8(src + (u >> shift) * tok + (u & (per - 1)) * 8, x);
    const u32x2 w = {kv8_encode4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                     kv8_encode4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv)};
    *(u32x2*)(pool + (int64_t)o0 * c.D + u * 8) = w;
  }
  if (!is_v && a.weights)
    for (int u = threadIdx.x; u < cnt; u += kThreads) a.weights[slab * c.B + o0 + u] = 0.0f;
}

}  // namespace

hipError_t launch_kv8_store(const Kv8StoreArgs& a, Dtype dt, hipStream_t stream) {
  const dim3 grid((unsigned)(a.n_tok / a.c.B + 2 * (int64_t)a.c.R), (unsigned)a.c.H, 2);
  if (dt == Dtype::BF16)
    kv8_store_kernel<__bf16><<<grid, kThreads, 0, stream>>>(a);
  else
    kv8_store_kernel<float><<<grid, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace helm
