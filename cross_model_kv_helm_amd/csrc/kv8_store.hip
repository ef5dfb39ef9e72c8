// kv8_store.hip — new tokens into the 8-bit paged cache (helm_kv8_store).
//
// Per (block, head, K or V): amax = max |x| over the block's new tokens,
// scale = the smallest power of two 2^e with amax <= 448 * 2^e (at least the
// block's own where it held tokens before), code = e4m3(x / scale), and where
// the scale grew the codes held before are taken to it.  Each value is read
// once and one byte is written for it: bound by memory.
//
// One wave owns one block of one head of K or V, so the scale needs neither
// atomics nor barriers and nothing is read that another wave writes; the new
// values stay in registers between finding their size and coding them (of
// blocks over 512 pieces a lane's share is read again, from the caches).  The
// host does not know which blocks the ragged requests touch: request r gets
// floor(n / B) + 2 items, enough for n new tokens at any offset, and the
// surplus ones leave at once.  Finding its block costs a workgroup four loads
// that wait for each other, so where there are many blocks its waves take
// several heads each (a workgroup per head and K|V took 62 us for 37,540
// tokens of 8 heads).
#include "serve.hpp"

namespace helm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// Pieces of 8 values, as loaded.
template <typename T>
struct Piece;
template <>
struct Piece<__bf16> {
  u32x4 w;
  __device__ __forceinline__ float at(int i) const {
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
};
template <>
struct Piece<float> {
  float w[8];
  __device__ __forceinline__ float at(int i) const { return w[i]; }
};

// U pieces a lane: a whole block where it has no more (WHOLE).
template <typename T, int U, bool WHOLE>
__global__ void __launch_bounds__(kThreads) kv8_store_kernel(Kv8StoreArgs a) {
  const Kv8Cache& c = a.c;
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

  const int lane = threadIdx.x & 63;
  const int per = c.D / 8, shift = 31 - __clz(per);   // pieces a token, a power of two
  const int all = cnt * per;
  for (int pair = blockIdx.y * kWaves + (threadIdx.x >> 6); pair < 2 * c.H; pair += gridDim.y * kWaves) {
    const bool is_v = pair >= c.H;
    const int h = is_v ? pair - c.H : pair;
    const int64_t tok = is_v ? a.v_tok : a.k_tok;
    const T* src = (is_v ? (const T*)a.v + h * a.v_head : (const T*)a.k + h * a.k_head) + (c0 + (t0 - start)) * tok;
    const int64_t slab = (int64_t)blk * c.H + h;
    uint8_t* pool = (is_v ? c.v_pool : c.k_pool) + slab * c.B * c.D;
    float* scale = (is_v ? c.v_scale : c.k_scale) + slab;
    const float was = o0 > 0 ? fmaxf(*scale, 0.0f) : 0.0f;   // NaN and negative: no scale, codes that stand for 0

    Piece<T> x[U];
    float amax = 0.0f;
    const auto load = [&](int u0) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int u = u0 + 64 * i + lane;
        x[i] = Piece<T>{};
        if (u < all) __builtin_memcpy(&x[i], src + (u >> shift) * tok + (u & (per - 1)) * 8, sizeof x[i]);
      }
    };
    const auto size = [&]() {
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, kv8_size(x[i].at(j)));
    };
    if constexpr (WHOLE) {
      load(0);
      size();
    } else {
      for (int u0 = 0; u0 < all; u0 += 64 * U) {
        load(u0);
        size();
      }
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
    const float now = fmaxf(kv8_scale_of(amax), was);
    const float inv = 1.0f / now;                       // exact for a power of two
    if (lane == 0) *scale = now;
    if (o0 > 0 && was != now) {
      const float ratio = was * inv;
      for (int u = lane; u < o0 * (c.D / 4); u += 64) {
        uint32_t* p = (uint32_t*)pool + u;
        const f32x4 y = kv8_decode4(was > 0.0f ? *p : 0u);
        *p = kv8_encode4(y[0] * ratio, y[1] * ratio, y[2] * ratio, y[3] * ratio);
      }
    }
    for (int u0 = 0; u0 < all; u0 += 64 * U) {
      if constexpr (!WHOLE) load(u0);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int u = u0 + 64 * i + lane;
        if (u < all)
          *(u32x2*)(pool + (int64_t)o0 * c.D + u * 8) =
              u32x2{kv8_encode4(x[i].at(0) * inv, x[i].at(1) * inv, x[i].at(2) * inv, x[i].at(3) * inv),
                    kv8_encode4(x[i].at(4) * inv, x[i].at(5) * inv, x[i].at(6) * inv, x[i].at(7) * inv)};
      }
    }
    if (!is_v && a.weights)
      for (int u = lane; u < cnt; u += 64) a.weights[slab * c.B + o0 + u] = 0.0f;
  }
}

template <typename T>
void store(const Kv8StoreArgs& a, hipStream_t stream) {
  const Kv8Cache& c = a.c;
  const int64_t items = a.n_tok / c.B + 2 * (int64_t)c.R;
  const int groups = (2 * c.H + kWaves - 1) / kWaves;    // workgroups a block, a wave per head and K|V
  const int64_t fill = 4096 / (items < 1 ? 1 : items);
  const dim3 grid((unsigned)items, (unsigned)(fill >= groups ? groups : fill < 1 ? 1 : fill));
  const int pieces = c.B * (c.D / 8);
  if (pieces <= 128)
    kv8_store_kernel<T, 2, true><<<grid, kThreads, 0, stream>>>(a);
  else if (pieces <= 256)
    kv8_store_kernel<T, 4, true><<<grid, kThreads, 0, stream>>>(a);
  else if (pieces <= 512)
    kv8_store_kernel<T, 8, true><<<grid, kThreads, 0, stream>>>(a);
  else
    kv8_store_kernel<T, 8, false><<<grid, kThreads, 0, stream>>>(a);
}

}  // namespace

hipError_t launch_kv8_store(const Kv8StoreArgs& a, Dtype dt, hipStream_t stream) {
  if (dt == Dtype::BF16)
    store<__bf16>(a, stream);
  else
    store<float>(a, stream);
  return hipGetLastError();
}

}  // namespace helm
