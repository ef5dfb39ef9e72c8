// rope.hip — rotary positions of queries and keys (helm_rope).
//
// Every head's first rot values are turned pair by pair through
// angle = position * freq[i] (see include/helm_kv.h for the layouts, the
// frequency scalings and the modes).  The operator moves each value once in
// and once out and does 3 flops per value: it is bound by memory, and at a
// few tokens by the launch.
//
// A workgroup takes a few tokens and a range of heads; the (cos, sin) of its
// tokens' pairs are formed once, in LDS, and serve all its heads.  The angle
// is reduced in fp64, as turns = position * freq/(2 pi) less the nearest whole
// number (positions up to 2^31 leave an error under 2e-7 rad), so that cos and
// sin can be fp32 functions of at most half a turn.
#include "internal.hpp"
#include "serve.hpp"

namespace helm {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__bf16>(__bf16 x) { return (float)x; }

// VEC values, at any element alignment.
template <typename T, int VEC>
struct Piece {
  T v[VEC];
};
template <typename T, int VEC>
__device__ __forceinline__ Piece<T, VEC> load_piece(const T* p) {
  Piece<T, VEC> x;
  __builtin_memcpy(&x, p, sizeof x);
  return x;
}
template <typename T, int VEC>
__device__ __forceinline__ void store_piece(T* p, const Piece<T, VEC>& x) {
  __builtin_memcpy(p, &x, sizeof x);
}

// One workgroup: tokens [blockIdx.x * tok, ...), heads blockIdx.y * heads_per
// onwards of the q heads followed by the k heads.  VEC values of a head (or of
// each half of its pairs) are one thread's piece.
template <typename T, int VEC, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeArgs a, RopeTurns f) {
  extern __shared__ float2 cs[];   // [tok][pairs]
  const int P = a.pairs;
  const int64_t t0 = (int64_t)blockIdx.x * a.tok;
  const int nt = (int)min((int64_t)a.tok, a.n_tok - t0);
  for (int e = threadIdx.x; e < nt * P; e += kThreads) {
    const int t = e / P, i = e - t * P;
    const double turns = (double)a.pos[t0 + t] * f.turn[i];
    const float frac = (float)(turns - rint(turns));
    float s, c;
    sincospif(2.0f * frac, &s, &c);
    cs[e] = make_float2(c * a.mag, s * a.mag * a.sign);
  }
  __syncthreads();

  const int h0 = blockIdx.y * a.heads_per;
  const int nh = min(a.heads_per, a.n_q + a.n_k - h0);
  const int turned = INTERLEAVED ? 2 * P / VEC : P / VEC;   // pieces that are turned
  const int pieces = turned + (a.D - 2 * P + VEC - 1) / VEC;
  const int total = nt * nh * pieces;
  for (int e = threadIdx.x; e < total; e += kThreads) {
    const int p = e % pieces, th = e / pieces;
    const int h = h0 + th % nh, t = th / nh;
    const bool is_q = h < a.n_q;
    const int hh = is_q ? h : h - a.n_q;
    const T* x = is_q ? (const T*)a.q + (t0 + t) * a.q_tok + hh * a.q_head
                      : (const T*)a.k + (t0 + t) * a.k_tok + hh * a.k_head;
    T* y = is_q ? (T*)a.out_q + (t0 + t) * a.oq_tok + hh * a.oq_head
                : (T*)a.out_k + (t0 + t) * a.ok_tok + hh * a.ok_head;
    if (p >= turned) {   // past the rotated part
      const int d = 2 * P + (p - turned) * VEC;
      if (d + VEC <= a.D) {
        store_piece<T, VEC>(y + d, load_piece<T, VEC>(x + d));
      } else {
        for (int j = d; j < a.D; ++j) y[j] = x[j];
      }
    } else if constexpr (INTERLEAVED) {
      auto v = load_piece<T, VEC>(x + p * VEC);
#pragma unroll
      for (int j = 0; j < VEC; j += 2) {
        const float2 w = cs[t * P + (p * VEC + j) / 2];
        const float u0 = to_f32<T>(v.v[j]), u1 = to_f32<T>(v.v[j + 1]);
        v.v[j] = (T)(u0 * w.x - u1 * w.y);
        v.v[j + 1] = (T)(u0 * w.y + u1 * w.x);
      }
      store_piece<T, VEC>(y + p * VEC, v);
    } else {
      auto u = load_piece<T, VEC>(x + p * VEC);
      auto v = load_piece<T, VEC>(x + P + p * VEC);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float2 w = cs[t * P + p * VEC + j];
        const float u0 = to_f32<T>(u.v[j]), u1 = to_f32<T>(v.v[j]);
        u.v[j] = (T)(u0 * w.x - u1 * w.y);
        v.v[j] = (T)(u0 * w.y + u1 * w.x);
      }
      store_piece<T, VEC>(y + p * VEC, u);
      store_piece<T, VEC>(y + P + p * VEC, v);
    }
  }
}

template <typename T, int VEC, bool INTERLEAVED>
hipError_t launch(RopeArgs a, const RopeTurns& f, hipStream_t stream) {
  // About 16 pieces a thread at most, and enough workgroups for 256 CUs when
  // there are few tokens: first one token and few heads, then more of both.
  const int heads = a.n_q + a.n_k;
  const int pieces = (INTERLEAVED ? a.D : a.D / 2) / VEC + 1;
  a.heads_per = heads;
  a.tok = 1;
  while (a.heads_per > 1 && a.heads_per * pieces > kThreads &&
         a.n_tok * ((heads + a.heads_per - 1) / a.heads_per) < 1024)
    a.heads_per = (a.heads_per + 1) / 2;
  while (a.tok < 16 && a.tok * heads * pieces < 4 * kThreads && a.n_tok / a.tok > 2048) a.tok *= 2;
  const dim3 grid((unsigned)((a.n_tok + a.tok - 1) / a.tok), (unsigned)((heads + a.heads_per - 1) / a.heads_per));
  rope_kernel<T, VEC, INTERLEAVED><<<grid, kThreads, (size_t)a.tok * a.pairs * sizeof(float2), stream>>>(a, f);
  return hipGetLastError();
}

template <typename T, int VEC>
hipError_t by_layout(const RopeArgs& a, const RopeTurns& f, bool interleaved, hipStream_t stream) {
  // 16-byte pieces where the turned part divides into them, else pair by pair
  if (interleaved)
    return 2 * a.pairs % VEC ? launch<T, 2, true>(a, f, stream) : launch<T, VEC, true>(a, f, stream);
  return a.pairs % VEC ? launch<T, 1, false>(a, f, stream) : launch<T, VEC, false>(a, f, stream);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, const RopeTurns& f, bool interleaved, Dtype dt, hipStream_t stream) {
  return dt == Dtype::BF16 ? by_layout<__bf16, 8>(a, f, interleaved, stream)
                           : by_layout<float, 4>(a, f, interleaved, stream);
}

}  // namespace helm
