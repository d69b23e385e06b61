// Attention of decoding requests that share a long prefix: each group's queries over its prefix as
// row tiles (cross_tile.cuh), the rest of every request by the decode kernels, and their join.
//
// A group of n requests has n G rows for each KV head, all of which see the prefix: as 128-row tiles
// they read it once (from HBM; tiles of the same group and keys run side by side and find it in L2)
// where n decode calls would read it n times.  What a request does not share is an ordinary decode
// from its own first token on; both leave a maximum, a sum and weighted values, joined here in a fixed
// order: the prefix's parts, then the request's own.  (A log-sum in place of the pair would round the
// sum's logarithm to the maximum's unit: at scores of 2^20, weights off by some hundredths.)
//
// Bound: the tensor cores over the prefixes, HBM over the rest, one after the other.  Measured: 64
// requests behind 32,768 tokens with 30 to 1,500 of their own, 4 x 8 heads of 256, 114 us (cut
// short behind the tiles 70, the decode 107, its fold 108); 13 groups of 1 to 24 behind 300 to 9,000 tokens
// with up to 2,500 of their own, 8 x 5 heads of 128 (491 MB), 115 us (62, 107, 109).
#include "cross_tile.cuh"

namespace tpk {

cudaError_t launch_shared_tiles(const PagedParams& p, int D, int dtype, int tiles, int groups, int splits, cudaStream_t stream) {
  return launch_tiles_of<kSharedPrefix>(p, D, dtype, tiles, groups, splits, stream);
}

// One warp per query row; kJoined parts' values in flight.  Bound: latency and the parts' bytes, which
// are in L2.
template <typename T, int D>
__global__ void __launch_bounds__(256) shared_join_kernel(const SharedJoinParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t rows = (int64_t)p.n_q * p.HQ, r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  wait_before();  // nothing is read before it
  if (r >= rows) return;
  const int b = (int)(r / p.HQ);
  float2 own[D / 64], all[D / 64], v[kJoined][D / 64];
#pragma unroll
  for (int e = 0; e < D / 64; ++e) own[e] = *reinterpret_cast<const float2*>(p.own_o + r * D + e * 64 + 2 * lane);
  const float2 own_ml = p.own_ml[r];
  const bool shares = p.own_begin[b] > 0;
  const int splits = shares ? p.splits : 0;
  float2 all_ml = make_float2(kNone, 0.f);
  if (p.whole_o && shares) {
#pragma unroll
    for (int e = 0; e < D / 64; ++e) all[e] = *reinterpret_cast<const float2*>(p.whole_o + r * D + e * 64 + 2 * lane);
    all_ml = p.whole_ml[r];
  }
  float2 ml = make_float2(kNone, 0.f);
  if (lane < splits) ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * (lane * rows + r));
  auto load = [&](int k0) {
#pragma unroll
    for (int j = 0; j < kJoined; ++j)
      if (k0 + j < splits)
#pragma unroll
        for (int e = 0; e < D / 64; ++e)
          v[j][e] = *reinterpret_cast<const float2*>(p.part_o + ((k0 + j) * rows + r) * D + e * 64 + 2 * lane);
  };
  load(0);
  auto maximum = [](float2 x) { return x.y == 0.f ? kNone : x.x; };
  float M = fmaxf(fmaxf(maximum(ml), maximum(own_ml)), maximum(all_ml));
  for (int k = lane + 32; k < splits; k += 32) {
    const float2 x = *reinterpret_cast<const float2*>(p.part_ml + 2 * (k * rows + r));
    M = fmaxf(M, maximum(x));
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  float L = 0.f, o[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
  auto add = [&](float m, float l, const float2 (&x)[D / 64]) {
    if (l == 0.f) return;
    const float f = exp2f(m - M);  // NaN where no part has a maximum: what sums there are are NaN
    L += f * l;
#pragma unroll
    for (int e = 0; e < D / 64; ++e) {
      o[2 * e] += f * x[e].x;
      o[2 * e + 1] += f * x[e].y;
    }
  };
  for (int k0 = 0; k0 < splits; k0 += kJoined) {
    if (k0 > 0) load(k0);
    if (k0 > 0 && (k0 & 31) == 0 && k0 + lane < splits)
      ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * ((k0 + lane) * rows + r));
#pragma unroll
    for (int j = 0; j < kJoined; ++j) {
      if (k0 + j >= splits) break;
      add(__shfl_sync(0xffffffffu, ml.x, (k0 + j) & 31), __shfl_sync(0xffffffffu, ml.y, (k0 + j) & 31), v[j]);
    }
  }
  add(all_ml.x, all_ml.y, all);
  add(own_ml.x, own_ml.y, own);
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const int64_t at = b * p.o_stride + (r - (int64_t)b * p.HQ) * D;
#pragma unroll
  for (int e = 0; e < D / 64; ++e) {
    const float x = o[2 * e] * inv, y = o[2 * e + 1] * inv;
    const int64_t c = at + e * 64 + 2 * lane;
    if (p.o_f32) *reinterpret_cast<float2*>(static_cast<float*>(p.o) + c) = make_float2(x, y);
    else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + c) = T::pack(x, y);
  }
  if (lane == 0) p.lse[r] = L == 0.f ? kNone : (M + log2f(L)) * kLn2;
}

template <typename T>
static cudaError_t launch_join(const SharedJoinParams& p, int D, cudaStream_t stream) {
  const unsigned blocks = (unsigned)(((int64_t)p.n_q * p.HQ + 7) / 8);
  auto kernel = D == 64 ? shared_join_kernel<T, 64> : D == 128 ? shared_join_kernel<T, 128> : shared_join_kernel<T, 256>;
  return launch_early(kernel, blocks, 256, 0, stream, p);
}

cudaError_t launch_shared_join(const SharedJoinParams& p, int D, int dtype, cudaStream_t stream) {
  return dtype == 0 ? launch_join<Bf16>(p, D, stream) : launch_join<F16>(p, D, stream);
}

}  // namespace tpk
