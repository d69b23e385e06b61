// Rotary positions with several axes, and the store of new keys and values into
// their pages: one pass over q, k and v.
//
// The angle of pair j at position x is x * inv_freq[j].  Only its fraction of a turn
// matters, so the frequency is held as F = frac(inv_freq / 2 pi) * 2^64, formed from
// the float's 24-bit significand and 96 bits of 1 / (2 pi) in integers (within one
// unit), and x * F mod 2^64 is the angle in units of 2^-64 turns whatever x: at a
// 32-bit position it is off by at most 2^-33 turns, where a float32 product is off by
// 10^-2 radians at 128K.  Its upper 32 bits, signed, go through sincospif.
//
// A block takes `per` tokens: their angles go to shared memory once and serve every
// head.  A task is 16 channels of one head (8 pairs, or 16 channels copied), two
// 16-byte loads and stores.  Bound: HBM, (2 HQ + 4 H) D * 2 bytes per token.
#include "paged.cuh"

namespace tpk {

constexpr int kRopeThreads = 256;
constexpr int kRopePairs = 256;  // angles a block holds: per * rot / 2
constexpr int kRopeUnroll = 4;

// frac(f / (2 pi)) in units of 2^-64 turns.
__device__ __forceinline__ uint64_t turns64(float f) {
  const uint32_t w = __float_as_uint(f);
  const int e = (w >> 23) & 0xff;
  const uint32_t m = (w & 0x7fffff) | (e ? 0x800000u : 0);
  // 1 / (2 pi) * 2^96
  const unsigned __int128 c = ((unsigned __int128)0x28be60dbu << 64) | 0x9391054a7f09d5f4ull;
  const int shift = 182 - (e ? e : 1);  // f = m 2^(e - 150), so F = m c 2^(e - 150) 2^(64 - 96)
  const unsigned __int128 x = m * c;
  uint64_t t;
  if (shift >= 128) t = 0;
  else if (shift >= 0) t = (uint64_t)(x >> shift);
  else t = shift > -64 ? (uint64_t)(x << -shift) : 0;
  return (w >> 31) ? 0 - t : t;
}

struct Two {
  uint4 a, b;
};

template <typename T, bool kPairs>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p, int per, int tasks,
                                                            int blocks16) {
  __shared__ float2 turn[kRopePairs];  // (cos, sin) of [token][pair]
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * per, nt = min(per, p.n_tokens - t0);
  const int half = p.rot >> 1, rot16 = p.rot >> 4;
  const int kheads = p.k ? p.H : 0;
  const int total = nt * tasks;

  // task -> token (within the block), head, and its two 8-channel pieces
  auto split = [&](int i, int& t, int& head, int& j, int& ca, int& cb) {
    t = i / tasks;
    const int r = i - t * tasks;
    head = r / blocks16;
    j = r - head * blocks16;
    const bool turned = j < rot16 && head < p.HQ + kheads;
    ca = (kPairs || !turned) ? 16 * j : 8 * j;
    cb = (kPairs || !turned) ? 16 * j + 8 : half + 8 * j;
    return turned;
  };
  auto load = [&](int i) {
    Two v;
    int t, head, j, ca, cb;
    split(i, t, head, j, ca, cb);
    const int64_t row = t0 + t;
    const uint16_t* src = head < p.HQ ? p.q + row * p.q_stride + head * p.D
                          : head < p.HQ + kheads ? p.k + row * p.k_stride + (head - p.HQ) * p.D
                                                 : p.v + row * p.v_stride + (head - p.HQ - kheads) * p.D;
    v.a = *reinterpret_cast<const uint4*>(src + ca);
    v.b = *reinterpret_cast<const uint4*>(src + cb);
    return v;
  };

  Two v[kRopeUnroll];
#pragma unroll
  for (int u = 0; u < kRopeUnroll; ++u)
    if (tid + u * kRopeThreads < total) v[u] = load(tid + u * kRopeThreads);
  for (int i = tid; i < nt * half; i += kRopeThreads) {
    const int t = i / half, j = i - t * half;
    const int64_t x = p.positions[(int64_t)p.axis_of[j] * p.n_tokens + t0 + t];
    const uint64_t a = turns64(p.inv_freq[j]) * (uint64_t)x;
    float s, c;
    sincospif((float)(int32_t)((a + 0x80000000u) >> 32) * 0x1p-31f, &s, &c);  // of pi * (2 * turns)
    turn[i] = make_float2(c, s);
  }
  __syncthreads();

  for (int i0 = tid; i0 < total; i0 += kRopeUnroll * kRopeThreads) {
    if (i0 != tid) {
#pragma unroll
      for (int u = 0; u < kRopeUnroll; ++u)
        if (i0 + u * kRopeThreads < total) v[u] = load(i0 + u * kRopeThreads);
    }
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      const int i = i0 + u * kRopeThreads;
      if (i >= total) break;
      int t, head, j, ca, cb;
      const bool turned = split(i, t, head, j, ca, cb);
      const int64_t slot = p.slot_map ? p.slot_map[t0 + t] : 0;
      if (slot < 0) continue;  // padding
      if (p.slot_map && slot >= p.slot_limit) {
        atomicOr(p.status, kStatusBadSlot);
        continue;
      }
      uint4 a = v[u].a, b = v[u].b;
      if (turned) {
        uint32_t* wa = reinterpret_cast<uint32_t*>(&a);
        uint32_t* wb = reinterpret_cast<uint32_t*>(&b);
        const float2* cs = turn + t * half + 8 * j;
        if (kPairs) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 x = T::unpack(wa[k]), y = T::unpack(wb[k]);
            const float2 e = cs[k], f = cs[k + 4];
            wa[k] = T::pack(x.x * e.x - x.y * e.y, x.y * e.x + x.x * e.y);
            wb[k] = T::pack(y.x * f.x - y.y * f.y, y.y * f.x + y.x * f.y);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 x = T::unpack(wa[k]), y = T::unpack(wb[k]);
            const float2 e = cs[2 * k], f = cs[2 * k + 1];
            wa[k] = T::pack(x.x * e.x - y.x * e.y, x.y * f.x - y.y * f.y);
            wb[k] = T::pack(y.x * e.x + x.x * e.y, y.y * f.x + x.y * f.y);
          }
        }
      }
      uint16_t* dst;
      if (head < p.HQ) {
        dst = p.q_out + (t0 + t) * p.q_out_stride + head * p.D;
      } else {
        const bool key = head < p.HQ + kheads;
        const int h = head - p.HQ - (key ? 0 : kheads);
        dst = (key ? p.k_pool : p.v_pool) + (((slot >> 6) * p.H + h) * kPageTokens + (slot & 63)) * (int64_t)p.D;
      }
      *reinterpret_cast<uint4*>(dst + ca) = a;
      *reinterpret_cast<uint4*>(dst + cb) = b;
    }
  }
}

cudaError_t launch_rope(const RopeParams& p, int dtype, int interleaved, cudaStream_t stream) {
  const int blocks16 = p.D / 16;
  const int tasks = (p.HQ + (p.k ? 2 * p.H : 0)) * blocks16;
  // tokens per block: six tasks per thread where there are many tokens (loads in
  // flight), one where the tokens hardly fill the device
  int per = max(1, min(8, 6 * kRopeThreads / tasks));
  if (p.rot > 0) per = min(per, 2 * kRopePairs / p.rot);
  per = max(1, min(per, p.n_tokens / 304));
  const int blocks = (p.n_tokens + per - 1) / per;
  if (dtype == 0) {
    if (interleaved) rope_kernel<Bf16, true><<<blocks, kRopeThreads, 0, stream>>>(p, per, tasks, blocks16);
    else rope_kernel<Bf16, false><<<blocks, kRopeThreads, 0, stream>>>(p, per, tasks, blocks16);
  } else {
    if (interleaved) rope_kernel<F16, true><<<blocks, kRopeThreads, 0, stream>>>(p, per, tasks, blocks16);
    else rope_kernel<F16, false><<<blocks, kRopeThreads, 0, stream>>>(p, per, tasks, blocks16);
  }
  return cudaGetLastError();
}

}  // namespace tpk
