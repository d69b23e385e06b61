// Rotary positions with several axes, and the store of new keys and values into
// their pages: one pass over q, k and v.
//
// The angle of pair j at position x is x * inv_freq[j].  Only its fraction of a turn
// matters, so the frequency is held as F = frac(inv_freq / 2 pi) * 2^64, formed from
// the float's 24-bit significand and 96 bits of 1 / (2 pi) in integers (within two units
// below 2^32: one for the digits left out, one for the bits shifted out), and x * F mod
// 2^64 is the angle in units of 2^-64 turns whatever x: at a 32-bit position it is off by
// at most 2^-32 turns, where a float32 product is off by 10^-2 radians at 128K.  Its upper
// 32 bits, rounded (2^-33) and signed, go through sincospif as a float32 (up to 2^-26 turns
// next to a half): 2^-26 + 2^-31 turns in all.
//
// A thread keeps one piece of every token's row -- 16 channels of one head: 8 pairs, or
// 16 channels copied; two 16-byte loads and stores -- so all index arithmetic is done
// once, and passes over the block's tokens, four in flight.  The tokens' angles go to
// shared memory once per block and serve every head.  Bound: HBM, (2 HQ + 4 H) D * 2
// bytes per token.  Measured: 8,200 tokens of 32 + 8 heads of 128 (202 MB) 33.6 us, 6.0
// TB/s; 16 tokens of 32 + 4 heads of 256 2.3 us.
#include "rope.cuh"

namespace tpk {

constexpr int kRopeThreads = 256;  // at most
constexpr int kRopePairs = 1024;   // angles a block holds: tokens * rot / 2
constexpr int kRopeTokens = 8;     // tokens of a block, at most (4: 39.1 us, 8: 36.5, 16: 40.9 at 8200 tokens)
constexpr int kRopeUnroll = 4;

template <typename T, bool kPairs>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p, int per, int tasks,
                                                            int passes) {
  // (cos, sin) of two pairs, [token][pair / 2 mod 4][pair / 8]: the lanes of a head read
  // neighbours
  __shared__ float4 turn[kRopePairs / 2];
  __shared__ int64_t place[kRopeTokens];
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x / passes * per, nt = min(per, p.n_tokens - t0);
  const int half = p.rot >> 1, pieces = p.D >> 4;
  const int kheads = p.k ? p.H : 0;

  // ---- this thread's piece
  const int task = blockIdx.x % passes * blockDim.x + tid;
  const bool mine = task < tasks;
  const int head = task / pieces, j = task - head * pieces;
  const bool query = head < p.HQ, key = !query && head < p.HQ + kheads;
  const bool turned = (query || key) && 16 * j < p.rot;
  const int ca = (kPairs || !turned) ? 16 * j : 8 * j;
  const int cb = (kPairs || !turned) ? 16 * j + 8 : half + 8 * j;
  const int h = query ? head : key ? head - p.HQ : head - p.HQ - kheads;
  const int64_t stride = query ? p.q_stride : key ? p.k_stride : p.v_stride;
  const uint16_t* src = (query ? p.q : key ? p.k : p.v) + (mine ? t0 * stride + h * p.D : 0);
  uint4 a[kRopeUnroll], b[kRopeUnroll];
  auto load = [&](int t) {
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u)
      if (mine && t + u < nt) {
        a[u] = *reinterpret_cast<const uint4*>(src + (t + u) * stride + ca);
        b[u] = *reinterpret_cast<const uint4*>(src + (t + u) * stride + cb);
      }
  };
  wait_before();
  load(0);

  // ---- the tokens' angles and places
  for (int i = tid; i < nt * half; i += blockDim.x) {
    const int t = i / half, x = i - t * half;
    const int64_t pos = p.positions[(int64_t)p.axis_of[x] * p.n_tokens + t0 + t];
    const float2 cs = turned_by(p.inv_freq[x], pos);
    reinterpret_cast<float2*>(turn + t * (half >> 1) + (x >> 1 & 3) * (half >> 3) + (x >> 3))[x & 1] = cs;
  }
  if (tid < nt) {
    const int64_t slot = p.slot_map ? p.slot_map[t0 + tid] : 0;
    const bool past = p.slot_map && slot >= p.slot_limit;
    if (past) atomicOr(p.status, kStatusBadSlot);
    place[tid] = past ? -1 : slot;
  }
  __syncthreads();
  if (!mine) return;

  uint16_t* const dst = query ? p.q_out + t0 * p.q_out_stride + h * p.D : key ? p.k_pool : p.v_pool;
  for (int t = 0; t < nt; t += kRopeUnroll) {
    if (t > 0) load(t);
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      if (t + u >= nt) break;
      const int64_t slot = place[t + u];
      if (slot < 0) continue;  // padding
      if (turned) {
        uint32_t* wa = reinterpret_cast<uint32_t*>(&a[u]);
        uint32_t* wb = reinterpret_cast<uint32_t*>(&b[u]);
        const float4* cs = turn + (t + u) * (half >> 1) + j;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 e = cs[k * (half >> 3)];  // pairs 8 j + 2 k and the next
          if (kPairs) {
            uint32_t* w = k < 2 ? wa + 2 * k : wb + 2 * k - 4;
            const float2 x = T::unpack(w[0]), y = T::unpack(w[1]);
            w[0] = T::pack(x.x * e.x - x.y * e.y, x.y * e.x + x.x * e.y);
            w[1] = T::pack(y.x * e.z - y.y * e.w, y.y * e.z + y.x * e.w);
          } else {
            const float2 x = T::unpack(wa[k]), y = T::unpack(wb[k]);
            wa[k] = T::pack(x.x * e.x - y.x * e.y, x.y * e.z - y.y * e.w);
            wb[k] = T::pack(y.x * e.x + x.x * e.y, y.y * e.z + x.y * e.w);
          }
        }
      }
      uint16_t* to = query ? dst + (t + u) * p.q_out_stride
                           : dst + (((slot >> 6) * p.H + h) * kPageTokens + (slot & 63)) * (int64_t)p.D;
      *reinterpret_cast<uint4*>(to + ca) = a[u];
      *reinterpret_cast<uint4*>(to + cb) = b[u];
    }
  }
}

cudaError_t launch_rope(const RopeParams& p, int dtype, int interleaved, cudaStream_t stream) {
  const int tasks = (p.HQ + (p.k ? 2 * p.H : 0)) * (p.D / 16);
  // equal passes over a row's pieces, in whole warps
  const int passes = (tasks + kRopeThreads - 1) / kRopeThreads;
  const int threads = ((tasks + passes - 1) / passes + 31) / 32 * 32;
  // tokens of a block: as many as leave every SM eight blocks, up to what shared memory
  // holds; one where the tokens hardly fill the device
  int per = (int)min((int64_t)kRopeTokens, (int64_t)p.n_tokens * passes / (8 * 152));
  if (p.rot > 0) per = min(per, 2 * kRopePairs / p.rot);
  per = max(1, per);
  const int blocks = ((p.n_tokens - 1) / per + 1) * passes;
  auto kernel = dtype == 0 ? (interleaved ? rope_kernel<Bf16, true> : rope_kernel<Bf16, false>)
                           : (interleaved ? rope_kernel<F16, true> : rope_kernel<F16, false>);
  return launch_early(kernel, blocks, threads, 0, stream, p, per, tasks, passes);
}

}  // namespace tpk
