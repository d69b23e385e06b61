// Norms of query and key heads, rotary positions and the store of new keys and values into
// their pages: one pass over q, k and v.
//
// A head x becomes y_c = x_c w_c / sqrt(sum_c x_c^2 / D + eps), its channels then turn in pairs
// as in kv_rope.cu.  A thread keeps one piece of every token's row: two chunks of 8 channels of one
// head, chosen so that neighbouring threads have neighbouring chunks and both channels of a pair
// are in one thread.  (Two chunks side by side instead, 7,001 tokens of 32 + 8 heads of 256: 77 us.)
// The D / 16 threads of a head lie side by side in a warp, so the sum of squares is a few shuffles
// over what they hold already, and each row is read and written once.
//
// Bound: HBM, (2 HQ + 4 H) D * 2 bytes per token.  A thread's work on a token is a chain (squares,
// shuffles, root, products), and between its tokens little would be in flight: so the rows of all
// of a block's tokens are asked for at the start, by asynchronous copies into places of shared
// memory that only the asking thread reads, without barriers, while the angles are formed.  (By
// loads into registers, one to four tokens ahead, the same prompt took 77 us and more.)  After
// that instructions count: the two floats of a word run as one packed operation, and the shuffles
// have their number and their lanes fixed at compile time.
// Measured: 7,001 tokens of 32 + 8 heads of 256, half of each rotated (287 MB), 45.1 us, 6.4 TB/s;
// 8,200 of 32 + 8 heads of 128 (202 MB) 36.5 us, 5.5 TB/s; 48 tokens 2.1 us.
#include "rope.cuh"

namespace tpk {

// 8,200 tokens of 32 + 8 heads of 128, 7,001 of 32 + 8 heads of 256: 256 threads 36.4 and 49.4 us, 320
// 36.5 and 45.1, 512 38.4 and 45.0, 640 37.5 and 56.6 (equal passes of whole warps each).  Two tokens
// a block took a third more time than four, six a twentieth more (in an earlier form).
constexpr int kNormThreads = 320;  // at most
constexpr int kNormTokens = 4;     // of a block, at most
constexpr int kNormPairs = 1024;  // angles a block holds: tokens * rot / 2

__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All groups but the last `left` have landed, for this thread.
__device__ __forceinline__ void copies_landed(int left) {
  static_assert(kNormTokens == 4, "cases");
  switch (left) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
  }
}

template <typename T>
__device__ __forceinline__ uint64_t widen(uint32_t w) {
  const float2 x = T::unpack(w);
  return pair(x.x, x.y);
}
template <typename T>
__device__ __forceinline__ uint32_t narrow(uint64_t v) {
  const float2 x = unpair(v);
  return T::pack(x.x, x.y);
}

// One over the root of a head's mean square, from 8 pairs of channels a thread and kPieces neighbouring
// threads of a converged warp.  Where the squares leave float32's range (bfloat16 has values past
// 2^60 and below 2^-50) the channels are scaled first, by a power of two, for the sum and for the
// caller.
template <int kPieces>
__device__ __forceinline__ float inverse_root(uint64_t (&x)[8], float eps) {
  auto mean = [&] {
    uint64_t s[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k & 1] = fma2(x[k], x[k], s[k & 1]);
    const float2 both = unpair(add2(s[0], s[1]));
    float sum = both.x + both.y;
#pragma unroll
    for (int d = kPieces >> 1; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    return sum * (1.f / (16 * kPieces));
  };
  float m = mean() + eps;
  const bool off = !(m < 0x1p120f) || m < 0x1p-100f;
  if (__any_sync(0xffffffffu, off)) {
    const float c = !off ? 1.f : m < 1.f ? 0x1p100f : 0x1p-70f;
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = mul2(x[k], pair(c, c));
    m = mean() + eps * c * c;
  }
  return rsqrtf(m);
}

template <typename T, int kPieces, bool kPairs>
__global__ void __launch_bounds__(kNormThreads) norm_rope_kernel(const __grid_constant__ RopeParams p, int per, int tasks,
                                                                 int passes) {
  constexpr int D = 16 * kPieces;
  extern __shared__ uint4 rows[];  // [token][half of a piece][thread]
  // (cos, sin) of two pairs: [token][pair / 2 mod 4][pair / 8], or for neighbouring pairs
  // [token][pair / 2 mod 2][pair / 4]: the lanes of a head read neighbours
  __shared__ float4 turn[kNormPairs / 2];
  __shared__ int64_t place[kNormTokens];
  const int tid = threadIdx.x, threads = blockDim.x;
  const int t0 = blockIdx.x / passes * per, nt = min(per, p.n_tokens - t0);
  const int half = p.rot >> 1;
  const int kheads = p.k ? p.H : 0;

  // ---- this thread's piece
  const int task = blockIdx.x % passes * threads + tid;
  const bool mine = task < tasks;
  const int head = task / kPieces, j = task % kPieces;
  const bool query = head < p.HQ, key = !query && head < p.HQ + kheads;
  const bool normed = query || key;
  // its chunks: halves of the rotated channels, and of the others; or of all
  const bool front = !kPairs && 16 * j < p.rot;
  const int from = kPairs || front ? 0 : p.rot, span = kPairs ? D : front ? p.rot : D - p.rot;
  const int ca = from + 8 * (j - (from >> 4)), cb = ca + (span >> 1);
  const bool turned_a = normed && ca < p.rot, turned_b = normed && cb < p.rot;
  const int h = query ? head : key ? head - p.HQ : head - p.HQ - kheads;
  wait_before();
  // What the angles and places are made of is asked for before the rows: behind them it would arrive
  // with the last of them (8,200 tokens of 32 + 8 heads of 128: 43.1 us behind, 37.3 before).
  const int angles = nt * half;
  auto load_angle = [&](int i, float& f, int& pos) {
    const int t = i / half, x = i - t * half;
    f = p.inv_freq[x];
    pos = p.positions[(int64_t)p.axis_of[x] * p.n_tokens + t0 + t];
  };
  float freq = 0.f;
  int pos = 0;
  int64_t slot = 0;
  if (tid < angles) load_angle(tid, freq, pos);
  if (tid < nt && p.slot_map) slot = p.slot_map[t0 + tid];
  const uint16_t* const weight = mine && normed ? (query ? p.q_weight : p.k_weight) : nullptr;
  uint4 wa = make_uint4(0, 0, 0, 0), wb = wa;
  if (weight) {
    wa = *reinterpret_cast<const uint4*>(weight + ca);
    wb = *reinterpret_cast<const uint4*>(weight + cb);
  }
  if (mine) {
    const int64_t stride = query ? p.q_stride : key ? p.k_stride : p.v_stride;
    const uint16_t* src = (query ? p.q : key ? p.k : p.v) + t0 * stride + h * D;
    for (int t = 0; t < nt; ++t, src += stride) {
      copy_async16(smem_u32(rows + 2 * t * threads + tid), src + ca);
      copy_async16(smem_u32(rows + (2 * t + 1) * threads + tid), src + cb);
      copies_end();
    }
  }

  // ---- the tokens' angles and places
  for (int i = tid; i < angles; i += threads) {
    if (i != tid) load_angle(i, freq, pos);
    const int t = i / half, x = i - t * half;
    const int to = kPairs ? (x >> 1 & 1) * (half >> 2) + (x >> 2) : (x >> 1 & 3) * (half >> 3) + (x >> 3);
    reinterpret_cast<float2*>(turn + t * (half >> 1) + to)[x & 1] = turned_by(freq, pos);
  }
  if (tid < nt) {
    const bool past = p.slot_map && slot >= p.slot_limit;
    if (past) atomicOr(p.status, kStatusBadSlot);
    place[tid] = past ? -1 : slot;
  }
  __syncthreads();
  uint64_t factor[8];  // of this thread's channels
#pragma unroll
  for (int k = 0; k < 8; ++k)
    factor[k] = weight ? widen<T>(reinterpret_cast<const uint32_t*>(k < 4 ? &wa : &wb)[k & 3]) : pair(1.f, 1.f);

  uint16_t* const dst = query ? p.q_out + t0 * p.q_out_stride + h * D : key ? p.k_pool : p.v_pool;
  for (int t = 0; t < nt; ++t) {
    copies_landed(nt - 1 - t);
    const int64_t slot = place[t];
    if (slot < 0) continue;  // padding
    uint32_t w[8];
    *reinterpret_cast<uint4*>(w) = rows[2 * t * threads + tid];
    *reinterpret_cast<uint4*>(w + 4) = rows[(2 * t + 1) * threads + tid];
    uint64_t x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = widen<T>(w[k]);
    const float root = inverse_root<kPieces>(x, p.eps);
    if (normed) {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = mul2(mul2(x[k], pair(root, root)), factor[k]);
      const float4* cs = turn + t * (half >> 1);
      if (kPairs) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          if (!(y == 0 ? turned_a : turned_b)) continue;
#pragma unroll
          for (int k = 0; k < 2; ++k) {  // two pairs
            const float4 e = cs[k * (half >> 2) + ((y == 0 ? ca : cb) >> 3)];
            const float2 u = unpair(x[4 * y + 2 * k]), v = unpair(x[4 * y + 2 * k + 1]);
            x[4 * y + 2 * k] = pair(u.x * e.x - u.y * e.y, u.y * e.x + u.x * e.y);
            x[4 * y + 2 * k + 1] = pair(v.x * e.z - v.y * e.w, v.y * e.z + v.x * e.w);
          }
        }
      } else if (turned_a) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 e = cs[k * (half >> 3) + j];
          const uint64_t cos = pair(e.x, e.z), a = x[k];
          x[k] = fma2(a, cos, mul2(x[k + 4], pair(-e.y, -e.w)));
          x[k + 4] = fma2(x[k + 4], cos, mul2(a, pair(e.y, e.w)));
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = narrow<T>(x[k]);
    }
    if (!mine) continue;
    uint16_t* to = query ? dst + t * p.q_out_stride
                         : dst + (((slot >> 6) * p.H + h) * kPageTokens + (slot & 63)) * D;
    *reinterpret_cast<uint4*>(to + ca) = *reinterpret_cast<uint4*>(w);
    *reinterpret_cast<uint4*>(to + cb) = *reinterpret_cast<uint4*>(w + 4);
  }
}

template <typename T, int kPieces, bool kPairs>
static cudaError_t launch_t(const RopeParams& p, cudaStream_t stream) {
  static DeviceOnce once;
  const cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(norm_rope_kernel<T, kPieces, kPairs>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kNormThreads * kNormTokens * 32);
  });
  if (e != cudaSuccess) return e;
  const int tasks = (p.HQ + (p.k ? 2 * p.H : 0)) * kPieces;
  // equal passes over a row's pieces, in whole warps
  const int passes = (tasks + kNormThreads - 1) / kNormThreads;
  const int threads = ((tasks + passes - 1) / passes + 31) / 32 * 32;
  // tokens of a block: as many as leave every SM four blocks; one where the tokens hardly fill the
  // device
  int per = (int)min((int64_t)kNormTokens, (int64_t)p.n_tokens * passes / (4 * 152));
  if (p.rot > 0) per = min(per, 2 * kNormPairs / p.rot);
  per = max(1, per);
  const int blocks = ((p.n_tokens - 1) / per + 1) * passes;
  return launch_early(norm_rope_kernel<T, kPieces, kPairs>, blocks, threads, (size_t)threads * per * 32, stream, p, per, tasks,
                      passes);
}

template <typename T, int kPieces>
static cudaError_t launch_pairs(const RopeParams& p, int interleaved, cudaStream_t stream) {
  return interleaved ? launch_t<T, kPieces, true>(p, stream) : launch_t<T, kPieces, false>(p, stream);
}

template <typename T>
static cudaError_t launch_dim(const RopeParams& p, int interleaved, cudaStream_t stream) {
  return p.D == 64 ? launch_pairs<T, 4>(p, interleaved, stream) : p.D == 128 ? launch_pairs<T, 8>(p, interleaved, stream)
                                                                             : launch_pairs<T, 16>(p, interleaved, stream);
}

cudaError_t launch_norm_rope(const RopeParams& p, int dtype, int interleaved, cudaStream_t stream) {
  return dtype == 0 ? launch_dim<Bf16>(p, interleaved, stream) : launch_dim<F16>(p, interleaved, stream);
}

}  // namespace tpk
