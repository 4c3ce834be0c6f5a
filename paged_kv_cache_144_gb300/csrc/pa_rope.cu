// pa_rope.cu - rotary positions of a step's queries and keys fused with the
// cache write of its keys and values.
//
// Angles: pa_rope.cuh.
//
// Work: a CTA takes kTokens tokens and a slice of their heads (a few tokens
// alone would not fill the device: the heads are then spread over more CTAs).
// Its threads move 8 elements (16 bytes) at a time: a unit is one 16-byte chunk
// of a head (interleaved pairs lie inside it) or, in the half layout, the two
// chunks that hold both halves of 8 pairs, so one thread reads and writes both
// elements of every pair it turns and q may be turned in place.  The loads of a
// thread's first units are on their way before the tokens' angles are computed
// (once per CTA, in shared memory).
//
// What bounds it: memory traffic.  8192 tokens of 32 + 2 x 8 heads of 128, bf16:
// 36 us, 5.6 TB/s of the 201 MB read and written (82 % of a plain copy); to FP8
// caches with half the columns turned, 2048 tokens: 12.6 us.  32 tokens: 4.4 us,
// the latency of a launch, the tokens' loads and one store.
#include "pa_rope.cuh"

namespace pa {
namespace {

// kHalfAny: half layout whose rotary_dim / 2 is no multiple of 8, so the second halves are not
// 16-byte chunks: one pair (or one passed column) per unit, 2-byte accesses.
enum Layout { kInterleaved = 0, kHalf = 1, kHalfAny = 2 };

// (8192 tokens of 32 + 2 x 8 heads, events around the call: 64 / 128 / 256 / 512 threads 46 / 44 / 49 / 66 us, 1 / 2 / 4 units in
// flight 44.5 / 44 / 48 us)
constexpr int kThreads = 128;
constexpr int kTokens = 2;
constexpr int kUnroll = 2;           // units whose loads a thread has in flight
constexpr unsigned kFillCtas = 1024;  // CTAs below which a token's heads are spread over several

// Unit x of a CTA's tokens.
struct Unit {
  int t;      // token of the CTA
  int which;  // 0 = q, 1 = k, 2 = v
  int head;
  int u;      // chunk, or pair of chunks, of the head
};

// turned: units of a turned head; magic = ceil(2^32 / turned) (x / turned = umulhi(x, magic) while x * turned < 2^32)
__device__ __forceinline__ Unit unit_of(int x, int units, int turned, uint32_t magic, int Hq, int Hk, int copied) {
  Unit n;
  n.t = x >= units ? 1 : 0;
  x -= n.t * units;
  const int both = (Hq + Hk) * turned;
  if (x < both) {
    n.head = static_cast<int>(__umulhi(static_cast<uint32_t>(x), magic));
    n.u = x - n.head * turned;
    n.which = n.head < Hq ? 0 : 1;
    n.head -= n.which ? Hq : 0;
  } else {
    x -= both;
    n.head = x / copied;
    n.u = x - n.head * copied;
    n.which = 2;
  }
  return n;
}

template <typename SRC, int MODE, int D, int LAYOUT>
__global__ void __launch_bounds__(kThreads) rope_and_cache_kernel(const RopeArgs a, const uint32_t magic) {
  griddep_launch_dependents();
  griddep_wait();
  static_assert(kTokens == 2, "unit_of");
  __shared__ float2 cs[kTokens][D / 2];
  __shared__ int64_t rows0[kTokens];
  const ReshapeArgs& w = a.w;
  const int half = a.rotary_dim >> 1;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kTokens;
  const int nt = static_cast<int>(min(static_cast<int64_t>(kTokens), w.num_tokens - n0));
  const int Hq = a.num_heads, Hk = w.num_kv_heads;
  const int turned = LAYOUT == kInterleaved ? D / 8
                     : LAYOUT == kHalf      ? (half >> 3) + (D - a.rotary_dim) / 8
                                            : half + (D - a.rotary_dim);
  constexpr int copied = D / 8;
  const int units = (Hq + Hk) * turned + Hk * copied;
  constexpr int kvb = MODE == kCopy ? 2 : 1;
  constexpr int U = LAYOUT == kHalfAny ? 1 : kUnroll;

  const int total = nt * units;
  const int per = ((total + static_cast<int>(gridDim.y) - 1) / static_cast<int>(gridDim.y) + kThreads - 1) / kThreads * kThreads;
  const int begin = static_cast<int>(blockIdx.y) * per, end = min(total, begin + per);

  auto src_row = [&](const Unit& n) -> const uint8_t* {
    const int64_t tok = n0 + n.t;
    const void* base = n.which == 0 ? a.q : n.which == 1 ? w.k : w.v;
    const int64_t stride = n.which == 0 ? a.q_stride : n.which == 1 ? w.k_stride : w.v_stride;
    return static_cast<const uint8_t*>(base) + (tok * stride + static_cast<int64_t>(n.head) * D) * 2;
  };
  // first column of a unit, and of its second chunk (half layout: the other halves of its pairs), or -1
  auto columns = [&](const Unit& n, int* second) -> int {
    *second = -1;
    if (n.which == 2 || LAYOUT == kInterleaved) return 8 * n.u;
    if (LAYOUT == kHalf && n.u < (half >> 3)) {
      *second = half + 8 * n.u;
      return 8 * n.u;
    }
    return a.rotary_dim + 8 * (n.u - (half >> 3));
  };

  bool angles = false;
  for (int x0 = begin; x0 < end || !angles; x0 += kThreads * U) {
    uint4 lo[U], hi[U];
    Unit n[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int x = x0 + k * kThreads + static_cast<int>(threadIdx.x);
      n[k].t = -1;
      if (x < end) {
        n[k] = unit_of(x, units, turned, magic, Hq, Hk, copied);
        if (LAYOUT != kHalfAny || n[k].which == 2) {
          const uint8_t* src = src_row(n[k]);
          int second;
          const int c = columns(n[k], &second);
          lo[k] = *reinterpret_cast<const uint4*>(src + 2 * c);
          if (second >= 0) hi[k] = *reinterpret_cast<const uint4*>(src + 2 * second);
        }
      }
    }
    if (!angles) {
      for (int x = threadIdx.x; x < nt * half; x += kThreads) {
        const int t = x >= half ? 1 : 0, i = x - t * half;
        cs[t][i] = rope_turn(__ldg(a.inv_freq + i), a.positions[n0 + t], a.rope_scale);
      }
      if (threadIdx.x < nt) {
        const int64_t slot = w.slot_mapping[n0 + threadIdx.x];
        int64_t row = -1;  // cache row of KV head 0
        if (slot >= w.num_blocks * w.block_size) {
          if (blockIdx.y == 0) raise_error(w.err, PA_DEVERR_SLOT);
        } else if (slot >= 0) {
          const int64_t blk = slot / w.block_size;
          row = blk * Hk * w.block_size + (slot - blk * w.block_size);
        }
        rows0[threadIdx.x] = row;
      }
      __syncthreads();
      angles = true;
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (n[k].t < 0) continue;
      const int64_t row0 = rows0[n[k].t];
      if (row0 < 0) continue;  // padding token, or outside the pool
      const int which = n[k].which, head = n[k].head, u = n[k].u;
      Dst d;
      d.cache = which != 0;
      d.inv = 1.f;
      d.zp = 0;
      if (which == 0) {
        d.row = static_cast<uint8_t*>(a.q_out) + ((n0 + n[k].t) * a.q_out_stride + static_cast<int64_t>(head) * D) * 2;
      } else {
        d.row = static_cast<uint8_t*>(which == 1 ? w.k_cache : w.v_cache) +
                (row0 + static_cast<int64_t>(head) * w.block_size) * D * kvb;
        if constexpr (MODE != kCopy) d.inv = __ldg((which == 1 ? w.k_inv_scale : w.v_inv_scale) + head);
        if constexpr (MODE == kToInt8) d.zp = __ldg((which == 1 ? w.k_zero_point : w.v_zero_point) + head);
      }
      const float2* const c2 = cs[n[k].t];
      if (LAYOUT == kHalfAny && which != 2) {
        const uint8_t* src = src_row(n[k]);
        if (u < half) {
          const float2 f = c2[u];
          const float p = load_scalar<SRC>(src, u), q = load_scalar<SRC>(src, half + u);
          store1<SRC, MODE>(d, u, p * f.x - q * f.y);
          store1<SRC, MODE>(d, half + u, q * f.x + p * f.y);
        } else {
          const int c = a.rotary_dim + (u - half);
          store1<SRC, MODE>(d, c, load_scalar<SRC>(src, c));
        }
        continue;
      }
      int second;
      const int c = columns(n[k], &second);
      float p[8];
      widen8<SRC>(lo[k], p);
      if (which != 2) {
        if constexpr (LAYOUT == kInterleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (4 * u + i < half) {
              const float2 f = c2[4 * u + i];
              const float y = p[2 * i], z = p[2 * i + 1];
              p[2 * i] = y * f.x - z * f.y;
              p[2 * i + 1] = z * f.x + y * f.y;
            }
          }
        } else if (second >= 0) {
          float q[8];
          widen8<SRC>(hi[k], q);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 f = c2[8 * u + i];
            const float y = p[i], z = q[i];
            p[i] = y * f.x - z * f.y;
            q[i] = z * f.x + y * f.y;
          }
          store8<SRC, MODE>(d, second, q);
        }
      }
      store8<SRC, MODE>(d, c, p);
    }
  }
}

template <typename SRC, int MODE, int D>
cudaError_t launch_layout(const RopeArgs& a, cudaStream_t stream) {
  const int layout = a.interleaved ? kInterleaved : (a.rotary_dim % 16 == 0 ? kHalf : kHalfAny);
  void (*kern)(RopeArgs, uint32_t) = layout == kInterleaved ? rope_and_cache_kernel<SRC, MODE, D, kInterleaved>
                                     : layout == kHalf      ? rope_and_cache_kernel<SRC, MODE, D, kHalf>
                                                            : rope_and_cache_kernel<SRC, MODE, D, kHalfAny>;
  const int half = a.rotary_dim / 2;
  const int turned = layout == kInterleaved ? D / 8 : layout == kHalf ? half / 8 + (D - a.rotary_dim) / 8 : half + D - a.rotary_dim;
  const uint32_t magic = static_cast<uint32_t>(((uint64_t{1} << 32) + turned - 1) / turned);
  const int units = kTokens * ((a.num_heads + a.w.num_kv_heads) * turned + a.w.num_kv_heads * (D / 8));
  const unsigned gx = static_cast<unsigned>((a.w.num_tokens + kTokens - 1) / kTokens);
  // slices of the heads: about kFillCtas CTAs, none with less than one unit per thread
  unsigned gy = gx < kFillCtas ? kFillCtas / gx : 1;
  const unsigned most = static_cast<unsigned>((units + kThreads - 1) / kThreads);
  gy = gy < most ? gy : most;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(gx, gy);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.w.pdl ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, magic);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename SRC>
cudaError_t launch_src(const RopeArgs& a, cudaStream_t stream) {
  const int mode = a.w.kv_dtype == PA_FP8_E4M3 ? kToFp8 : (a.w.kv_dtype == PA_INT8 ? kToInt8 : kCopy);
  if (a.w.head_dim == 128) {
    if (mode == kToFp8) return launch_layout<SRC, kToFp8, 128>(a, stream);
    if (mode == kToInt8) return launch_layout<SRC, kToInt8, 128>(a, stream);
    return launch_layout<SRC, kCopy, 128>(a, stream);
  }
  if (mode == kToFp8) return launch_layout<SRC, kToFp8, 64>(a, stream);
  if (mode == kToInt8) return launch_layout<SRC, kToInt8, 64>(a, stream);
  return launch_layout<SRC, kCopy, 64>(a, stream);
}

}  // namespace

cudaError_t launch_rope_and_cache(const RopeArgs& a, cudaStream_t stream) {
  (void)cudaGetLastError();
  return a.w.src_dtype == PA_F16 ? launch_src<f16_t>(a, stream) : launch_src<bf16_t>(a, stream);
}

}  // namespace pa
