// pa_norm.cu - norms of a step's queries and keys for each head, their rotary
// positions and the cache write of its keys and values, in one launch; also
// every write into a 4-bit cache.
//
// Mathematics: a row x of D values becomes x * (sum x^2 / D + eps)^-1/2 * (w +
// offset), its pairs are turned (pa_rope.cuh), all in float32, and the result is
// rounded once to q_out's or the cache's type.  A 4-bit row is stored as codes
// 0 .. 15 between its smallest and largest value (store_int4).
//
// Work: D / 16 threads share a row and hold 16 of its values each, so a norm's
// sum and a 4-bit row's bounds take log2(D / 16) exchanges within a warp.  In the
// half layout a thread takes the two 8-value chunks that hold both halves of 8
// pairs, else two neighbouring ones: every pair lies in one thread and the row is
// read and written in 16-byte pieces (a 4-bit row: a word of 8 codes per chunk).
// A CTA takes kTokens tokens and a slice of their heads, as in pa_rope.cu.
#include "pa_rope.cuh"

namespace pa {
namespace {

// kHalfAny: half layout whose rotary_dim / 2 is no multiple of 8: a pair's values
// lie in two threads and are exchanged through shared memory.
enum Layout { kInterleaved = 0, kHalf = 1, kHalfAny = 2 };

constexpr int kThreads = 128;
constexpr int kTokens = 2;
constexpr int kUnroll = 2;            // rows whose loads a thread has in flight
constexpr unsigned kFillCtas = 1024;  // CTAs below which a token's heads are spread over several

__device__ __forceinline__ float load_weight(const void* w, int dtype, int i) {
  return dtype == PA_F32 ? static_cast<const float*>(w)[i]
                         : (dtype == PA_BF16 ? load_scalar<bf16_t>(w, i) : load_scalar<f16_t>(w, i));
}

// One 4-bit row by `lanes` neighbouring threads (a power of two), 16 values each,
// chunks ca and cb: zero = the smallest value and scale = (largest - zero) / 15,
// both rounded to float16, code = the nearest of 0 .. 15 to (x - zero) / scale
// (a true quotient: between 16-bit values exact halves are common, and go to the
// even code).  Bounds are clipped to +-2^15, so that every stored value is a
// finite float16; NaN does not count for the bounds and takes code 0.
template <int LANES>
__device__ __forceinline__ void store_int4(uint8_t* codes, uint8_t* pair, int l, int ca, int cb, const float (&p)[8],
                                           const float (&q)[8], bool live) {
  float lo = fminf(p[0], q[0]), hi = fmaxf(p[0], q[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = fminf(lo, fminf(p[i], q[i]));
    hi = fmaxf(hi, fmaxf(p[i], q[i]));
  }
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  if (!live) return;
  lo = lo != lo ? 0.f : fminf(fmaxf(lo, -32768.f), 32768.f);  // (NaN: the row holds nothing else)
  hi = hi != hi ? 0.f : fminf(fmaxf(hi, -32768.f), 32768.f);
  const __half hz = __float2half_rn(lo);
  const float zero = __half2float(hz);
  const __half hs = __float2half_rn(fmaxf(__fdiv_rn(hi - zero, 15.f), 0.f));
  const float scale = __half2float(hs);
  const float step = scale > 0.f ? scale : INFINITY;  // a row of one value: code 0
  auto word = [&](const float (&x)[8]) {
    uint32_t w = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = fminf(fmaxf(rintf(__fdiv_rn(x[i] - zero, step)), 0.f), 15.f);
      w |= static_cast<uint32_t>(c) << (16 * (i & 1) + 4 * (i >> 1));
    }
    return w;
  };
  reinterpret_cast<uint32_t*>(codes)[ca] = word(p);
  reinterpret_cast<uint32_t*>(codes)[cb] = word(q);
  if (l == 0)
    *reinterpret_cast<uint32_t*>(pair) =
        static_cast<uint32_t>(__half_as_ushort(hs)) | (static_cast<uint32_t>(__half_as_ushort(hz)) << 16);
}

template <typename SRC, int MODE, int D, int LAYOUT>
__global__ void __launch_bounds__(kThreads) norm_rope_and_cache_kernel(const NormArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int L = D / 16;                  // threads of a row
  constexpr int PASS = kThreads / L;         // rows of a pass over the CTA
  __shared__ float2 cs[kTokens][D / 2];
  __shared__ __align__(16) float weights[2][D];
  __shared__ int64_t block_of[kTokens];
  __shared__ int row_of[kTokens];
  __shared__ float row_buf[LAYOUT == kHalfAny ? PASS : 1][LAYOUT == kHalfAny ? D + 1 : 1];
  const RopeArgs& r = a.r;
  const ReshapeArgs& w = r.w;
  const int half = r.rotary_dim >> 1;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kTokens;
  const int nt = static_cast<int>(min(static_cast<int64_t>(kTokens), w.num_tokens - n0));
  const int Hq = r.num_heads, Hk = w.num_kv_heads;
  const int rows = Hq + 2 * Hk, total = nt * rows;
  const int per = ((total + static_cast<int>(gridDim.y) - 1) / static_cast<int>(gridDim.y) + PASS - 1) / PASS * PASS;
  const int begin = static_cast<int>(blockIdx.y) * per, end = min(total, begin + per);
  constexpr int kvb = MODE == kCopy ? 2 : 1;
  const int l = static_cast<int>(threadIdx.x) % L, slot_row = static_cast<int>(threadIdx.x) / L;
  // the thread's two 8-value chunks
  const bool paired = LAYOUT == kHalf && l < (half >> 3);
  const int ca = paired ? l : 2 * l, cb = paired ? l + (half >> 3) : 2 * l + 1;

  bool ready = false;
  for (int x0 = begin; x0 < end || !ready; x0 += PASS * kUnroll) {
    uint4 lo[kUnroll], hi[kUnroll];
    int tok[kUnroll], which[kUnroll], head[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int x = x0 + k * PASS + slot_row;
      tok[k] = -1;
      which[k] = head[k] = 0;
      lo[k] = hi[k] = make_uint4(0u, 0u, 0u, 0u);
      if (x < end) {
        tok[k] = x >= rows ? 1 : 0;
        const int h = x - tok[k] * rows;
        which[k] = h < Hq ? 0 : (h < Hq + Hk ? 1 : 2);
        head[k] = h - (which[k] == 0 ? 0 : which[k] == 1 ? Hq : Hq + Hk);
        const void* base = which[k] == 0 ? r.q : which[k] == 1 ? w.k : w.v;
        const int64_t stride = which[k] == 0 ? r.q_stride : which[k] == 1 ? w.k_stride : w.v_stride;
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const uint8_t*>(base) + ((n0 + tok[k]) * stride + static_cast<int64_t>(head[k]) * D) * 2);
        lo[k] = src[ca];
        hi[k] = src[cb];
      }
    }
    if (!ready) {
      for (int x = threadIdx.x; x < nt * half; x += kThreads) {
        const int t = x >= half ? 1 : 0, i = x - t * half;
        cs[t][i] = rope_turn(__ldg(r.inv_freq + i), r.positions[n0 + t], r.rope_scale);
      }
      for (int x = threadIdx.x; x < 2 * D; x += kThreads) {
        const void* g = x < D ? a.q_weight : a.k_weight;
        if (g) weights[x / D][x % D] = load_weight(g, a.weight_dtype, x % D) + a.weight_offset;
      }
      if (threadIdx.x < nt) {
        const int64_t slot = w.slot_mapping[n0 + threadIdx.x];
        int64_t blk = -1;
        if (slot >= w.num_blocks * w.block_size) {
          if (blockIdx.y == 0) raise_error(w.err, PA_DEVERR_SLOT);
        } else if (slot >= 0) {
          blk = slot / w.block_size;
          row_of[threadIdx.x] = static_cast<int>(slot - blk * w.block_size);
        }
        block_of[threadIdx.x] = blk;
      }
      __syncthreads();
      ready = true;
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int wh = which[k];
      const int64_t blk = tok[k] >= 0 ? block_of[tok[k]] : -1;
      const bool live = blk >= 0;  // not: past the end, a padding token, or outside the pool
      float p[8], q[8];
      widen8<SRC>(lo[k], p);
      widen8<SRC>(hi[k], q);
      const void* const g = wh == 0 ? a.q_weight : (wh == 1 ? a.k_weight : nullptr);
      if (a.q_weight || a.k_weight) {  // (the same for all threads: the exchanges below)
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(p[i], p[i], fmaf(q[i], q[i], ss));
#pragma unroll
        for (int o = 1; o < L; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (g) {
          const float inv = rsqrtf(fmaf(ss, 1.f / D, a.eps));
          const float* const gw = weights[wh];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            p[i] *= inv * gw[8 * ca + i];
            q[i] *= inv * gw[8 * cb + i];
          }
        }
      }
      if (half > 0) {
        const float2* const c2 = cs[tok[k] > 0 ? 1 : 0];
        if constexpr (LAYOUT == kHalf) {
          if (paired && wh != 2) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 f = c2[8 * l + i];
              const float y = p[i], z = q[i];
              p[i] = y * f.x - z * f.y;
              q[i] = z * f.x + y * f.y;
            }
          }
        } else if constexpr (LAYOUT == kInterleaved) {
          if (wh != 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (8 * l + i < half) {
                const float2 f = c2[8 * l + i];
                const float y = p[2 * i], z = p[2 * i + 1];
                p[2 * i] = y * f.x - z * f.y;
                p[2 * i + 1] = z * f.x + y * f.y;
              }
              if (8 * l + 4 + i < half) {
                const float2 f = c2[8 * l + 4 + i];
                const float y = q[2 * i], z = q[2 * i + 1];
                q[2 * i] = y * f.x - z * f.y;
                q[2 * i + 1] = z * f.x + y * f.y;
              }
            }
          }
        } else {
          float* const buf = row_buf[slot_row];  // the row's threads are in one warp
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            buf[16 * l + i] = p[i];
            buf[16 * l + 8 + i] = q[i];
          }
          __syncwarp();
          if (wh != 2) {
            auto turn = [&](int c, float x) {
              if (c < half) return x * c2[c].x - buf[c + half] * c2[c].y;
              if (c < 2 * half) return x * c2[c - half].x + buf[c - half] * c2[c - half].y;
              return x;
            };
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              p[i] = turn(16 * l + i, p[i]);
              q[i] = turn(16 * l + 8 + i, q[i]);
            }
          }
        }
      }
      Dst d;
      d.cache = wh != 0;
      d.inv = 1.f;
      d.zp = 0;
      d.row = nullptr;
      [[maybe_unused]] uint8_t* pair = nullptr;  // 4-bit: where the row's scale and zero go
      if (live) {
        if (wh == 0) {
          d.row = static_cast<uint8_t*>(r.q_out) + ((n0 + tok[k]) * r.q_out_stride + static_cast<int64_t>(head[k]) * D) * 2;
        } else {
          uint8_t* const cache = static_cast<uint8_t*>(wh == 1 ? w.k_cache : w.v_cache);
          const int64_t tile = blk * Hk + head[k];
          const int row = row_of[tok[k]];
          if constexpr (MODE == kToInt4) {
            uint8_t* const at = cache + tile * (static_cast<int64_t>(w.block_size) * int4_row_bytes(D));
            d.row = at + row * (D / 2);
            pair = at + w.block_size * (D / 2) + 4 * row;
          } else {
            d.row = cache + (tile * w.block_size + row) * D * kvb;
            if constexpr (MODE != kCopy) d.inv = __ldg((wh == 1 ? w.k_inv_scale : w.v_inv_scale) + head[k]);
            if constexpr (MODE == kToInt8) d.zp = __ldg((wh == 1 ? w.k_zero_point : w.v_zero_point) + head[k]);
          }
        }
      }
      if constexpr (MODE == kToInt4) {
        store_int4<L>(d.row, pair, l, ca, cb, p, q, live && d.cache);  // (exchanges within the warp)
        if (live && !d.cache) {
          store8<SRC, kCopy>(d, 8 * ca, p);
          store8<SRC, kCopy>(d, 8 * cb, q);
        }
      } else if (live) {
        store8<SRC, MODE>(d, 8 * ca, p);
        store8<SRC, MODE>(d, 8 * cb, q);
      }
    }
  }
}

template <typename SRC, int MODE, int D>
cudaError_t launch_layout(const NormArgs& a, cudaStream_t stream) {
  const RopeArgs& r = a.r;
  // (no position: the half layout without pairs)
  const int layout = r.interleaved && r.rotary_dim > 0 ? kInterleaved : (r.rotary_dim % 16 == 0 ? kHalf : kHalfAny);
  void (*kern)(NormArgs) = layout == kInterleaved ? norm_rope_and_cache_kernel<SRC, MODE, D, kInterleaved>
                           : layout == kHalf      ? norm_rope_and_cache_kernel<SRC, MODE, D, kHalf>
                                                  : norm_rope_and_cache_kernel<SRC, MODE, D, kHalfAny>;
  constexpr int PASS = kThreads / (D / 16);
  const int rows = kTokens * (r.num_heads + 2 * r.w.num_kv_heads);
  const unsigned gx = static_cast<unsigned>((r.w.num_tokens + kTokens - 1) / kTokens);
  // slices of the heads: about kFillCtas CTAs, none with less than one pass
  unsigned gy = gx < kFillCtas ? kFillCtas / gx : 1;
  const unsigned most = static_cast<unsigned>((rows + PASS - 1) / PASS);
  gy = gy < most ? gy : most;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(gx, gy);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = r.w.pdl ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename SRC>
cudaError_t launch_src(const NormArgs& a, cudaStream_t stream) {
  const int kv = a.r.w.kv_dtype;
  if (kv == PA_INT4) return launch_layout<SRC, kToInt4, 128>(a, stream);
  if (a.r.w.head_dim == 128) {
    if (kv == PA_FP8_E4M3) return launch_layout<SRC, kToFp8, 128>(a, stream);
    if (kv == PA_INT8) return launch_layout<SRC, kToInt8, 128>(a, stream);
    return launch_layout<SRC, kCopy, 128>(a, stream);
  }
  if (kv == PA_FP8_E4M3) return launch_layout<SRC, kToFp8, 64>(a, stream);
  if (kv == PA_INT8) return launch_layout<SRC, kToInt8, 64>(a, stream);
  return launch_layout<SRC, kCopy, 64>(a, stream);
}

}  // namespace

cudaError_t launch_norm_rope_and_cache(const NormArgs& a, cudaStream_t stream) {
  (void)cudaGetLastError();
  return a.r.w.src_dtype == PA_F16 ? launch_src<f16_t>(a, stream) : launch_src<bf16_t>(a, stream);
}

}  // namespace pa
