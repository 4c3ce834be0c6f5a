// pa_rope.cuh - device code shared by the kernels that write rotated keys and
// values into the cache: the angle of a position, and the stores of a row's
// elements in each cache type.
//
// Mathematics: pair i of a head at position p turns by the angle a = p *
// inv_freq[i].  In units of a full turn, t = inv_freq / 2 pi is held as a
// signed 64-bit fraction of a turn (its distance from the nearest whole turn
// times 2^64); p * t then wraps modulo one turn by itself in 64-bit integer
// arithmetic, so the reduction of a far position's angle loses nothing and needs
// no 64-bit floating point per token.  The top 32 bits of the product, rounded
// to a float32, go to sincospif: 2^-26 turns at most from p * t.  t itself is a
// product in 53 bits, off by at most 2^-54.6 turns for frequencies up to 1,
// which p multiplies: 2^-23.6 turns (5e-7 radians) at |p| = 2^31.
#pragma once

#include <type_traits>

#include "pa_common.cuh"
#include "pa_ops.h"

namespace pa {

enum Mode { kCopy = 0, kToFp8 = 1, kToInt8 = 2, kToInt4 = 3 };

// (cos, sin) * scale of the angle position * inv_freq
__device__ __forceinline__ float2 rope_turn(float inv_freq, int64_t position, float scale) {
  const double turns = static_cast<double>(inv_freq) * 0.15915494309189533577;  // 1 / 2 pi
  const double frac = turns - rint(turns);
  const unsigned long long step = static_cast<unsigned long long>(__double2ll_rn(frac * 18446744073709551616.0));
  const unsigned long long phase = step * static_cast<unsigned long long>(position);
  const float half_turns = static_cast<float>(static_cast<int>(phase >> 32)) * 4.656612873077393e-10f;  // 2^-31
  float sn, c;
  sincospif(half_turns, &sn, &c);
  return make_float2(c * scale, sn * scale);
}

struct Dst {  // where a head's row goes
  uint8_t* row;
  float inv;  // 8-bit caches
  int zp;     // INT8
  bool cache;
};

// 8 consecutive values from column c on
template <typename SRC, int MODE>
__device__ __forceinline__ void store8(const Dst& d, int c, const float (&x)[8]) {
  constexpr bool BF = std::is_same<SRC, bf16_t>::value;
  if (MODE == kCopy || !d.cache) {
    uint4 w;
    w.x = pack2<BF>(x[0], x[1]);
    w.y = pack2<BF>(x[2], x[3]);
    w.z = pack2<BF>(x[4], x[5]);
    w.w = pack2<BF>(x[6], x[7]);
    *reinterpret_cast<uint4*>(d.row + 2 * c) = w;
  } else {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(x[i], d.inv);
    uint32_t w[2];
    if constexpr (MODE == kToFp8) {
      w[0] = e4m3x2_code(y[0], y[1]) | (e4m3x2_code(y[2], y[3]) << 16);
      w[1] = e4m3x2_code(y[4], y[5]) | (e4m3x2_code(y[6], y[7]) << 16);
    } else {
      w[0] = w[1] = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i >> 2] |= (static_cast<uint32_t>(int8_code(y[i], d.zp)) & 0xffu) << (8 * (i & 3));
    }
    *reinterpret_cast<uint2*>(d.row + c) = make_uint2(w[0], w[1]);
  }
}

template <typename SRC, int MODE>
__device__ __forceinline__ void store1(const Dst& d, int c, float x) {
  if (MODE == kCopy || !d.cache) {
    reinterpret_cast<uint16_t*>(d.row)[c] =
        static_cast<uint16_t>(pack2<std::is_same<SRC, bf16_t>::value>(x, 0.f) & 0xffffu);
  } else if constexpr (MODE == kToFp8) {
    d.row[c] = static_cast<uint8_t>(e4m3x2_code(__fmul_rn(x, d.inv), 0.f) & 0xffu);
  } else {
    d.row[c] = static_cast<uint8_t>(int8_code(__fmul_rn(x, d.inv), d.zp));
  }
}

template <typename SRC>
__device__ __forceinline__ void widen8(const uint4& w, float (&x)[8]) {
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = widen2<SRC>(r[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

}  // namespace pa
