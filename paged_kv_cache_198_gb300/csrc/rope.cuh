// rope.cuh -- the rotary embedding of rows of 64 values, eight lanes a row.
#pragma once

#include <cmath>

#include <cuda_bf16.h>

#include "device.cuh"

namespace tvl {
namespace {

constexpr int kD = 64;
constexpr unsigned kFull = 0xffffffffu;

// theta^(-2i/D) / (2 pi) in units of 2^-64 turns, from a double: position times
// this, modulo 2^64, is the angle reduced without further error, so it is off by
// position * 2^-53 of a step, 2 10^-7 at most (position 2^31).
struct RopeTurns {
  unsigned long long f[kD / 2];
  unsigned long long axis;     // two bits a pair: the axis whose position turns it
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A row's eight values of this lane, as four pairs.
struct Eight {
  float2 v[4];
};
__device__ __forceinline__ Eight widen(uint4 w) {
  return {{bf16x2_to_float2(w.x), bf16x2_to_float2(w.y), bf16x2_to_float2(w.z),
           bf16x2_to_float2(w.w)}};
}
__device__ __forceinline__ uint4 narrow(const Eight& x) {
  return make_uint4(pack_bf16(x.v[0].x, x.v[0].y), pack_bf16(x.v[1].x, x.v[1].y),
                    pack_bf16(x.v[2].x, x.v[2].y), pack_bf16(x.v[3].x, x.v[3].y));
}

// This lane's share of the rotation: dimensions 8 c .. 8 c + 7 of a row, whose
// partners (d, d + 32) are lane c ^ 4's; sn carries the sign.
struct Turn {
  float2 cs[4], sn[4];
};
__device__ __forceinline__ uint4 rotate(uint4 w, const Turn& t) {
  uint4 o;
  o.x = __shfl_xor_sync(kFull, w.x, 4);
  o.y = __shfl_xor_sync(kFull, w.y, 4);
  o.z = __shfl_xor_sync(kFull, w.z, 4);
  o.w = __shfl_xor_sync(kFull, w.w, 4);
  Eight x = widen(w);
  const Eight y = widen(o);
#pragma unroll
  for (int j = 0; j < 4; ++j) x.v[j] = __ffma2_rn(x.v[j], t.cs[j], __fmul2_rn(y.v[j], t.sn[j]));
  return narrow(x);
}

// A token's angles: lane i takes pair i's in [-1/2, 1/2) turns at its axis' position
// (positions [A, num_tokens]) and leaves its cosine and sine in trig; lane c & 7 of a
// row then gathers those of its eight dimensions.
__device__ __forceinline__ Turn token_turn(const int32_t* positions, long long num_tokens, long long t,
                                           const RopeTurns& turns, float2 (&trig)[kD / 2]) {
  const int lane = threadIdx.x & 31, c = lane & 7;
  const long long pos = positions[static_cast<long long>(turns.axis >> (2 * lane) & 3) * num_tokens + t];
  const unsigned long long a = static_cast<unsigned long long>(pos) * turns.f[lane];
  float sn, cs;
  sincospif(__ll2float_rn(static_cast<long long>(a)) * 1.0842021724855044e-19f, &sn, &cs);  // 2^-63
  trig[lane] = make_float2(cs, sn);
  __syncwarp();
  const float4* tr = reinterpret_cast<const float4*>(&trig[8 * (c & 3)]);
  const float sign = c < 4 ? -1.f : 1.f;
  Turn turn;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 f = tr[j];
    turn.cs[j] = make_float2(f.x, f.z);
    turn.sn[j] = make_float2(f.y * sign, f.w * sign);
  }
  return turn;
}

// The turns of theta, with the pairs shared out among axes (`axis`, two bits a pair).
inline RopeTurns rope_turns(float theta, unsigned long long axis) {
  static thread_local float have = 0.f;
  static thread_local RopeTurns t = {};
  if (have != theta) {
    for (int i = 0; i < kD / 2; ++i)
      t.f[i] = static_cast<unsigned long long>(
          std::llrint(std::pow(static_cast<double>(theta), -2.0 * i / kD) / 6.283185307179586476925 *
                      4611686018427387904.0)) << 2;      // 2^62 steps a turn, then 2^64
    have = theta;
  }
  RopeTurns r = t;
  r.axis = axis;
  return r;
}

}  // namespace
}  // namespace tvl
