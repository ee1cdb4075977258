// kv4.cu -- writing rows into the 4-bit paged cache and expanding its blocks
// back to bf16 (the layout is kv4.cuh's).
//
// Write: for each token, optionally the rotary embedding of its q heads (in
// place) and of its new K heads, then each K and V row x (64 values) becomes
//   z = min x,  s = bf16 rounded up of (max x - z) / 15,
//   c_d = min(15, rint((x_d - z) / s))   (ties to even; s = 0: all 0),
// with max x - z and x_d - z in fp32 (exact unless the magnitudes are some 2^16
// apart), so |s c_d + z - x_d| <= s / 2 + 2^-19 s.  s is rounded up, so the largest
// value needs no code above 15.  bf16 inputs make exact ties common, so the
// quotients' roundings are the exact ones (row_codes).
//
// Bound: HBM bandwidth for a prefill chunk (per token 256 Hkv bytes in, 72 Hkv
// out, and q both ways), latency for a decode step.  16 chunks of 700 tokens, 32/8
// heads: 23-24 us, of which the 121 MB are 18, and 6-8 for expanding their blocks; issue slots
// (72-74% full) hold it back.  Eight lanes hold a row, 16 bytes each; a warp takes 16 q rows
// or 8 K and V rows of a token (in one list) with all loads in flight, the parts of a
// token next to each other in the grid, so that q's traffic goes on beside the codes'
// arithmetic, and a decode step of 64 tokens is spread over 256 warps.  What brought it
// there, us for write and expansion: packed minima and maxima, codes from one side of the
// residual, a reciprocal within an ulp and 16 K and V rows in two warps 35.5 -> 31.2; two
// batches of q rows a warp 29.2; 48 registers (10 CTAs an SM) 28.9.
#include <cuda_bf16.h>

#include "device.cuh"
#include "kernels.h"
#include "kv4.cuh"
#include "rope.cuh"

namespace tvl {
namespace {

constexpr int kWarps = 4;              // per CTA
constexpr int kRowsQ = 16, kRowsKv = 8;   // rows a warp has in flight
// Beyond this many q rows a warp takes two batches of them with one set of angles: 8192
// tokens of 32 heads 17.6 us, 18.5 with a batch a warp; 1536 (49152 rows) 6.1 and 5.7,
// 1024 of 64 (65536) 6.3 and 5.7, 2048 of 32 (65536) 6.6 and 6.9, 1536 of 64 7.1 and 7.4.
constexpr int kManyRows = 80000;

struct WriteParams {
  __nv_bfloat16* q;
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  uint8_t* cache;
  const int32_t* slots;
  const int32_t* positions;     // [axes, T]; null: no rotation
  int num_tokens, hq, hkv, parts_q, parts, batches;
  long long num_slots;
  uint32_t* status;
};

// A row's minimum and its range, in all eight lanes that hold it; a NaN in the row makes
// both NaN, an infinity the range infinite or NaN.  The values are bf16, so packed minima
// are exact; a word holds (min, -max) and one reduction finds both.
struct RowRange {
  float mn, range;
};
__device__ __forceinline__ RowRange row_range(uint4 w) {
  auto as = [](uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); };
  auto bits = [](__nv_bfloat162 x) { return *reinterpret_cast<const uint32_t*>(&x); };
  const uint32_t lo = bits(__hmin2_nan(__hmin2_nan(as(w.x), as(w.y)), __hmin2_nan(as(w.z), as(w.w))));
  const uint32_t hi = bits(__hmax2_nan(__hmax2_nan(as(w.x), as(w.y)), __hmax2_nan(as(w.z), as(w.w))));
  const uint32_t nh = hi ^ 0x80008000u;
  uint32_t x = bits(__hmin2_nan(as(__byte_perm(lo, nh, 0x5410)), as(__byte_perm(lo, nh, 0x7632))));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) x = bits(__hmin2_nan(as(x), as(__shfl_xor_sync(kFull, x, o))));
  const float2 e = bf16x2_to_float2(x);
  return {e.x, -e.y - e.x};
}

// A row's (s, z) from its extremes, and the codes of this lane's eight values.
//
// c = rint(d / s), d = x - z in fp32, ties to even, without a division a value: r =
// rint((x - (z + s / 2)) / s) is c or c - 1, as what it rounds is off by 2^-10 at most (a
// row's s is at least 2^-12 of |z|, but for rows of one value).  The residual e = d - r s
// is exact and in about [0, s] (r = -1: d is about 0 and e about s), and c = r + 1 where
// e > s / 2, or e = s / 2 and r is odd: positive floats compare as integers, a negative
// one is a negative integer.  Rows whose scale is too small for 1 / s take the division.
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));    // within one ulp
  return y;
}
__device__ __forceinline__ uint32_t row_codes(const Eight& x, float mn, float s) {
  constexpr float kMagic = 12582912.f;             // 1.5 * 2^23: adding it rounds to an integer
  if (s < 1e-36f) {
    uint32_t code = 0;
    if (s > 0.f) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = (j & 1) ? x.v[j >> 1].y : x.v[j >> 1].x;
        code |= static_cast<uint32_t>(min(__float2int_rn(__fdiv_rn(v - mn, s)), 15)) << (4 * j);
      }
    }
    return code;
  }
  const float inv = rcp(s), half = 0.5f * s, low = -(mn + half);
  const int half_bits = __float_as_int(half);
  float c[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 d = __fadd2_rn(x.v[j], make_float2(-mn, -mn));
    const float2 t = __ffma2_rn(__fadd2_rn(x.v[j], make_float2(low, low)), make_float2(inv, inv),
                                make_float2(kMagic, kMagic));
    const float2 r = __fadd2_rn(t, make_float2(-kMagic, -kMagic));
    const float2 e = __ffma2_rn(r, make_float2(-s, -s), d);
    c[2 * j] = r.x + (__float_as_int(e.x) + (__float_as_int(t.x) & 1) > half_bits ? 1.0f : 0.0f);
    c[2 * j + 1] = r.y + (__float_as_int(e.y) + (__float_as_int(t.y) & 1) > half_bits ? 1.0f : 0.0f);
  }
  // four codes are exact in one float: c0 + 16 c1 + 256 c2 + 4096 c3
  const float lo = fmaf(4096.f, c[3], fmaf(256.f, c[2], fmaf(16.f, c[1], c[0]))) + kMagic;
  const float hi = fmaf(4096.f, c[7], fmaf(256.f, c[6], fmaf(16.f, c[5], c[4]))) + kMagic;
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x5410);
}

// Block x: kWarps tokens, and of each part x % parts: parts_q of `batches` times kRowsQ q
// rows, then parts of kRowsKv K and V rows, in one list.
__global__ void __launch_bounds__(kWarps * 32, 10)
    kv4_write_kernel(const WriteParams p, const RopeTurns turns) {
  __shared__ float2 trig[kWarps][kD / 2];
  grid_dependency_wait();
  grid_dependents_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int step = blockIdx.x / p.parts, part = blockIdx.x - step * p.parts;
  const long long t = static_cast<long long>(step) * kWarps + warp;
  if (t >= p.num_tokens) return;
  const int c = lane & 7;
  if (part < p.parts_q) {
    constexpr int kIt = kRowsQ / 4;
    uint4* q = reinterpret_cast<uint4*>(p.q + t * p.hq * kD) + c;
    int row0 = part * p.batches * kRowsQ + (lane >> 3);
    uint4 w[kIt];
    auto load = [&]() {
#pragma unroll
      for (int i = 0; i < kIt; ++i) {
        const int r = row0 + 4 * i;
        w[i] = r < p.hq ? __ldcs(q + r * (kD / 8)) : make_uint4(0, 0, 0, 0);
      }
    };
    load();
    const Turn turn = token_turn(p.positions, p.num_tokens, t, turns, trig[warp]);
#pragma unroll 1
    for (int k = 0;;) {
#pragma unroll
      for (int i = 0; i < kIt; ++i) {
        const int r = row0 + 4 * i;
        const uint4 y = rotate(w[i], turn);
        if (r < p.hq) q[r * (kD / 8)] = y;
      }
      if (++k == p.batches) break;
      row0 += kRowsQ;
      load();
    }
    return;
  }
  constexpr int kIt = kRowsKv / 4;
  const int first = (part - p.parts_q) * kRowsKv;
  const int row0 = first + (lane >> 3);
  uint4 w[kIt];
#pragma unroll
  for (int i = 0; i < kIt; ++i) {
    const int r = row0 + 4 * i;
    const __nv_bfloat16* src = r < p.hkv ? p.k_new + (t * p.hkv + r) * kD
                                         : p.v_new + (t * p.hkv + r - p.hkv) * kD;
    w[i] = r < 2 * p.hkv ? __ldcs(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0, 0, 0, 0);
  }
  const long long slot = p.slots[t];
  const bool rope = p.positions != nullptr && first < p.hkv;
  if (rope) {
    // the K that is quantised is the bf16 row the bf16 cache would hold
    const Turn turn = token_turn(p.positions, p.num_tokens, t, turns, trig[warp]);
#pragma unroll
    for (int i = 0; i < kIt; ++i) {
      const uint4 y = rotate(w[i], turn);
      if (row0 + 4 * i < p.hkv) w[i] = y;
    }
  }
  if (slot < 0) return;
  if (slot >= p.num_slots) {
    if (lane == 0) report(p.status, TVL_DEV_BAD_SLOT);
    return;
  }
  // records of the token's 16-token group, one a head; its place in them
  const int tok = static_cast<int>(slot & (kRecTokens - 1));
  uint8_t* group = p.cache + slot / kRecTokens * p.hkv * kRecBytes;
#pragma unroll
  for (int i = 0; i < kIt; ++i) {
    const int r = row0 + 4 * i;
    const bool is_v = r >= p.hkv;
    const RowRange e = row_range(w[i]);
    if (r >= 2 * p.hkv) continue;
    uint32_t code = 0;
    uint32_t sz = 0x7fc07fc0u;          // a row that is not finite stands for NaN
    if (e.range < INFINITY) {
      const uint32_t sb = (__float_as_uint(__fdiv_rn(e.range, 15.0f)) + 0xffffu) & 0xffff0000u;
      sz = (sb >> 16) | (__float_as_uint(e.mn) & 0xffff0000u);
      code = row_codes(widen(w[i]), e.mn, __uint_as_float(sb));
    } else if (c == 0) {
      report(p.status, TVL_DEV_NONFINITE);
    }
    uint8_t* rec = group + (r - (is_v ? p.hkv : 0)) * kRecBytes;
    reinterpret_cast<uint32_t*>(rec + (is_v ? kRecV : 0) + tok * kRowCodes)[c] = code;
    if (c == 0) reinterpret_cast<uint32_t*>(rec + (is_v ? kRecVMeta : kRecKMeta))[tok] = sz;
  }
}

// One warp per record: its 16 K rows and 16 V rows, four at a time (eight
// lanes a row, 4 bytes of codes in, 16 bytes of bf16 out), the codes of all
// eight steps in flight.
__global__ void __launch_bounds__(kWarps * 32)
    kv4_expand_kernel(__nv_bfloat16* k_cache, __nv_bfloat16* v_cache, const uint8_t* cache,
                      const int32_t* src, const int32_t* dst, long long records, int hkv, int cpb,
                      int src_blocks, int dst_blocks, uint32_t* status) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long id = static_cast<long long>(blockIdx.x) * kWarps + warp;
  if (id >= records) return;
  const int h = static_cast<int>(id % hkv);
  const long long rest = id / hkv;
  const int sub = static_cast<int>(rest % cpb);
  const long long i = rest / cpb;
  const int from = src[i], to = dst[i];
  if (from < 0 || from >= src_blocks || to < 0 || to >= dst_blocks) {
    if (lane == 0) report(status, TVL_DEV_BAD_BLOCK_ID);
    return;
  }
  const uint8_t* rec = cache + ((static_cast<long long>(from) * cpb + sub) * hkv + h) * kRecBytes;
  const int c = lane & 7, g = lane >> 3;
  uint32_t code[8], sz[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {          // k < 4: K rows, else V rows
    const int tok = (k & 3) * 4 + g;
    code[k] = __ldcs(reinterpret_cast<const uint32_t*>(rec + (k < 4 ? 0 : kRecV) + tok * kRowCodes) + c);
    sz[k] = __ldcs(reinterpret_cast<const uint32_t*>(rec + (k < 4 ? kRecKMeta : kRecVMeta)) + tok);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int tok = (k & 3) * 4 + g;
    const float2 m = bf16x2_to_float2(sz[k]);
    const uint32_t even = code[k] & 0x0f0f0f0fu, odd = (code[k] >> 4) & 0x0f0f0f0fu;
    uint32_t y[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {        // a code under 2^23's exponent is 2^23 + code
      const float2 v = __fadd2_rn(make_float2(__uint_as_float(__byte_perm(even, 0x4b000000u, 0x7440 | b)),
                                              __uint_as_float(__byte_perm(odd, 0x4b000000u, 0x7440 | b))),
                                  make_float2(-8388608.f, -8388608.f));
      const float2 u = __ffma2_rn(v, make_float2(m.x, m.x), make_float2(m.y, m.y));
      y[b] = pack_bf16(u.x, u.y);
    }
    __nv_bfloat16* out = (k < 4 ? k_cache : v_cache) +
                         ((static_cast<long long>(to) * cpb + sub) * kRecTokens + tok) * hkv * kD + h * kD;
    reinterpret_cast<uint4*>(out)[c] = make_uint4(y[0], y[1], y[2], y[3]);
  }
}

}  // namespace

cudaError_t launch_kv4_write(const Kv4WriteArgs& a, cudaStream_t stream) {
  if (a.num_tokens == 0) return cudaSuccess;
  WriteParams p;
  p.q = static_cast<__nv_bfloat16*>(a.q);
  p.k_new = static_cast<const __nv_bfloat16*>(a.k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(a.v_new);
  p.cache = static_cast<uint8_t*>(a.cache);
  p.slots = a.slot_mapping;
  p.positions = a.positions;
  p.num_tokens = a.num_tokens;
  p.hq = a.q && a.positions ? a.num_q_heads : 0;
  p.hkv = a.num_kv_heads;
  p.batches = p.hq > kRowsQ && static_cast<long long>(a.num_tokens) * p.hq > kManyRows ? 2 : 1;
  p.parts_q = (p.hq + kRowsQ * p.batches - 1) / (kRowsQ * p.batches);
  p.parts = p.parts_q + (2 * p.hkv + kRowsKv - 1) / kRowsKv;
  const long long ctas = static_cast<long long>((a.num_tokens - 1) / kWarps + 1) * p.parts;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  p.num_slots = a.num_slots;
  p.status = a.status;
  static const RopeTurns none = {};
  return launch_pdl(kv4_write_kernel, dim3(static_cast<unsigned>(ctas)),
                    dim3(kWarps * 32), 0, stream, p,
                    a.positions ? rope_turns(a.rope_theta, a.axis_of) : none);
}

cudaError_t launch_kv4_expand(const Kv4ExpandArgs& a, cudaStream_t stream) {
  if (a.n == 0) return cudaSuccess;
  const int cpb = a.block_size / kRecTokens;
  const long long records = static_cast<long long>(a.n) * cpb * a.num_kv_heads;
  return launch_pdl(kv4_expand_kernel, dim3(static_cast<unsigned>((records + kWarps - 1) / kWarps)),
                    dim3(kWarps * 32), 0, stream, static_cast<__nv_bfloat16*>(a.k_cache),
                    static_cast<__nv_bfloat16*>(a.v_cache), static_cast<const uint8_t*>(a.cache),
                    a.src, a.dst, records, a.num_kv_heads, cpb, a.num_blocks, a.out_blocks,
                    a.status);
}

}  // namespace tvl
