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
// heads: 30 us, of which the 121 MB are 18, and 8 for expanding their blocks; at 68
// registers 37% of the warps' places are used, too few to keep loads and the
// codes' arithmetic (62% of issue slots) both going.  At 64 registers (8 bytes
// spilled) 34.6 us for both, against 35.1.  Eight lanes hold a row, 16
// bytes each; a warp takes 16 rows of a token (q, K and V rows in one list)
// with all loads in flight, so a token with 48 rows is spread over three warps
// and a decode step of 64 tokens over 192.
#include <cuda_bf16.h>

#include "device.cuh"
#include "kernels.h"
#include "kv4.cuh"
#include "rope.cuh"

namespace tvl {
namespace {

constexpr int kWarps = 4;              // per CTA
constexpr int kRowsPerWarp = 16;

struct WriteParams {
  __nv_bfloat16* q;
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  uint8_t* cache;
  const int32_t* slots;
  const int32_t* positions;     // [axes, T]; null: no rotation
  int num_tokens, hq, hkv, parts_q;
  long long num_slots;
  uint32_t* status;
};

// A row's (s, z) from its extremes, and the codes of this lane's eight values.
//
// c = rint(d / s), d = x - z in fp32, ties to even, without a division a value: t = d * inv
// rounded to an integer is off by at most one, and only next to a tie (inv is
// within 2^-24 of 1 / s and d / s <= 15).  The residual e = d - t s is exact, so
// |e| > s / 2, or = with t odd, says that the other neighbour is the nearer or
// the even one.  Rows whose scale is too small for 1 / s take the division.
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
  const float inv = __fdiv_rn(1.0f, s), half = 0.5f * s;
  float c[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 d = __fadd2_rn(x.v[j], make_float2(-mn, -mn));
    const float2 t = __ffma2_rn(d, make_float2(inv, inv), make_float2(kMagic, kMagic));
    const float2 r = __fadd2_rn(t, make_float2(-kMagic, -kMagic));
    const float2 e = __ffma2_rn(r, make_float2(-s, -s), d);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float ev = k ? e.y : e.x;
      const int odd = __float_as_int(k ? t.y : t.x) & 1;
      // over > 0, or = +0 with an odd code
      const float over = fabsf(ev) - half;
      const bool fix = __float_as_int(over) + odd > 0;
      c[2 * j + k] = (k ? r.y : r.x) + (fix ? copysignf(1.0f, ev) : 0.0f);
    }
  }
  // four codes are exact in one float: c0 + 16 c1 + 256 c2 + 4096 c3
  const float lo = fmaf(4096.f, c[3], fmaf(256.f, c[2], fmaf(16.f, c[1], c[0]))) + kMagic;
  const float hi = fmaf(4096.f, c[7], fmaf(256.f, c[6], fmaf(16.f, c[5], c[4]))) + kMagic;
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x5410);
}

// Block (x, y): 4 tokens, and of each the 16-row part y: parts_q of q rows, then
// K and V rows.
__global__ void __launch_bounds__(kWarps * 32)
    kv4_write_kernel(const WriteParams p, const RopeTurns turns) {
  __shared__ float2 trig[kWarps][kD / 2];
  grid_dependency_wait();
  grid_dependents_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long t = static_cast<long long>(blockIdx.x) * kWarps + warp;
  if (t >= p.num_tokens) return;
  const int c = lane & 7;
  constexpr int kIt = kRowsPerWarp / 4;
  const bool is_q = static_cast<int>(blockIdx.y) < p.parts_q;
  const int row0 = (blockIdx.y - (is_q ? 0 : p.parts_q)) * kRowsPerWarp + (lane >> 3);
  const int rows = is_q ? p.hq : 2 * p.hkv;

  uint4 w[kIt];
#pragma unroll
  for (int i = 0; i < kIt; ++i) {
    const int r = row0 + 4 * i;
    w[i] = make_uint4(0, 0, 0, 0);
    if (r < rows) {
      const __nv_bfloat16* src = is_q        ? p.q + (t * p.hq + r) * kD
                                 : r < p.hkv ? p.k_new + (t * p.hkv + r) * kD
                                             : p.v_new + (t * p.hkv + r - p.hkv) * kD;
      w[i] = __ldcs(reinterpret_cast<const uint4*>(src) + c);
    }
  }
  Turn turn;
  const bool rope = p.positions != nullptr && row0 - (lane >> 3) < (is_q ? p.hq : p.hkv);
  if (rope) {
    turn = token_turn(p.positions, p.num_tokens, t, turns, trig[warp]);
  }
  if (is_q) {
#pragma unroll
    for (int i = 0; i < kIt; ++i) {
      const int r = row0 + 4 * i;
      const uint4 y = rotate(w[i], turn);
      if (r < rows) reinterpret_cast<uint4*>(p.q + (t * p.hq + r) * kD)[c] = y;
    }
    return;
  }
  const long long slot = p.slots[t];
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
    if (rope && r - (lane >> 3) < p.hkv) {       // the step holds a K row
      // the K that is quantised is the bf16 row the bf16 cache would hold
      const uint4 y = rotate(w[i], turn);
      if (!is_v) w[i] = y;
    }
    const Eight x = widen(w[i]);
    float mn = x.v[0].x, mx = mn;
    float2 fin = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      mn = fminf(mn, fminf(x.v[j].x, x.v[j].y));
      mx = fmaxf(mx, fmaxf(x.v[j].x, x.v[j].y));
      fin = __ffma2_rn(x.v[j], make_float2(0.f, 0.f), fin);    // 0 unless something is not finite
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      mn = fminf(mn, __shfl_xor_sync(kFull, mn, o));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
    }
    const float range = mx - mn;
    const bool bad = !(range < INFINITY) || fin.x + fin.y != 0.f;   // NaN != 0
    const bool row_bad = ((__ballot_sync(kFull, bad) >> (lane & 24)) & 0xffu) != 0;
    if (r >= rows) continue;
    uint32_t code = 0;
    uint32_t sz = 0x7fc07fc0u;          // a row that is not finite stands for NaN
    if (!row_bad) {
      const uint32_t sb = (__float_as_uint(__fdiv_rn(range, 15.0f)) + 0xffffu) & 0xffff0000u;
      sz = (sb >> 16) | (__float_as_uint(mn) & 0xffff0000u);
      code = row_codes(x, mn, __uint_as_float(sb));
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
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      y[j] = fmaf(m.x, static_cast<float>((code[k] >> (4 * j)) & 15u), m.y);
    __nv_bfloat16* out = (k < 4 ? k_cache : v_cache) +
                         ((static_cast<long long>(to) * cpb + sub) * kRecTokens + tok) * hkv * kD + h * kD;
    reinterpret_cast<uint4*>(out)[c] = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]),
                                                  pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
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
  p.parts_q = (p.hq + kRowsPerWarp - 1) / kRowsPerWarp;
  const int parts_kv = (2 * p.hkv + kRowsPerWarp - 1) / kRowsPerWarp;
  p.num_slots = a.num_slots;
  p.status = a.status;
  static const RopeTurns none = {};
  return launch_pdl(kv4_write_kernel, dim3((a.num_tokens - 1) / kWarps + 1, p.parts_q + parts_kv),
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
