// rope_axes.cu -- the paged KV write with rotary positions of several axes (time,
// height and width of image and video tokens).
//
// What it computes [tiny-vllm README, curriculum "RoPE" and "Paged KV cache"]: pair
// (x_i, x_{i+32}) of every q and K head of token t is turned by
// positions[axis(i)][t] * theta^(-2i/64); the K and V rows go to the token's slot.
//
// Bound: HBM bandwidth for a chunk (q both ways, K and V in and out: 256 (Hq + 2 Hkv)
// bytes a token), latency for a decode step.  A token has Hq + 2 Hkv rows of 128
// bytes; eight lanes hold a row, 16 bytes each, and a warp takes 16 rows of a token
// with all its loads in flight, so a token with 48 rows is spread over three warps.
// The angles cost each of them one sine and cosine a lane, shared by its rows.
//
// Measured: 16 x 700 tokens, 32/8 heads, 3 axes (137.8 MB) 23.9 us, 5.8 TB/s (8 rows a
// warp 25.4, 32 26.8; 8 warps a CTA 25.8; plain loads 26.9, streaming stores 26.3); a
// step of 64 tokens 4.1 us.
#include <cuda_bf16.h>

#include "device.cuh"
#include "kernels.h"
#include "rope.cuh"

namespace tvl {
namespace {

constexpr int kWarps = 4;              // per CTA
constexpr int kRowsPerWarp = 16;

struct AxesParams {
  __nv_bfloat16* q;
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  __nv_bfloat16* k_cache;
  __nv_bfloat16* v_cache;
  const int32_t* slots;
  const int32_t* positions;
  int num_tokens, hq, hkv, parts_q;
  long long num_slots;
  uint32_t* status;
};

// Block (x, y): 4 tokens, and of each the 16-row part y: parts_q of q rows, then
// K and V rows in one list.
__global__ void __launch_bounds__(kWarps * 32)
    rope_axes_write_kernel(const AxesParams p, const RopeTurns turns) {
  __shared__ float2 trig[kWarps][kD / 2];
  grid_dependency_wait();
  grid_dependents_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long t = static_cast<long long>(blockIdx.x) * kWarps + warp;
  if (t >= p.num_tokens) return;
  const int c = lane & 7;
  constexpr int kIt = kRowsPerWarp / 4;
  const bool is_q = static_cast<int>(blockIdx.y) < p.parts_q;
  const int first = (blockIdx.y - (is_q ? 0 : p.parts_q)) * kRowsPerWarp;
  const int row0 = first + (lane >> 3);
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
  long long slot = 0;
  if (!is_q) {
    slot = p.slots[t];
    if (slot < 0) return;                    // padding token: nothing to store
    if (slot >= p.num_slots) {
      if (lane == 0) report(p.status, TVL_DEV_BAD_SLOT);
      return;
    }
  }
  const int turned = is_q ? p.hq : p.hkv;    // rows that are rotated
  if (first < turned) {
    const Turn turn = token_turn(p.positions, p.num_tokens, t, turns, trig[warp]);
#pragma unroll
    for (int i = 0; i < kIt; ++i) {
      const uint4 y = rotate(w[i], turn);
      if (row0 + 4 * i < turned) w[i] = y;
    }
  }
#pragma unroll
  for (int i = 0; i < kIt; ++i) {
    const int r = row0 + 4 * i;
    if (r >= rows) break;
    __nv_bfloat16* dst = is_q        ? p.q + (t * p.hq + r) * kD
                         : r < p.hkv ? p.k_cache + (slot * p.hkv + r) * kD
                                     : p.v_cache + (slot * p.hkv + r - p.hkv) * kD;
    reinterpret_cast<uint4*>(dst)[c] = w[i];
  }
}

}  // namespace

cudaError_t launch_rope_axes_write(const RopeAxesWriteArgs& a, cudaStream_t stream) {
  if (a.num_tokens == 0) return cudaSuccess;
  AxesParams p;
  p.q = static_cast<__nv_bfloat16*>(a.q);
  p.k_new = static_cast<const __nv_bfloat16*>(a.k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(a.v_new);
  p.k_cache = static_cast<__nv_bfloat16*>(a.k_cache);
  p.v_cache = static_cast<__nv_bfloat16*>(a.v_cache);
  p.slots = a.slot_mapping;
  p.positions = a.positions;
  p.num_tokens = a.num_tokens;
  p.hq = a.q ? a.num_q_heads : 0;
  p.hkv = a.num_kv_heads;
  p.parts_q = (p.hq + kRowsPerWarp - 1) / kRowsPerWarp;
  const int parts_kv = (2 * p.hkv + kRowsPerWarp - 1) / kRowsPerWarp;
  p.num_slots = a.num_slots;
  p.status = a.status;
  return launch_pdl(rope_axes_write_kernel, dim3((a.num_tokens - 1) / kWarps + 1, p.parts_q + parts_kv),
                    dim3(kWarps * 32), 0, stream, p, rope_turns(a.rope_theta, a.axis_of));
}

}  // namespace tvl
