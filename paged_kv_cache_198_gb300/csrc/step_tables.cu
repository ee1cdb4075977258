// step_tables.cu -- an engine step's bookkeeping on the GPU: block tables, query
// starts, cache slots and positions from request lengths, over a stack of free
// blocks.
//
// [nano-vLLM guide ch. 4 "PagedAttention" (the block allocator), ch. 5 "The
// Scheduler" (sequences join and leave the batch every step)]
//
// What it computes, for rows s with cached_lens c_s and new_lens n_s:
//   had_s = ceil(c_s / bs); n_s < 0: the row is done, give_s = had_s, length 0;
//   else need_s = ceil((c_s + n_s) / bs) - had_s and length c_s + n_s.
// The blocks given back go onto the stack in row order, then the k-th new block
// (rows in order, positions in order) is free[count + sum give - 1 - k]; the
// tokens are packed in row order, and token i of row s at position p has slot
// table[s][p / bs] * bs + p % bs.
//
// Split.  Everything that depends on all rows (three sums and their scans) and
// everything that is updated (stack, tables, lengths) is done by one CTA: it reads
// all it needs before it writes, so lengths and count may be updated in place,
// and nothing has to be handed between CTAs.
#include "device.cuh"
#include "kernels.h"

namespace tvl {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kFillPerThread = 4;
constexpr int kFillRows = 4096;          // rows whose starts a fill CTA keeps in shared memory
constexpr unsigned kFull = 0xffffffffu;

struct Row {
  int cached, had, give, need, add, len;
  bool bad;
};

__device__ __forceinline__ int blocks_of(int tokens, int bs) { return tokens / bs + (tokens % bs != 0 ? 1 : 0); }

__device__ __forceinline__ Row load_row(const StepTablesArgs& p, int s) {
  Row r = {0, 0, 0, 0, 0, 0, false};
  if (s >= p.num_seqs) return r;
  const int c = p.cached_lens[s], n = p.new_lens[s];
  const long long cap = static_cast<long long>(p.max_blocks) * p.block_size;
  r.cached = c;
  r.bad = c < 0 || c > cap || (n > 0 && static_cast<long long>(c) + n > cap);
  if (r.bad) return r;
  r.had = blocks_of(c, p.block_size);
  if (n < 0) {
    r.give = r.had;
  } else {
    r.add = n;
    r.len = c + n;                       // <= cap < 2^31
    r.need = blocks_of(r.len, p.block_size) - r.had;
  }
  return r;
}

// Sum of v over the block, in every thread.  tmp: 32 values; ends with a barrier.
__device__ __forceinline__ long long block_sum(long long v, long long* tmp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
  __syncthreads();
  v = tmp[threadIdx.x & 31];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  __syncthreads();
  return v;
}

// Sum of v over the threads before this one; the block's sum goes to total.
__device__ __forceinline__ int block_scan(int v, int& total, int* tmp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) tmp[warp] = x;
  __syncthreads();
  const int part = tmp[lane];
  total = __reduce_add_sync(kFull, part);
  const int before = __reduce_add_sync(kFull, lane < warp ? part : 0);
  __syncthreads();
  return before + x - v;
}

// The last i in [0, n) with start[i] <= x; start[0] <= x, non-decreasing.
__device__ __forceinline__ int last_at_most(const int* start, int n, int x) {
  int lo = 0, hi = n;                    // start[lo] <= x; hi == n or start[hi] > x
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// Slot and position of packed token i of row s, whose tokens end before `end`.
__device__ __forceinline__ void fill_token(const StepTablesArgs& p, int i, int s, int end, int len) {
  const int pos = len - (end - i);
  const int b = pos / p.block_size;
  const int id = p.block_tables[static_cast<long long>(s) * p.max_blocks + b];
  int slot = -1;
  if (id >= 0 && id < p.num_blocks)
    slot = id * p.block_size + (pos - b * p.block_size);   // NB * bs < 2^31
  else
    report(p.status, TVL_DEV_BAD_BLOCK_ID);
  p.slot_mapping[i] = slot;
  if (p.positions != nullptr) p.positions[i] = pos;
}
__device__ __forceinline__ void fill_padding(const StepTablesArgs& p, int i) {
  p.slot_mapping[i] = -1;
  if (p.positions != nullptr) p.positions[i] = 0;
}

template <bool kFill>
__global__ void __launch_bounds__(kPlanThreads) step_plan_kernel(const StepTablesArgs p) {
  __shared__ long long sums[32];
  __shared__ int scan[32];
  __shared__ int off[kPlanThreads], had[kPlanThreads], starts[kPlanThreads], lens[kPlanThreads];
  const int tid = threadIdx.x, S = p.num_seqs;
  grid_dependency_wait();
  grid_dependents_launch();

  long long give = 0, need = 0, add = 0;
  bool bad = false;
  for (int s = tid; s < S; s += kPlanThreads) {
    const Row r = load_row(p, s);
    give += r.give;
    need += r.need;
    add += r.add;
    bad |= r.bad;
  }
  const long long count = *p.free_count;
  give = block_sum(give, sums);
  need = block_sum(need, sums);
  add = block_sum(add, sums);
  uint32_t why = __syncthreads_or(bad) ? TVL_DEV_BAD_CONTEXT_LEN : 0u;
  if (add > p.max_tokens) why |= TVL_DEV_BAD_QUERY_LEN;
  if (count < 0 || count + give > p.num_blocks)
    why |= TVL_DEV_BAD_BLOCK_ID;
  else if (need > count + give)
    why |= TVL_DEV_OUT_OF_BLOCKS;
  if (why != 0) {                        // the whole step is refused
    if (tid == 0) {
      report(p.status, why);
      p.query_start_loc[S] = 0;
      *p.free_count_out = static_cast<int>(count);
    }
    for (int s = tid; s < S; s += kPlanThreads) {
      p.context_lens[s] = p.cached_lens[s];
      p.query_start_loc[s] = 0;
    }
    if (kFill)
      for (int i = tid; i < p.max_tokens; i += kPlanThreads) fill_padding(p, i);
    return;
  }

  // from here every sum is at most max(NB, max_tokens) < 2^31
  const int have = static_cast<int>(count), top = have + static_cast<int>(give);
  if (give > 0) {
    int done = 0;
    for (int s0 = 0; s0 < S; s0 += kPlanThreads) {
      const Row r = load_row(p, s0 + tid);
      int n;
      off[tid] = block_scan(r.give, n, scan);
      __syncthreads();
      for (int i = tid; i < n; i += kPlanThreads) {
        const int k = last_at_most(off, kPlanThreads, i);
        p.free_blocks[have + done + i] =
            p.block_tables[static_cast<long long>(s0 + k) * p.max_blocks + i - off[k]];
      }
      done += n;
      __syncthreads();
    }
  }
  int taken = 0, tokens = 0;
  for (int s0 = 0; s0 < S; s0 += kPlanThreads) {
    const Row r = load_row(p, s0 + tid);
    int n, t;
    off[tid] = block_scan(r.need, n, scan);
    had[tid] = r.had;
    const int start = tokens + block_scan(r.add, t, scan);
    if (kFill) {
      starts[tid] = start;
      lens[tid] = r.len;
    }
    if (s0 + tid < S) {
      p.context_lens[s0 + tid] = r.len;
      p.query_start_loc[s0 + tid] = start;
    }
    __syncthreads();
    for (int i = tid; i < n; i += kPlanThreads) {
      const int k = last_at_most(off, kPlanThreads, i);
      const int id = p.free_blocks[top - 1 - taken - i];
      if (id < 0 || id >= p.num_blocks) report(p.status, TVL_DEV_BAD_BLOCK_ID);
      p.block_tables[static_cast<long long>(s0 + k) * p.max_blocks + had[k] + i - off[k]] = id;
    }
    taken += n;
    tokens += t;
    __syncthreads();
  }
  if (tid == 0) {
    p.query_start_loc[S] = tokens;
    *p.free_count_out = top - taken;
  }
  if (kFill) {                           // S <= kPlanThreads: starts and lens are complete
    for (int i = tid; i < p.max_tokens; i += kPlanThreads) {
      if (i >= tokens) {
        fill_padding(p, i);
        continue;
      }
      const int s = last_at_most(starts, S, i);
      fill_token(p, i, s, s + 1 < S ? starts[s + 1] : tokens, lens[s]);
    }
  }
}

// Slots and positions of many tokens, from the plan's starts, lengths and tables.
__global__ void __launch_bounds__(kFillThreads) step_fill_kernel(const StepTablesArgs p) {
  __shared__ int kept[kFillRows];
  const int S = p.num_seqs;
  grid_dependency_wait();
  grid_dependents_launch();
  const int tokens = p.query_start_loc[S];
  const long long i0 = static_cast<long long>(blockIdx.x) * kFillThreads * kFillPerThread;
  const int* starts = p.query_start_loc;
  if (S <= kFillRows && i0 < tokens) {
    for (int s = threadIdx.x; s < S; s += kFillThreads) kept[s] = p.query_start_loc[s];
    starts = kept;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kFillPerThread; ++j) {
    const long long i = i0 + j * kFillThreads + threadIdx.x;
    if (i >= p.max_tokens) return;
    if (i >= tokens) {
      fill_padding(p, static_cast<int>(i));
      continue;
    }
    const int s = last_at_most(starts, S, static_cast<int>(i));
    fill_token(p, static_cast<int>(i), s, s + 1 < S ? starts[s + 1] : tokens, p.context_lens[s]);
  }
}

// Up to this many (padded) tokens the plan's CTA fills them in itself.
constexpr int kPlanFills = 4096;

}  // namespace

cudaError_t launch_step_tables(const StepTablesArgs& a, cudaStream_t stream) {
  if (a.max_tokens <= kPlanFills && a.num_seqs <= kPlanThreads)
    return launch_pdl(step_plan_kernel<true>, dim3(1), dim3(kPlanThreads), 0, stream, a);
  cudaError_t e = launch_pdl(step_plan_kernel<false>, dim3(1), dim3(kPlanThreads), 0, stream, a);
  if (e != cudaSuccess || a.max_tokens == 0) return e;
  constexpr int per = kFillThreads * kFillPerThread;
  return launch_pdl(step_fill_kernel, dim3((a.max_tokens - 1) / per + 1), dim3(kFillThreads), 0, stream, a);
}

}  // namespace tvl
