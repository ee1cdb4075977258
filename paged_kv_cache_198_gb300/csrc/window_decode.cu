// window_decode.cu -- decode attention on the tensor cores, over a bf16 or a
// 4-bit paged cache, with an optional sliding window and sinks.
//
// What it computes: for each sequence s (one query token at position ctx - 1)
// and query head h,
//   out[s,h,:] = sum_j softmax_j(scale * q[s,h,:] . K_j) V_j
// over the visible tokens j < ctx: all of them without a window, else those
// with j >= ctx - window or j < sinks.
//
// Bound: every visible K/V byte is read once, so HBM bandwidth -- provided
// that the arithmetic keeps up.  At 4 bits an SM is handed a 16-token record
// of one head (1152 bytes) every 49 cycles (6.8 TB/s, 152 SMs, 1.9 GHz), 196
// issue slots of its four schedulers together; one fp32 FMA per (value, query
// head) would need 256 for four heads.  So both products run on mma.sync
// m16n8k16 with the tokens (Q K^T) or the dimensions (P V) as the 16 rows and
// the query heads of the GQA group as the 8 columns (a single token's few
// heads leave a tcgen05 tile of 128 rows nearly empty); the operands come
// straight from shared memory into registers, with no dequantised copy: 38
// cycles a record and head with all warps busy.
//
// 4-bit codes as operands.  A code in the low bits of a 16-bit word is the
// fp16 subnormal c * 2^-24, in bits 4..7 it is 16 c * 2^-24: one AND turns two
// codes into an operand register, and the factors 2^24 and 16 go into q and the
// final scale.  The k order of a product is free, so lane t of a row takes
// the row's dimensions 16 t .. 16 t + 15 as one 8-byte load.  Per row
//   scale q . K_j = s_j (q . c_j) F + z_j sum(q),
// and for V the weight p_j s_j multiplies c_j - 7.5 (one packed operation)
// while p_j (z_j + 7.5 s_j) is summed in fp32 beside it: centred codes keep the
// long sum as small as the output, so fp32 accumulation loses nothing to
// cancellation.  That operation also makes them normal numbers: subnormal ones
// cost ten times the error (4 10^-6 of the output's norm against 3 10^-7, 64
// sequences of 0.5-4k tokens), as if the tensor core aligned a sum's terms by
// their exponent fields and left its upper bits empty.  q (bf16) is exact in fp16
// after a power-of-two scale of its head's.
//
// P in parts.  The weights p are fp32; two fp16 parts keep 22 bits of them,
// three bf16 parts all 24, so the fp32 output carries no rounding of P.  With
// four query heads or fewer the products' spare columns 4..7 take another
// chunk (4-bit) or the lo parts (bf16) at no cost; with five to eight each part
// takes a product of its own.  The tensor cores truncate what they add, so a sum
// runs through four products at most (4-bit: a head's q . c, a stage's P V; bf16: the
// parts of P): each stage starts a fresh one, added in fp32.
//
// Work split.  The visible 16-token chunks of all sequences form one line, cut
// into equal ranges, one CTA per SM and KV-head group, each sequence start
// counted as `seg_weight` chunks more.  A range's piece of a sequence is a
// segment; one that covers its whole sequence writes the output, any other a
// partial (m, l, acc) record; the CTA that holds a split sequence's first
// chunk lists it for the merge kernel.  (Merged by the last CTA to finish, found
// through counters, the launch was slower: 29.2 against 27.6 us, batch of 64.)
//
// CTA.  Consumer warps, `wph` per KV head, each with its own ring of
// shared-memory stages of up to four chunks, one mbarrier each, so no warp waits
// for another's stage; stage k of a segment goes to the head's warp k mod wph.
// min(wph, 4) producer warps fill the rings (bulk copies of whole 16-token runs
// of the 4-bit cache, swizzled tensor copies of the bf16 one): a stage costs a
// producer some 1300 cycles of look-ups, waits and issue, one after the other
// (8 sequences of 32k-128k tokens, 4 bits: 103 us with one, 80 with two, 67 with
// three, one a ring).  More would have to share rings, whose parities cannot
// tell fills two laps apart.  The warps of a head combine at a segment's end
// through shared memory.  All waits are bounded.
//
// Measured, us per call: 4 bits, G = 4: 64 sequences of 0.5-4k tokens 26.3 (the
// copies alone: 21.7), 8 of 32k-128k 67.2 (0.80 of HBM; copies alone 61.3); G =
// 8: 256 with a window of 2048 41.6 (copies alone 29.4; 16 consumer warps of 96
// registers, a chunk at a time, 45.9; four chunks a stage, 44.2).  bf16: 256
// sequences, window 1024, 50.6, which is the copies alone; 8 long ones 84 to 85
// (0.94 of HBM).  A call's fixed part is about 9 us: the schedule 1.4, the first data
// 3 to 4.6, the merge 4.4.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <mutex>

#include "device.cuh"
#include "kernels.h"
#include "kv4.cuh"
#include "tc.cuh"

namespace tvl {
namespace {

constexpr int kD = 64;
constexpr int kChunk = 16;
constexpr int kMaxProducers = 4;
constexpr int kMaxThreads = (12 + kMaxProducers) * 32;
constexpr uint32_t kBf16Tile = kChunk * kD * 2;   // one head's K (or V) of a chunk
constexpr float kMaxSum = 256.0f;             // a lane's weights under the reference maximum
constexpr float kMaxProduct = 32768.0f;        // 4-bit: a lane's weights times its V scales
// 4-bit: the weights are held against max(V scale, kLeastScale), so that rows of one
// value (scale 0) count too: with V below 2^60 a lane's weights stay below 2^49 and
// their sums with the offsets below 2^109 a stage: room for 2^14 stages of a column's
// eight lanes (10^6 tokens of a warp).
constexpr float kLeastScale = 5.820766091346741e-11f;      // 2^-34
constexpr float kLog2e = 1.4426950408889634f;
constexpr unsigned kFull = 0xffffffffu;
constexpr uint32_t kSmemLimit = 227 * 1024;
// Cost of a sequence start, in chunks: a partly filled stage, the warps' meeting
// and the store.  Measured on batches of 64 (4-bit, 0.5k-4k tokens: 28.4 us at
// 4, 27.3 at 16, 27.7 at 32) and 256 (bf16, window 1024: 51.2 us at 1, 50.9 at
// 4, 51.6 at 6).
constexpr int kSegWeight4 = 14, kSegWeight16 = 3;

// First token of a chunk that stands in for a missing one: past every context (at
// most 2^31 - 128 tokens), and its 16 tokens still fit 32 bits.
constexpr int kUnseenToken = 0x7fffffe0;

constexpr int kCombPitch = 72;                // floats a head of a warp hands over: 64 + m, l

enum Format : int { kBf16 = 0, k4Bit = 1 };
// Bits of a stage's flags: the warp's first and last stage of the segment; no
// more stages; not all chunks present and visible.  From bit 8: how many of a
// head's warps have stages of the segment.
enum : int { kSegFirst = 1, kSegLast = 2, kTerminate = 4, kPartial = 8, kPartsShift = 8 };

// chunks of a stage: what a warp works on at once (independent work in flight)
template <int F, bool kLoCols>
__host__ __device__ constexpr int chunks_per_stage() { return F == k4Bit ? (kLoCols ? 4 : 2) : 1; }
template <int F, bool kLoCols>
__host__ __device__ constexpr int max_warps() { return F == k4Bit ? 12 : 8; }
template <int F, bool kLoCols>
__host__ __device__ constexpr int max_heads() { return F == k4Bit ? 4 : 8; }

struct alignas(16) StageMeta {
  int seq, record, flags, n;   // n: chunks in the stage
  int v0, ns, delta, ctx;      // first virtual chunk; sink chunks; token chunk = v + (v >= ns) * delta
};

struct Params {
  float* out;
  const __nv_bfloat16* q;
  const uint8_t* kv4;
  const int32_t* block_tables;
  const int32_t* context_lens;
  int num_seqs, hq, hkv, group, num_blocks, max_blocks;
  int cpb_log2;          // log2 of the 16-token chunks in a block
  int window, sinks;     // window 0: none
  int hpc, wph, cps_log2;
  int stages, ring;      // wph rings of `ring` stages
  int producers;         // warps that fill them: warp j the rings j, j + producers, ...
  uint32_t stage_bytes, kv_bytes;
  float scale_log2;
  int ctas, seg_weight;
  int small;             // schedule_small serves
  float* ws_m;           // records [2 * ctas][hq]
  float* ws_l;
  float* ws_acc;
  int4* ws_split;        // split sequences: (seq or -1, first record, first CTA, last CTA); entry
                         // per sequence, or per CTA that holds the first chunk when there are
                         // more sequences than CTAs
  long long* ws_total;   // length of the cost line
  uint32_t* status;
};

struct Layout {
  uint32_t meta, bars, comb, sched, total;
};

__host__ __device__ inline uint32_t align_up(uint32_t x, uint32_t a) { return (x + a - 1) / a * a; }

__host__ __device__ inline Layout make_layout(int stages, uint32_t stage_bytes, int hpc, int wph,
                                              int group) {
  Layout l;
  uint32_t off = stages * stage_bytes;
  l.meta = off;
  off += stages * sizeof(StageMeta);
  l.bars = off;                                        // full, empty; hand-over full, empty a warp
  off += (2 * stages + 2 * hpc * wph) * 8;
  l.comb = align_up(off, 16);
  off = l.comb + wph * hpc * group * kCombPitch * 4;
  l.sched = align_up(off, 16);                         // the schedule, scan totals, lengths
  off = l.sched + 64 + 32 * 8 + kMaxThreads * 4;
  l.total = off;
  return l;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Weight of a partial result with reference maximum m under the common one.
// m = -inf with anything in it means scores that were all NaN: kept as NaN.
__device__ __forceinline__ float weight_of(float m, float common) {
  return m == -INFINITY ? 1.f : ex2(m - common);
}

__device__ __forceinline__ int load_ctx(const Params& p, int s) {
  int c = p.context_lens[s];
  const long long cap = static_cast<long long>(p.max_blocks) << (p.cpb_log2 + 4);
  if (c < 0 || c > cap) {
    report(p.status, TVL_DEV_BAD_CONTEXT_LEN);
    c = c < 0 ? 0 : static_cast<int>(cap);
  }
  return c;
}

// The visible chunks of a sequence: ns chunks from 0 (sinks), then the window's
// from w0.  Virtual chunk v is token chunk v for v < ns, else v - ns + w0.
struct Visible {
  int ns, delta, n;
};
__device__ __forceinline__ Visible visible_of(const Params& p, int ctx) {
  const int first = p.window > 0 && ctx > p.window ? ctx - p.window : 0;
  const int w0 = first / kChunk;
  const int sc = p.sinks / kChunk + (p.sinks % kChunk != 0 ? 1 : 0);
  Visible v;
  v.ns = min(sc, w0);
  v.delta = w0 - v.ns;
  v.n = (ctx + kChunk - 1) / kChunk - v.delta;
  return v;
}
__device__ __forceinline__ long long seq_cost(int n, int w) { return n > 0 ? n + w : 0; }

// ------------------------------------------------------------------ schedule

struct Schedule {
  int seq0, v0;          // first sequence and virtual chunk
  int seq_end, v_end;    // ends before chunk v_end of sequence seq_end
  long long total, hi;   // the cost line's length, this CTA's end on it
};

__device__ void block_scan(long long v, long long& incl, long long& total, long long* tmp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) tmp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    long long w = lane < nw ? tmp[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(kFull, w, o);
      if (lane >= o) w += y;
    }
    if (lane < nw) tmp[lane] = w;
  }
  __syncthreads();
  incl = x + (warp > 0 ? tmp[warp - 1] : 0);
  total = tmp[nw - 1];
  __syncthreads();
}

// A batch of at most one sequence a thread whose line surely fits 32 bits times
// the CTAs (the host checks): one scan, each warp adding up the totals of those
// before it, and the threads whose sequences hold the CTA's two ends record
// them.  Every thread whose sequence has chunks in the range prefetches their
// block table entries for the producer.
__device__ __forceinline__ void schedule_small(const Params& p, Schedule* sc, int* tmp, int* lens) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  const int w = p.seg_weight;
  Visible vis = {0, 0, 0};
  if (tid < p.num_seqs) {
    const int ctx = load_ctx(p, tid);
    lens[tid] = ctx;                       // for the producer
    vis = visible_of(p, ctx);
  }
  const int mine = vis.n > 0 ? vis.n + w : 0;
  int x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) tmp[warp] = x;
  if (tid == 0) {
    sc->seq0 = sc->seq_end = p.num_seqs;
    sc->v0 = sc->v_end = 0;
  }
  __syncthreads();
  const int part = lane < nw ? tmp[lane] : 0;
  const int total = __reduce_add_sync(kFull, part);
  const int excl = __reduce_add_sync(kFull, lane < warp ? part : 0) + x - mine;
  const int lo = static_cast<uint32_t>(total) * blockIdx.x / static_cast<uint32_t>(p.ctas);
  const int hi = static_cast<uint32_t>(total) * (blockIdx.x + 1) / static_cast<uint32_t>(p.ctas);
  if (mine > 0 && excl <= lo && lo < excl + mine) {
    sc->seq0 = tid;
    sc->v0 = max(0, lo - excl - w);
  }
  if (mine > 0 && excl <= hi && hi < excl + mine) {
    sc->seq_end = tid;
    sc->v_end = max(0, hi - excl - w);
  }
  if (tid == 0) {
    sc->total = total;
    sc->hi = hi;
  }
  const int a = max(0, lo - excl - w), b = min(vis.n, hi - excl - w);
  const int32_t* row = p.block_tables + static_cast<long long>(tid) * p.max_blocks;
  for (int v = a; v < b; v += 32 << p.cpb_log2)
    asm volatile("prefetch.global.L1 [%0];" ::"l"(row + ((v < vis.ns ? v : v + vis.delta) >> p.cpb_log2)));
}

// Every thread sums the costs of a contiguous slice of the sequences; one
// scan places the slices on the line, and the threads whose slices hold this
// CTA's two ends walk them again.
__device__ __noinline__ void make_schedule(const Params& p, Schedule* sc, long long* tmp) {
  const int tid = threadIdx.x, cta = blockIdx.x, w = p.seg_weight;
  const int per = (p.num_seqs + blockDim.x - 1) / blockDim.x;
  const int s_lo = min(p.num_seqs, tid * per), s_hi = min(p.num_seqs, s_lo + per);
  long long mine = 0;
  for (int s = s_lo; s < s_hi; ++s) mine += seq_cost(visible_of(p, load_ctx(p, s)).n, w);
  if (tid == 0) {
    sc->seq0 = sc->seq_end = p.num_seqs;
    sc->v0 = sc->v_end = 0;
  }
  long long incl, total;
  block_scan(mine, incl, total, tmp);      // its barriers order the initial values
  const long long excl = incl - mine;
  const long long lo = total * cta / p.ctas, hi = total * (cta + 1) / p.ctas;
  auto locate = [&](long long x, int& seq, int& v) {
    long long run = excl;
    for (int s = s_lo; s < s_hi; ++s) {
      const long long c = seq_cost(visible_of(p, load_ctx(p, s)).n, w);
      if (x < run + c) {
        seq = s;
        v = static_cast<int>(x - run - w > 0 ? x - run - w : 0);
        return;
      }
      run += c;
    }
  };
  if (mine > 0 && excl <= lo && lo < incl) locate(lo, sc->seq0, sc->v0);
  if (mine > 0 && excl <= hi && hi < incl) locate(hi, sc->seq_end, sc->v_end);
  if (tid == 0) {
    sc->total = total;
    sc->hi = hi;
  }
}

// ------------------------------------------------------------------ producer

struct Segment {
  int s, v, e, ctx, ns, delta, n, record, window;
};

template <int F>
__device__ void producer(const Params& p, const Schedule& sc, uint8_t* smem, const Layout& L, int pj,
                         const CUtensorMap* tm_k, const CUtensorMap* tm_v) {
  const int lane = threadIdx.x & 31;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L.bars);
  uint64_t* empty = full + p.stages;
  StageMeta* meta = reinterpret_cast<StageMeta*>(smem + L.meta);
  const int hpc = p.hpc, h0 = blockIdx.z * hpc, cta = blockIdx.x;
  const uint32_t chunk_bytes = hpc * (F == k4Bit ? kRecBytes : 2 * kBf16Tile);
  const uint32_t q_bytes = hpc * p.group * kD * 2;
  const uint64_t stream_policy = policy_evict_first();
  const uint64_t keep_policy = policy_evict_last();
  if (F == kBf16 && lane == 0) {
    prefetch_tensormap(tm_k);
    prefetch_tensormap(tm_v);
  }

  const int cps = 1 << p.cps_log2, wph = p.wph, ring = p.ring;
  // Stage k of a segment goes to the head's warps k % wph, each with a ring of
  // its own.  Lane w < wph: warps w's next stage, in bit 8 its fill's parity and
  // in bit 9 whether every stage of the ring has been filled.
  int state = 0;
  bool ok = true;

  // lens: the lengths, of a small batch; else lane i's win_ctx: sequence win + i's
  const int* lens = reinterpret_cast<const int*>(smem + L.sched + 64 + 32 * 8);
  int win = -64, win_ctx = 0;
  // The segment that starts at chunk v of sequence s or after it; false: none left.
  auto find = [&](int s, int v, bool first, Segment& g) {
    for (;; ++s, v = 0) {
      if (s >= p.num_seqs || s > sc.seq_end || (s == sc.seq_end && v >= sc.v_end)) return false;
      if (p.small) {
        g.ctx = lens[s];
      } else {
        if (s < win || s >= win + 32) {
          win = s;
          win_ctx = s + lane < p.num_seqs ? load_ctx(p, s + lane) : 0;
        }
        g.ctx = __shfl_sync(kFull, win_ctx, s - win);
      }
      const Visible vis = visible_of(p, g.ctx);
      if (v >= vis.n) continue;
      g.s = s;
      g.v = v;
      g.e = s == sc.seq_end ? min(sc.v_end, vis.n) : vis.n;
      g.ns = vis.ns;
      g.delta = vis.delta;
      g.n = vis.n;
      g.window = p.window > 0 ? min(p.window, g.ctx) : g.ctx;
      g.record = v == 0 && g.e == vis.n ? -1 : 2 * cta + (first ? 0 : 1);
      return true;
    }
  };
  // this lane's block table entry: chunk vb + lane of the segment
  auto entry = [&](const Segment& g, int vb) {
    const int v = vb + lane;
    if (v >= g.e) return 0;
    const int c = v < g.ns ? v : v + g.delta;
    return p.block_tables[static_cast<long long>(g.s) * p.max_blocks + (c >> p.cpb_log2)];
  };

  const bool by_seq = p.num_seqs <= p.ctas && blockIdx.z == 0;
  int4 split = make_int4(-1, 0, 0, 0);
  Segment g;
  bool have = find(sc.seq0, sc.v0, true, g);
  int tbl = have ? entry(g, g.v) : 0;
  while (have && ok) {
    if (g.v == 0 && g.e < g.n) {
      // a split sequence's first piece: it ends at this CTA's end of the
      // line, and the sequence's last chunk lies g.n - g.e - 1 places on
      const long long x = sc.hi + (g.n - g.e) - 1;
      split = make_int4(g.s, g.record, cta, static_cast<int>(((x + 1) * p.ctas - 1) / sc.total));
    }
    if (by_seq && pj == 0 && g.v == 0 && lane == 0)
      p.ws_split[g.s] = g.e < g.n ? split : make_int4(-1, 0, 0, 0);
    Segment nx;
    const bool have_next = find(g.s, g.e, false, nx);
    const int n_stages = (g.e - g.v + cps - 1) >> p.cps_log2;
    const int parts = min(wph, n_stages);
    // the producer's own stages: k (of warp w) with w = k % wph, w % producers == pj
    int k = pj, w = pj, vb = g.v;
    int ntbl = vb + 32 < g.e ? entry(g, vb + 32) : (have_next ? entry(nx, nx.v) : 0);
    for (;;) {
      const int v = g.v + (k << p.cps_log2);
      if (v >= g.e) break;
      while (v >= vb + 32) {          // the next 32 entries (of this segment or the next)
        vb += 32;                     // are fetched while this batch's copies are issued
        tbl = ntbl;
        ntbl = vb + 32 < g.e ? entry(g, vb + 32) : (have_next ? entry(nx, nx.v) : 0);
      }
      const int n = min(cps, g.e - v);                  // lane i < n: chunk v + i
      const int rs = __shfl_sync(kFull, state, w);
      const int at = rs & 0xff, slot = w * ring + at;
      const uint32_t sp = rs >> 8 & 1;
      uint8_t* base = smem + static_cast<size_t>(slot) * p.stage_bytes;
      const int vv = v + lane;
      const int c = vv < g.ns ? vv : vv + g.delta;
      const bool whole = c * kChunk + kChunk <= g.ctx &&
                         (c * kChunk >= g.ctx - g.window || c * kChunk + kChunk <= p.sinks);
      const bool all = __all_sync(kFull, lane >= n || whole);
      int page = __shfl_sync(kFull, tbl, (v - vb + lane) & 31);
      if (lane < n && (page < 0 || page >= p.num_blocks)) {
        report(p.status, TVL_DEV_BAD_BLOCK_ID);
        page = 0;
      }
      const long long chunk = (static_cast<long long>(page) << p.cpb_log2) + (c & ((1 << p.cpb_log2) - 1));
      const bool first = k < wph;
      if (rs >> 9 && !__all_sync(kFull, mbar_wait(&empty[slot], sp ^ 1))) {
        ok = false;
        break;
      }
      if (lane == 0) {
        StageMeta m;
        m.seq = g.s;
        m.record = g.record;
        m.flags = parts << kPartsShift | (first ? kSegFirst : 0) |
                  (k + wph >= n_stages ? kSegLast : 0) | (all && n == cps ? 0 : kPartial);
        m.n = n;
        m.v0 = v;
        m.ns = g.ns;
        m.delta = g.delta;
        m.ctx = g.ctx;
        meta[slot] = m;
        mbar_arrive_expect_tx(&full[slot], n * chunk_bytes + (first ? q_bytes : 0));
      }
      __syncwarp();
      if (lane < n) {
        if (F == k4Bit) {
          bulk_load(base + lane * chunk_bytes, p.kv4 + (chunk * p.hkv + h0) * kRecBytes, chunk_bytes,
                    &full[slot], stream_policy);
        } else {
          const int tok = static_cast<int>(chunk * kChunk);
          const uint32_t half = hpc * kBf16Tile;
          tma_load_3d(base + lane * half, tm_k, 0, tok, h0, &full[slot]);
          tma_load_3d(base + p.kv_bytes / 2 + lane * half, tm_v, 0, tok, h0, &full[slot]);
        }
      }
      if (first && lane == 31)
        bulk_load(base + p.kv_bytes,
                  p.q + (static_cast<size_t>(g.s) * p.hq + static_cast<size_t>(h0) * p.group) * kD,
                  q_bytes, &full[slot], keep_policy);
      if (lane == w) state = at + 1 == ring ? (rs ^ 0x100) - at | 0x200 : rs + 1;
      if (w + p.producers < wph) {
        w += p.producers;
        k += p.producers;
      } else {
        k += wph - w + pj;
        w = pj;
      }
    }
    // the next segment's first entries: already at hand in the last batch
    if (have_next) tbl = vb + 32 < g.e ? entry(nx, nx.v) : ntbl;
    g = nx;
    have = have_next;
  }
  if (blockIdx.z == 0 && lane == 0 && pj == 0) {
    if (!by_seq) p.ws_split[cta] = split;
    if (cta == 0) *p.ws_total = sc.total;
  }
  int pos = state & 0xff;
  uint32_t ph = state >> 8 & 1;
  bool used = state >> 9 != 0;
  if (lane < wph && lane % p.producers == pj) {   // each ring's last stage; then its copies land
    if (ok && used) ok = mbar_wait(&empty[lane * ring + pos], ph ^ 1);
    if (ok) {
      meta[lane * ring + pos].flags = kTerminate;
      mbar_arrive(&full[lane * ring + pos]);
      if (++pos == ring) {
        pos = 0;
        ph ^= 1;
        used = true;
      }
    } else {
      report(p.status, kDevTimeout);
    }
    const int fills = used ? ring : pos;
    for (int i = 0; i < fills; ++i) {
      if (--pos < 0) {
        pos = ring - 1;
        ph ^= 1;
      }
      if (!mbar_wait(&full[lane * ring + pos], ph)) report(p.status, kDevTimeout);
    }
  }
}

// ----------------------------------------------------------------- consumers

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same with a zero accumulator in
__device__ __forceinline__ void mma_f16_0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16_0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                           uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ float2 add2(float a0, float a1, float b0, float b1) {
  return __fadd2_rn(make_float2(a0, a1), make_float2(b0, b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// the 8 x 8 matrix of 16-bit elements held one row per lane quad, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// 2^15 a + b on fp16 pairs
__device__ __forceinline__ uint32_t half2_raise(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(0x78007800u), "r"(b));
  return d;
}
__device__ __forceinline__ float2 meta_sz(uint32_t w) { return bf16x2_to_float2(w); }
// a K row's (s, z) times the softmax scale's magnitude: what then brings a score to
// log2 is a power of two, so that the exponent x kf - m is exact for the largest
// score, however large (with the scale in kf: NaN past 2^26; now 0.4% slower)
__device__ __forceinline__ float2 k_scaled(const Params& p, uint32_t w) {
  const float f = fabsf(p.scale_log2);
  return __fmul2_rn(meta_sz(w), make_float2(f, f));
}
// a V row's scale s and the offset z + 7.5 s of its centred codes
__device__ __forceinline__ float2 v_scale_offset(uint32_t w) {
  const float2 m = meta_sz(w);
  return make_float2(m.x, fmaf(7.5f, m.x, m.y));
}

template <int F>
__device__ __forceinline__ uint32_t pack16(float2 v) {
  if constexpr (F == k4Bit) {
    const __half2 h = __floats2half2_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <int F>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
  if constexpr (F == k4Bit) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return bf16x2_to_float2(w);
}

// Row r of the 16 rows of a product is token row_token(r) of the chunk.  With
// 4-bit rows of 32 bytes this order leaves both the K loads (8 bytes a lane,
// rows 0..3 and 4..7 a half warp each) and the V loads (4 bytes a lane, rows of
// one parity together) free of bank conflicts: tokens of a group differ mod 4.
template <int F>
__device__ __forceinline__ int row_token(int r) {   // r < 8
  if (F == kBf16) return r;
  return (0x57463120 >> (4 * r)) & 7;               // 0 2 1 3 6 4 7 5
}

// A lane (g = lane / 4, t = lane % 4) holds columns 2 t and 2 t + 1: `x`, `y`.
struct State {
  uint32_t qf[4][2];   // q as the column operand
  uint32_t qg[4][2];   // 4-bit, up to four heads: qf has columns 0..3, qg columns 4..7
  float acc[4][4];     // output rows, see out_dim
  float2 m, l, zs;     // reference maximum (log2), sum of p, sum of p (z + 7.5 s)
  float2 qsum;         // 4-bit: sum(q), in the units of q . c
  float2 kf;           // 4-bit: from those units to log2, powers of two
};

// acc[i][0..1] is output dimension out_dim(i, 0), acc[i][2..3] out_dim(i, 1)
template <int F>
__device__ __forceinline__ int out_dim(int g, int i, int half) {
  return F == k4Bit ? 8 * g + 2 * i + half : 16 * i + 8 * half + g;
}

template <int F, bool kLoCols>
__device__ __forceinline__ void load_q(State& st, const Params& p, const uint8_t* qbase) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int h = kLoCols ? (g & 3) : g;
  const bool live = h < p.group;
  const uint32_t* q = reinterpret_cast<const uint32_t*>(qbase + (live ? h : 0) * (kD * 2));
  if constexpr (F == kBf16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      st.qf[i][0] = live ? q[8 * i + t] : 0u;
      st.qf[i][1] = live ? q[8 * i + t + 4] : 0u;
    }
  } else {
    float v[16];
    float sum = 0.f, mx = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = bf16x2_to_float2(live ? q[8 * t + i] : 0u);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
      sum += f.x + f.y;
      if (fabsf(f.x) < INFINITY) mx = fmaxf(mx, fabsf(f.x));
      if (fabsf(f.y) < INFINITY) mx = fmaxf(mx, fabsf(f.y));
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {       // over the head's four lanes
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
      sum += __shfl_xor_sync(kFull, sum, o);
    }
    // the sign of the scale goes into q (and a zero scale makes q zero), so that
    // kf is positive and a masked -inf stays one
    const float sign = p.scale_log2 > 0.f ? 1.f : p.scale_log2 < 0.f ? -1.f : 0.f;
    // the head's largest |q| to [2^14, 2^15): exact in fp16 for every element down
    // to 2^-27 of it (a bf16 has 8 significant bits)
    int e = static_cast<int>(__float_as_uint(mx) >> 23) - 127;
    e = max(-100, min(100, e));
    const float up = sign * __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
    const float up16 = up * 0.0625f;
    const float kf = __uint_as_float(static_cast<uint32_t>(127 + 10 + e) << 23);
    st.kf.x = __shfl_sync(kFull, kf, 8 * t);
    st.kf.y = __shfl_sync(kFull, kf, 8 * t + 4);
    sum *= up * 5.9604644775390625e-08f;                             // 2^-24: a code's
    st.qsum.x = __shfl_sync(kFull, sum, 8 * t);
    st.qsum.y = __shfl_sync(kFull, sum, 8 * t + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = (i >> 1) * 8 + (i & 1) * 2;
      st.qf[i][0] = pack16<k4Bit>(make_float2(v[d] * up, v[d + 4] * up));
      st.qf[i][1] = pack16<k4Bit>(make_float2(v[d + 1] * up16, v[d + 5] * up16));
      if (kLoCols) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          st.qg[i][k] = g >= 4 ? st.qf[i][k] : 0u;
          if (g >= 4) st.qf[i][k] = 0u;
        }
      }
    }
  }
}

// Moves the reference maximum to cover mx (this lane's largest scores, log2), and
// rescales what is summed so far.  4-bit: the weights meet the V scales before
// they are rounded to fp16, so mx is the largest of score + log2 of the V row's
// scale (scaled_score) and the reference, a whole number (see normalise), is put
// where the largest product of a weight and a scale is 2^5 to 2^7.  It moves when a
// lane's bound on them passes 2^15, and only to such a place, so the largest
// product so far is at least 2^5 and the two fp16 parts keep every product to
// 2^-22 of itself or 2^-30 of the largest, however the scales are spread (below
// kLeastScale: of that scale's).  One reference scales numerator and denominator:
// the result does not depend on it.
template <int F, bool kPair>
__device__ __forceinline__ void move_reference(State& st, float2 mx) {
  constexpr int kFirst = kPair ? 2 : 4;      // a pair's two chunks share the columns' reference
#pragma unroll
  for (int o = kFirst; o < 32; o <<= 1) {
    mx.x = fmaxf(mx.x, __shfl_xor_sync(kFull, mx.x, o));
    mx.y = fmaxf(mx.y, __shfl_xor_sync(kFull, mx.y, o));
  }
  if (F == k4Bit) {
    mx.x = ceilf(mx.x) - 6.f;
    mx.y = ceilf(mx.y) - 6.f;
  }
  // never down: what was summed stays covered
  mx.x = fmaxf(mx.x, st.m.x);
  mx.y = fmaxf(mx.y, st.m.y);
  const float2 f = make_float2(ex2(st.m.x - mx.x), ex2(st.m.y - mx.y));
  st.m = mx;
  st.l = __fmul2_rn(st.l, f);
  st.zs = __fmul2_rn(st.zs, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    st.acc[i][0] *= f.x;
    st.acc[i][1] *= f.y;
    st.acc[i][2] *= f.x;
    st.acc[i][3] *= f.y;
  }
}

// scores x (in units of kf) of a row with V scale s, plus floor(log2 s)
__device__ __forceinline__ float2 scaled_score(float2 x, float2 kf, float s) {
  const int e = static_cast<int>(__float_as_uint(fmaxf(s, kLeastScale)) >> 23) - 127;
  const float f = static_cast<float>(e);
  return make_float2(fmaf(x.x, kf.x, f), fmaf(x.y, kf.y, f));
}
__device__ __forceinline__ float2 max2(float2 a, float2 b) {
  return make_float2(fmaxf(a.x, b.x), fmaxf(a.y, b.y));
}

// 4-bit: a column's sums, whose reference depends on the scales of V, in the units
// of its largest weight's power of two (m is a whole number, so this is exact):
// what is merged next then differs in m by no more than the scores do.
__device__ __forceinline__ void normalise(float& m, float& l, float (&o)[8]) {
  const int e = min(static_cast<int>(__float_as_uint(l) >> 23) - 127, 126);
  const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  m += static_cast<float>(e);
  l *= f;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] *= f;
}

__device__ __forceinline__ void add_to(float (&acc)[4], const float (&sum)[4]) {
  // The tensor core truncates what it accumulates, which over a long context
  // would pull the sums towards zero; across stages they add up here, rounded.
  const float2 a = add2(acc[0], acc[1], sum[0], sum[1]), b = add2(acc[2], acc[3], sum[2], sum[3]);
  acc[0] = a.x;
  acc[1] = a.y;
  acc[2] = b.x;
  acc[3] = b.y;
}

__device__ __forceinline__ uint32_t lds32(const uint8_t* p) {
  return *reinterpret_cast<const uint32_t*>(p);
}

constexpr uint32_t kLo = 0x000f000fu, kHi = 0x00f000f0u;
// fp16 pairs: -7.5 and -127.5 times 2^-9
constexpr uint32_t kMinus7 = 0xa380a380u, kMinus127 = 0xb3f8b3f8u;

// Scores of a 4-bit chunk's 16 rows: c = q . codes
__device__ __forceinline__ void codes_dot(float (&c)[4], const uint8_t* rec, const uint32_t (&qf)[4][2],
                                          int r0, int t) {
  const uint2 a = *reinterpret_cast<const uint2*>(rec + r0 * kRowCodes + t * 8);
  const uint2 b = *reinterpret_cast<const uint2*>(rec + (8 + r0) * kRowCodes + t * 8);
  mma_f16_0(c, a.x & kLo, b.x & kLo, a.x & kHi, b.x & kHi, qf[0][0], qf[0][1]);
  mma_f16(c, (a.x >> 8) & kLo, (b.x >> 8) & kLo, (a.x >> 8) & kHi, (b.x >> 8) & kHi, qf[1][0],
          qf[1][1]);
  mma_f16(c, a.y & kLo, b.y & kLo, a.y & kHi, b.y & kHi, qf[2][0], qf[2][1]);
  mma_f16(c, (a.y >> 8) & kLo, (b.y >> 8) & kLo, (a.y >> 8) & kHi, (b.y >> 8) & kHi, qf[3][0],
          qf[3][1]);
}

// The V codes of this lane's four tokens and eight dimensions, two tokens'
// codes of a dimension side by side: w[0..1] tokens (0, 1), w[2..3] tokens (8, 9)
// of the product's k order; byte pairs of dimensions 0..3 and 4..7.
__device__ __forceinline__ void load_v(uint32_t (&w)[4], const uint8_t* rec, int g, int t) {
  const uint8_t* vb = rec + kRecV + g * 4;
  const int ta = row_token<k4Bit>(2 * t) * kRowCodes, tb = row_token<k4Bit>(2 * t + 1) * kRowCodes;
  const uint32_t y0 = lds32(vb + ta), y1 = lds32(vb + tb);
  const uint32_t y2 = lds32(vb + ta + 8 * kRowCodes), y3 = lds32(vb + tb + 8 * kRowCodes);
  w[0] = __byte_perm(y0, y1, 0x5410);
  w[1] = __byte_perm(y0, y1, 0x7632);
  w[2] = __byte_perm(y2, y3, 0x5410);
  w[3] = __byte_perm(y2, y3, 0x7632);
}
// Rows 2 i, 2 i + 1 of the lane's dimensions as the row operand, centred: the
// even dimension's codes, 2^-9 (c - 7.5), and the whole bytes, 2^-9 (b - 127.5).  As b =
// c + 16 c', the odd dimension's 2^-5 (c' - 7.5) is the difference, taken once at the
// segment's end; a byte costs one operation to isolate, its high half two.
__device__ __forceinline__ void v_operand(uint32_t (&a)[4], const uint32_t (&w)[4], int i) {
  constexpr uint32_t kByte = 0x00ff00ffu;
  const uint32_t u0 = (i & 1) ? __byte_perm(w[i >> 1], 0, 0x4341) : w[i >> 1] & kByte;
  const uint32_t u1 = (i & 1) ? __byte_perm(w[2 + (i >> 1)], 0, 0x4341) : w[2 + (i >> 1)] & kByte;
  a[0] = half2_raise(u0 & kLo, kMinus7);
  a[1] = half2_raise(u0, kMinus127);
  a[2] = half2_raise(u1 & kLo, kMinus7);
  a[3] = half2_raise(u1, kMinus127);
}

// NP pairs of chunks, A and B, of a 4-bit head with at most four query heads.
// The product has eight columns; A's scores are formed in columns 0..3 (q is
// zero in the others) and B's in columns 4..7, so one pass of the softmax
// arithmetic serves both.  For P V the lo halves cross over (lane ^ 2): A's
// operand is (hi A, lo A), B's is (lo B, hi B); columns n and n + 4 are added
// at the segment's end.  tok: the first token of this lane's chunk of each pair.
template <int NP, bool kMasked>
__device__ __forceinline__ void process_pairs(State& st, const Params& p, const uint8_t* const (&ra)[NP],
                                              const uint8_t* const (&rb)[NP], const int (&tok)[NP],
                                              int ctx) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const bool second = t >= 2;
  const int r0 = row_token<k4Bit>(g);
  float2 x0[NP], x1[NP], v0[NP], v1[NP], w0[NP], w1[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const uint8_t* mine = second ? rb[i] : ra[i];
    const float2 k0 = k_scaled(p, lds32(mine + kRecKMeta + r0 * 4));
    const float2 k1 = k_scaled(p, lds32(mine + kRecKMeta + r0 * 4 + 32));
    v0[i] = v_scale_offset(lds32(mine + kRecVMeta + r0 * 4));
    v1[i] = v_scale_offset(lds32(mine + kRecVMeta + r0 * 4 + 32));
    float a[4], b[4];
    codes_dot(a, ra[i], st.qf, r0, t);
    codes_dot(b, rb[i], st.qg, r0, t);
    add_to(a, b);            // each is zero in the other's columns
    x0[i] = make_float2(fmaf(a[0], k0.x, st.qsum.x * k0.y), fmaf(a[1], k0.x, st.qsum.y * k0.y));
    x1[i] = make_float2(fmaf(a[2], k1.x, st.qsum.x * k1.y), fmaf(a[3], k1.x, st.qsum.y * k1.y));
    if (kMasked) {
      const int first = p.window > 0 && ctx > p.window ? ctx - p.window : 0;
      const int k = tok[i] + r0;
      if (!(k < ctx && (k >= first || k < p.sinks))) {
        x0[i] = make_float2(-INFINITY, -INFINITY);
        v0[i] = make_float2(0.f, 0.f);
      }
      if (!(k + 8 < ctx && (k + 8 >= first || k + 8 < p.sinks))) {
        x1[i] = make_float2(-INFINITY, -INFINITY);
        v1[i] = make_float2(0.f, 0.f);
      }
    }
  }
  float2 sum;
  auto weights = [&]() {
    const float2 nm = make_float2(-st.m.x, -st.m.y), kf = st.kf;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const float2 d0 = __ffma2_rn(x0[i], kf, nm), d1 = __ffma2_rn(x1[i], kf, nm);
      w0[i] = make_float2(ex2(d0.x), ex2(d0.y));
      w1[i] = make_float2(ex2(d1.x), ex2(d1.y));
      sum = i == 0 ? __fadd2_rn(w0[0], w1[0]) : __fadd2_rn(sum, __fadd2_rn(w0[i], w1[i]));
    }
  };
  weights();
  float sv = kLeastScale;
#pragma unroll
  for (int i = 0; i < NP; ++i) sv = fmaxf(sv, fmaxf(v0[i].x, v1[i].x));
  if (__any_sync(kFull, !(fmaxf(sum.x, sum.y) * sv <= kMaxProduct))) {
    float2 mx = make_float2(-INFINITY, -INFINITY);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      mx = max2(mx, scaled_score(x0[i], st.kf, v0[i].x));
      mx = max2(mx, scaled_score(x1[i], st.kf, v1[i].x));
    }
    move_reference<k4Bit, true>(st, mx);
    weights();
  }
  st.l = __fadd2_rn(st.l, sum);
  uint32_t oa[NP][2], ob[NP][2];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    st.zs.x = fmaf(w1[i].x, v1[i].y, fmaf(w0[i].x, v0[i].y, st.zs.x));
    st.zs.y = fmaf(w1[i].y, v1[i].y, fmaf(w0[i].y, v0[i].y, st.zs.y));
    w0[i] = make_float2(w0[i].x * v0[i].x, w0[i].y * v0[i].x);
    w1[i] = make_float2(w1[i].x * v1[i].x, w1[i].y * v1[i].x);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float2 w = r == 0 ? w0[i] : w1[i];
      const uint32_t hi = pack16<k4Bit>(w);
      const float2 back = unpack16<k4Bit>(hi);
      const uint32_t lo =
          __shfl_xor_sync(kFull, pack16<k4Bit>(make_float2(w.x - back.x, w.y - back.y)), 2);
      oa[i][r] = transpose8(second ? lo : hi);
      ob[i][r] = transpose8(second ? hi : lo);
    }
  }
  float d[4][4];
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    uint32_t wa[4], wb[4];
    load_v(wa, ra[k], g, t);
    load_v(wb, rb[k], g, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t a[4];
      v_operand(a, wa, i);
      if (k == 0)
        mma_f16_0(d[i], a[0], a[1], a[2], a[3], oa[k][0], oa[k][1]);
      else
        mma_f16(d[i], a[0], a[1], a[2], a[3], oa[k][0], oa[k][1]);
      v_operand(a, wb, i);
      mma_f16(d[i], a[0], a[1], a[2], a[3], ob[k][0], ob[k][1]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) add_to(st.acc[i], d[i]);
}

// N chunks of a 4-bit head with five to eight query heads; tok: their first
// tokens.  Every column is a query head, and the lo halves take products of
// their own.
template <int N, bool kMasked>
__device__ __forceinline__ void process_wide(State& st, const Params& p, const uint8_t* const (&rec)[N],
                                             const int (&tok)[N], int ctx) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int r0 = row_token<k4Bit>(g);
  float2 x[N][2], mv[N][2], w[N][2];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float c[4];
    codes_dot(c, rec[i], st.qf, r0, t);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float2 m = k_scaled(p, lds32(rec[i] + kRecKMeta + (r0 + 8 * r) * 4));
      mv[i][r] = v_scale_offset(lds32(rec[i] + kRecVMeta + (r0 + 8 * r) * 4));
      x[i][r] = make_float2(fmaf(c[2 * r], m.x, st.qsum.x * m.y),
                            fmaf(c[2 * r + 1], m.x, st.qsum.y * m.y));
      if (kMasked) {
        const int first = p.window > 0 && ctx > p.window ? ctx - p.window : 0;
        const int k = tok[i] + r0 + 8 * r;
        if (!(k < ctx && (k >= first || k < p.sinks))) {
          x[i][r] = make_float2(-INFINITY, -INFINITY);
          mv[i][r] = make_float2(0.f, 0.f);
        }
      }
    }
  }
  float2 sum;
  auto weights = [&]() {
    const float2 nm = make_float2(-st.m.x, -st.m.y), kf = st.kf;
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float2 d = __ffma2_rn(x[i][r], kf, nm);
        w[i][r] = make_float2(ex2(d.x), ex2(d.y));
        sum = i + r == 0 ? w[0][0] : __fadd2_rn(sum, w[i][r]);
      }
    }
  };
  weights();
  float sv = kLeastScale;
#pragma unroll
  for (int i = 0; i < N; ++i) sv = fmaxf(sv, fmaxf(mv[i][0].x, mv[i][1].x));
  if (__any_sync(kFull, !(fmaxf(sum.x, sum.y) * sv <= kMaxProduct))) {
    float2 mx = make_float2(-INFINITY, -INFINITY);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) mx = max2(mx, scaled_score(x[i][r], st.kf, mv[i][r].x));
    move_reference<k4Bit, false>(st, mx);
    weights();
  }
  st.l = __fadd2_rn(st.l, sum);
  uint32_t hi[N][2], lo[N][2];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float sc = mv[i][r].x;
      st.zs.x = fmaf(w[i][r].x, mv[i][r].y, st.zs.x);
      st.zs.y = fmaf(w[i][r].y, mv[i][r].y, st.zs.y);
      const float2 v = make_float2(w[i][r].x * sc, w[i][r].y * sc);
      const uint32_t h = pack16<k4Bit>(v);
      const float2 back = unpack16<k4Bit>(h);
      hi[i][r] = transpose8(h);
      lo[i][r] = transpose8(pack16<k4Bit>(make_float2(v.x - back.x, v.y - back.y)));
    }
  float d[4][4];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    uint32_t wv[4];
    load_v(wv, rec[k], g, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t a[4];
      v_operand(a, wv, i);
      if (k == 0)
        mma_f16_0(d[i], a[0], a[1], a[2], a[3], hi[k][0], hi[k][1]);
      else
        mma_f16(d[i], a[0], a[1], a[2], a[3], hi[k][0], hi[k][1]);
      mma_f16(d[i], a[0], a[1], a[2], a[3], lo[k][0], lo[k][1]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) add_to(st.acc[i], d[i]);
}

// One chunk of the bf16 cache: `chunk` is the K tile, the V tile lies v_off
// behind.  P is three bf16 parts: hi and lo share the columns with up to four
// query heads, and take a product each with more.
template <bool kLoCols, bool kMasked>
__device__ __forceinline__ void process_bf16(State& st, const Params& p, const uint8_t* chunk,
                                             uint32_t v_off, int tok0, int ctx) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int first = p.window > 0 && ctx > p.window ? ctx - p.window : 0;
  auto seen = [&](int tok) { return tok < ctx && (tok >= first || tok < p.sinks); };

  // --- scores: x[0] row g, x[1] row g + 8
  float2 x[2];
  {
    float c[4];
    const uint32_t base = smem_addr(chunk);
    const int row = (lane & 7) + (lane & 8);          // matrices 1 and 3: rows 8..15
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t a[4];
      ldsm4(a, base + row * 128 + (((2 * i + (lane >> 4)) ^ (row & 7)) << 4));
      // four sums of 16 products, added with rounding (see add_to)
      float d[4];
      mma_bf16_0(i == 0 ? c : d, a[0], a[1], a[2], a[3], st.qf[i][0], st.qf[i][1]);
      if (i > 0) add_to(c, d);
    }
    const float2 sl = make_float2(p.scale_log2, p.scale_log2);
    x[0] = __fmul2_rn(make_float2(c[0], c[1]), sl);
    x[1] = __fmul2_rn(make_float2(c[2], c[3]), sl);
  }
  if (kMasked) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
      if (!seen(tok0 + g + 8 * r)) x[r] = make_float2(-INFINITY, -INFINITY);
  }
  // --- online softmax
  float2 w[2], sum;
  auto weights = [&]() {
    const float2 nm = make_float2(-st.m.x, -st.m.y);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float2 d = __fadd2_rn(x[r], nm);
      w[r] = make_float2(ex2(d.x), ex2(d.y));
    }
    sum = __fadd2_rn(w[0], w[1]);
  };
  weights();
  if (__any_sync(kFull, !(fmaxf(sum.x, sum.y) <= kMaxSum))) {
    move_reference<kBf16, false>(st, max2(x[0], x[1]));
    weights();
  }
  st.l = __fadd2_rn(st.l, sum);
  // --- weights as the column operand of P V: rows of the transposed matrix are
  // the heads, its columns the tokens
  uint32_t hi[2], lo[2], lo2[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    hi[r] = pack16<kBf16>(w[r]);
    float2 back = unpack16<kBf16>(hi[r]);
    const float2 rest = make_float2(w[r].x - back.x, w[r].y - back.y);
    lo[r] = pack16<kBf16>(rest);
    back = unpack16<kBf16>(lo[r]);
    lo2[r] = transpose8(pack16<kBf16>(make_float2(rest.x - back.x, rest.y - back.y)));
    if (kLoCols && t >= 2) hi[r] = lo[r];
    hi[r] = transpose8(hi[r]);
    if (!kLoCols) lo[r] = transpose8(lo[r]);
  }
  if (kLoCols && g >= 4) lo2[0] = lo2[1] = 0u;        // columns 4..7 hold the lo parts' sums
  // --- O^T += V^T P^T
  const uint32_t base = smem_addr(chunk + v_off);
  const int tok = (lane & 7) + ((lane >> 4) << 3);    // matrices 2 and 3: tokens 8..15
  uint32_t keep[2] = {kFull, kFull};
  if (kMasked) {                                      // unseen slots may hold anything
#pragma unroll
    for (int r = 0; r < 2; ++r)
      keep[r] = (seen(tok0 + 8 * r + 2 * t) ? 0x0000ffffu : 0u) |
                (seen(tok0 + 8 * r + 2 * t + 1) ? 0xffff0000u : 0u);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t a[4];
    float o[4];
    ldsm4_t(a, base + tok * 128 + (((2 * i + ((lane >> 3) & 1)) ^ (tok & 7)) << 4));
    if (kMasked) {
      a[0] &= keep[0];
      a[1] &= keep[0];
      a[2] &= keep[1];
      a[3] &= keep[1];
    }
    mma_bf16_0(o, a[0], a[1], a[2], a[3], hi[0], hi[1]);
    if (!kLoCols) mma_bf16(o, a[0], a[1], a[2], a[3], lo[0], lo[1]);
    mma_bf16(o, a[0], a[1], a[2], a[3], lo2[0], lo2[1]);
    add_to(st.acc[i], o);
  }
}

// Sums the lanes' shares of a warp's state; o[column][2 i + half] is dimension
// out_dim(g, i, half) of the lane's columns.
template <int F, bool kLoCols>
__device__ __forceinline__ void lane_sums(State& st, float (&o)[2][8]) {
  constexpr bool kPair = F == k4Bit && kLoCols;
#pragma unroll
  for (int x = kPair ? 2 : 4; x < 32; x <<= 1) {
    st.l.x += __shfl_xor_sync(kFull, st.l.x, x);
    st.l.y += __shfl_xor_sync(kFull, st.l.y, x);
    if (F == k4Bit) {
      st.zs.x += __shfl_xor_sync(kFull, st.zs.x, x);
      st.zs.y += __shfl_xor_sync(kFull, st.zs.y, x);
    }
  }
  const float f0 = F == k4Bit ? 512.f : 1.f;          // the codes' 2^-9
  const float f1 = F == k4Bit ? f0 * 0.0625f : 1.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (kLoCols) st.acc[i][k] += __shfl_xor_sync(kFull, st.acc[i][k], 2);
    if (F == k4Bit) {           // bytes less their low halves (see v_operand)
      st.acc[i][2] -= st.acc[i][0];
      st.acc[i][3] -= st.acc[i][1];
    }
    o[0][2 * i] = fmaf(st.acc[i][0], f0, F == k4Bit ? st.zs.x : 0.f);
    o[1][2 * i] = fmaf(st.acc[i][1], f0, F == k4Bit ? st.zs.y : 0.f);
    o[0][2 * i + 1] = fmaf(st.acc[i][2], f1, F == k4Bit ? st.zs.x : 0.f);
    o[1][2 * i + 1] = fmaf(st.acc[i][3], f1, F == k4Bit ? st.zs.y : 0.f);
  }
  if (F == k4Bit) {
    normalise(st.m.x, st.l.x, o[0]);
    normalise(st.m.y, st.l.y, o[1]);
  }
}

// Ends a warp's part of a segment.  A head's warp 0, which has the segment's
// first stage, combines: the others with stages of it hand (m, l, o) over to it
// through shared memory, and it stores the output or the record.  handed: warp
// 0: bit i, the phase of warp i's next hand-over; else the hand-overs so far.
// False: a bounded wait ran out.
template <int F, bool kLoCols>
__device__ bool finish(State& st, const Params& p, uint8_t* smem, const Layout& L, int h, int w,
                       int& handed, int flags, int seq, int record) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint64_t* cfull = reinterpret_cast<uint64_t*>(smem + L.bars) + 2 * p.stages;
  uint64_t* cempty = cfull + p.hpc * p.wph;
  float* comb = reinterpret_cast<float*>(smem + L.comb);
  const int G = p.group;
  float o[2][8];
  lane_sums<F, kLoCols>(st, o);
  float m[2] = {st.m.x, st.m.y}, l[2] = {st.l.x, st.l.y};
  // columns 2 t and 2 t + 1 are heads of the group (not the lo halves' copies)
  const bool live[2] = {2 * t < G && !(kLoCols && t >= 2), 2 * t + 1 < G && !(kLoCols && t >= 2)};
  // a warp's hand-over of a head: eight floats a lane in lane order, then m, l
  if (w > 0) {
    const int me = w * p.hpc + h;
    if (handed > 0 && !mbar_wait(&cempty[me], (handed - 1) & 1)) return false;
    ++handed;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (!live[j]) continue;
      float* dst = comb + (me * G + 2 * t + j) * kCombPitch;
      reinterpret_cast<float4*>(dst)[2 * g] = make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
      reinterpret_cast<float4*>(dst)[2 * g + 1] = make_float4(o[j][4], o[j][5], o[j][6], o[j][7]);
      if (g == 0) *reinterpret_cast<float2*>(dst + 64) = make_float2(m[j], l[j]);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&cfull[me]);
    return true;
  }
  const int parts = flags >> kPartsShift;
  for (int i = 1; i < parts; ++i) {
    const int from = i * p.hpc + h;
    if (!mbar_wait(&cfull[from], handed >> i & 1)) return false;
    handed ^= 1 << i;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (!live[j]) continue;
      const float* src = comb + (from * G + 2 * t + j) * kCombPitch;
      const float4 a = reinterpret_cast<const float4*>(src)[2 * g];
      const float4 b = reinterpret_cast<const float4*>(src)[2 * g + 1];
      const float2 ml = *reinterpret_cast<const float2*>(src + 64);
      const float mn = fmaxf(m[j], ml.x);
      const float fa = weight_of(m[j], mn), fb = weight_of(ml.x, mn);
      m[j] = mn;
      l[j] = l[j] * fa + ml.y * fb;
      const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) o[j][k] = o[j][k] * fa + v[k] * fb;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&cempty[from]);
  }
  const int kvh = blockIdx.z * p.hpc + h;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (!live[j]) continue;
    const float sc = record < 0 ? 1.0f / l[j] : 1.0f;
    const long long row = static_cast<long long>(record < 0 ? seq : record) * p.hq + kvh * G + 2 * t + j;
    float* dst = (record < 0 ? p.out : p.ws_acc) + row * kD;
    if constexpr (F == k4Bit) {
      float4* d4 = reinterpret_cast<float4*>(dst + 8 * g);
      d4[0] = make_float4(o[j][0] * sc, o[j][1] * sc, o[j][2] * sc, o[j][3] * sc);
      d4[1] = make_float4(o[j][4] * sc, o[j][5] * sc, o[j][6] * sc, o[j][7] * sc);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) dst[out_dim<F>(g, k >> 1, k & 1)] = o[j][k] * sc;
    }
    if (record >= 0 && g == 0) {
      p.ws_m[row] = m[j];
      p.ws_l[row] = l[j];
    }
  }
  return true;
}

template <int F, bool kLoCols, int W>
__device__ void consumer(const Params& p, uint8_t* smem, const Layout& L) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = warp % p.hpc, w = warp / p.hpc;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L.bars);
  uint64_t* empty = full + p.stages;
  const StageMeta* meta = reinterpret_cast<const StageMeta*>(smem + L.meta);
  constexpr bool kPair = F == k4Bit && kLoCols;
  constexpr int NC = chunks_per_stage<F, kLoCols>();
  constexpr uint32_t kTile = F == k4Bit ? kRecBytes : kBf16Tile;
  const uint32_t mine = h * kTile;                          // the head's first chunk in a stage
  const uint32_t step = (W > 0 ? W : p.hpc) * kTile;       // to its next
  const uint32_t v_off = p.kv_bytes / 2;

  State st;
  int handed = 0;
  const int ring0 = w * p.ring;  // the warp's ring
  int stage = ring0;
  uint32_t ph = 0;
  auto release = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[stage]);
  };
  auto advance = [&]() {
    if (++stage == ring0 + p.ring) {
      stage = ring0;
      ph ^= 1;
    }
  };
  for (;;) {
    // whole stages inside a segment: a loop of their own, so that the compiler
    // keeps its registers for them
    int flags;
    const uint8_t* at;
    for (;;) {
      if (!mbar_wait(&full[stage], ph)) {
        if (lane == 0) report(p.status, kDevTimeout);
        return;
      }
      flags = meta[stage].flags;
      at = smem + static_cast<size_t>(stage) * p.stage_bytes + mine;
      if (flags & (kSegFirst | kSegLast | kTerminate | kPartial)) break;
      if constexpr (kPair) {
        constexpr int NP = NC / 2;
        const uint8_t *ra[NP], *rb[NP];
        int tok[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          ra[i] = at + 2 * i * step;
          rb[i] = ra[i] + step;
          tok[i] = 0;
        }
        process_pairs<NP, false>(st, p, ra, rb, tok, 0);
      } else if constexpr (F == k4Bit) {
        const uint8_t* rec[NC];
        int tok[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          rec[i] = at + i * step;
          tok[i] = 0;
        }
        process_wide<NC, false>(st, p, rec, tok, 0);
      } else {
#pragma unroll 1
        for (int i = 0; i < 1 << p.cps_log2; ++i)
          process_bf16<kLoCols, false>(st, p, at + i * step, v_off, 0, 0);
      }
      release();
      advance();
    }
    if (flags & kTerminate) return;
    const StageMeta& md = meta[stage];
    if (flags & kSegFirst) {
      load_q<F, kLoCols>(st, p, at - mine + p.kv_bytes + h * p.group * (kD * 2));
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) st.acc[i][k] = 0.f;
      st.m = make_float2(-INFINITY, -INFINITY);
      st.l = st.zs = make_float2(0.f, 0.f);
    }
    {
      // a segment's ends, a short stage, or one with slots that are not visible
      const int n = md.n, ctx = md.ctx, v0 = md.v0, ns = md.ns, delta = md.delta;
      auto token_of = [&](int j) { return (v0 + j < ns ? v0 + j : v0 + j + delta) * kChunk; };
      // a missing chunk of a group is stood in for by the first, all unseen
      auto rec_of = [&](int i) { return at + (i < n ? i : 0) * step; };
      auto tok_of = [&](int i) { return i < n ? token_of(i) : kUnseenToken; };
      if constexpr (kPair) {
        if (n > 2) {
          const uint8_t* ra[2] = {rec_of(0), rec_of(2)};
          const uint8_t* rb[2] = {rec_of(1), rec_of(3)};
          const int o = (lane & 2) >> 1;
          const int tok[2] = {tok_of(o), tok_of(2 + o)};
          process_pairs<2, true>(st, p, ra, rb, tok, ctx);
        } else {
          const uint8_t* ra[1] = {rec_of(0)};
          const uint8_t* rb[1] = {rec_of(1)};
          const int tok[1] = {tok_of((lane & 2) >> 1)};
          process_pairs<1, true>(st, p, ra, rb, tok, ctx);
        }
      } else if constexpr (F == k4Bit) {
        if (n > 1) {
          const uint8_t* rec[2] = {rec_of(0), rec_of(1)};
          const int tok[2] = {tok_of(0), tok_of(1)};
          process_wide<2, true>(st, p, rec, tok, ctx);
        } else {
          const uint8_t* rec[1] = {rec_of(0)};
          const int tok[1] = {tok_of(0)};
          process_wide<1, true>(st, p, rec, tok, ctx);
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < n; ++i)
          process_bf16<kLoCols, true>(st, p, rec_of(i), v_off, tok_of(i), ctx);
      }
    }
    const int seq = md.seq, record = md.record;
    release();
    if (flags & kSegLast) {
      if (!finish<F, kLoCols>(st, p, smem, L, h, w, handed, flags, seq, record)) {
        if (lane == 0) report(p.status, kDevTimeout);
        return;
      }
    }
    advance();
  }
}

template <int F, bool kLoCols, int W>
__global__ void __launch_bounds__((max_warps<F, kLoCols>() + kMaxProducers) * 32, 1)
    window_decode_kernel(const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  // 128-byte-swizzled tiles repeat every 1024 bytes
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const Layout L = make_layout(p.stages, p.stage_bytes, p.hpc, p.wph, p.group);
  Schedule* sched = reinterpret_cast<Schedule*>(smem + L.sched);
  long long* tmp = reinterpret_cast<long long*>(smem + L.sched + 64);
  int* lens = reinterpret_cast<int*>(smem + L.sched + 64 + 32 * 8);
  const int tid = threadIdx.x, warp = tid >> 5;
  const int consumers = p.hpc * p.wph;
  if (tid == 0) {
    uint64_t* b = reinterpret_cast<uint64_t*>(smem + L.bars);
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&b[i], 1);
      mbar_init(&b[p.stages + i], p.hpc);
    }
    for (int i = 0; i < 2 * consumers; ++i) mbar_init(&b[2 * p.stages + i], 1);
    fence_barrier_init();
  }
  grid_dependency_wait();        // inputs may come from the preceding kernel
  grid_dependents_launch();
  if (p.small)
    schedule_small(p, sched, reinterpret_cast<int*>(tmp), lens);
  else
    make_schedule(p, sched, tmp);
  __syncthreads();
  const Schedule sc = *sched;
  if (warp >= consumers) {
    producer<F>(p, sc, smem, L, warp - consumers, &tm_k, &tm_v);
  } else {
    // empty contexts have no chunk and so no segment: zero rows, dealt out
    const int n = p.hpc * p.group * kD;
    for (int s = blockIdx.x; s < p.num_seqs; s += p.ctas) {
      if (p.context_lens[s] > 0) continue;
      if (tid == 0 && blockIdx.z == 0 && p.num_seqs <= p.ctas) p.ws_split[s] = make_int4(-1, 0, 0, 0);
      float* dst = p.out + (static_cast<long long>(s) * p.hq + blockIdx.z * p.hpc * p.group) * kD;
      for (int i = tid; i < n; i += consumers * 32) dst[i] = 0.f;
    }
    consumer<F, kLoCols, W>(p, smem, L);
  }
}

// -------------------------------------------------------------------- direct

// Small batches of bounded length: CTA (x, z) does KV head z of sequence x alone,
// in one launch.  Warp w takes chunks w, w + 16, ... : it fetches their block
// ids, issues their copies (all of them fit) and q's loads, waits once, and the
// warps meet at the end.  Bound by latency: four dependent memory round trips.
// One sequence with a window of 512 (bf16) takes 4.7 us, against 9.6 through the
// schedule and the merge; one of 777 tokens (4 bits) 5.3 against 7.8.  A CTA must hold
// the whole sequence at once, and past one CTA an SM the balanced split wins.
constexpr int kDirectWarps = 16;
constexpr int kDirectChunks4 = 128, kDirectChunks16 = 48;    // longest sequence (chunks),
constexpr uint32_t kDirectSmem = kSmemLimit - 1024;          // if it fits (bf16, G = 8: 32)

template <int F, bool kLoCols>
__global__ void __launch_bounds__(kDirectWarps * 32, 1)
    window_direct_kernel(const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const Params p, int per_warp) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[kDirectWarps];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  constexpr uint32_t kBytes = F == k4Bit ? kRecBytes : 2 * kBf16Tile;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int seq = blockIdx.x, kvh = blockIdx.z, G = p.group;
  uint8_t* mine = smem + static_cast<size_t>(w) * per_warp * kBytes;
  float* comb = reinterpret_cast<float*>(smem + static_cast<size_t>(kDirectWarps) * per_warp * kBytes);
  if (lane == 0) {
    if (F == kBf16) {
      prefetch_tensormap(&tm_k);
      prefetch_tensormap(&tm_v);
    }
    mbar_init(&bars[w], 1);
    fence_barrier_init();
  }
  __syncwarp();
  grid_dependency_wait();
  grid_dependents_launch();
  const int ctx = load_ctx(p, seq);
  const Visible vis = visible_of(p, ctx);
  auto chunk_of = [&](int i) {               // the warp's i-th chunk as a token chunk
    const int v = w + kDirectWarps * i;
    return v < vis.ns ? v : v + vis.delta;
  };
  const int n = w < vis.n ? (vis.n - w + kDirectWarps - 1) / kDirectWarps : 0;   // <= per_warp <= 8
  if (n > 0) {
    int page = 0;
    if (lane < n) page = p.block_tables[static_cast<long long>(seq) * p.max_blocks + (chunk_of(lane) >> p.cpb_log2)];
    if (lane == 0) mbar_arrive_expect_tx(&bars[w], n * kBytes);
    __syncwarp();
    if (lane < n) {
      if (page < 0 || page >= p.num_blocks) {
        report(p.status, TVL_DEV_BAD_BLOCK_ID);
        page = 0;
      }
      const long long chunk = (static_cast<long long>(page) << p.cpb_log2) +
                              (chunk_of(lane) & ((1 << p.cpb_log2) - 1));
      if (F == k4Bit) {
        bulk_load(mine + lane * kBytes, p.kv4 + (chunk * p.hkv + kvh) * kRecBytes, kBytes, &bars[w],
                  policy_evict_first());
      } else {
        const int tok = static_cast<int>(chunk * kChunk);
        tma_load_3d(mine + lane * kBytes, &tm_k, 0, tok, kvh, &bars[w]);
        tma_load_3d(mine + lane * kBytes + kBf16Tile, &tm_v, 0, tok, kvh, &bars[w]);
      }
    }
  }
  State st;
  load_q<F, kLoCols>(st, p, reinterpret_cast<const uint8_t*>(
                                p.q + (static_cast<size_t>(seq) * p.hq + static_cast<size_t>(kvh) * G) * kD));
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) st.acc[i][k] = 0.f;
  st.m = make_float2(-INFINITY, -INFINITY);
  st.l = st.zs = make_float2(0.f, 0.f);
  if (n > 0 && !mbar_wait(&bars[w], 0) && lane == 0) report(p.status, kDevTimeout);
  // a missing second chunk is stood in for by the first, all unseen
  auto rec_of = [&](int i) -> const uint8_t* { return mine + (i < n ? i : 0) * kBytes; };
  auto tok_of = [&](int i) { return i < n ? chunk_of(i) * kChunk : kUnseenToken; };
#pragma unroll 1
  for (int i = 0; i < n; i += 2) {
    if constexpr (F == k4Bit && kLoCols) {
      const uint8_t* ra[1] = {rec_of(i)};
      const uint8_t* rb[1] = {i + 1 < n ? rec_of(i + 1) : rec_of(i)};
      const int tok[1] = {tok_of(i + ((lane & 2) >> 1))};
      process_pairs<1, true>(st, p, ra, rb, tok, ctx);
    } else if constexpr (F == k4Bit) {
      const uint8_t* rec[2] = {rec_of(i), rec_of(i + 1)};
      const int tok[2] = {tok_of(i), tok_of(i + 1)};
      process_wide<2, true>(st, p, rec, tok, ctx);
    } else {
      process_bf16<kLoCols, true>(st, p, rec_of(i), kBf16Tile, tok_of(i), ctx);
      if (i + 1 < n) process_bf16<kLoCols, true>(st, p, rec_of(i + 1), kBf16Tile, tok_of(i + 1), ctx);
    }
  }
  float o[2][8];
  lane_sums<F, kLoCols>(st, o);
  const float m[2] = {st.m.x, st.m.y}, l[2] = {st.l.x, st.l.y};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (2 * t + j >= G || (kLoCols && t >= 2)) continue;
    float* dst = comb + (w * G + 2 * t + j) * kCombPitch;
    reinterpret_cast<float4*>(dst)[2 * g] = make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
    reinterpret_cast<float4*>(dst)[2 * g + 1] = make_float4(o[j][4], o[j][5], o[j][6], o[j][7]);
    if (g == 0) *reinterpret_cast<float2*>(dst + 64) = make_float2(m[j], l[j]);
  }
  __syncthreads();
  if (w >= G) return;
  // warp w: query head w of the group, two dimensions a lane; lane i knows warp i's weight
  const float2 ml = lane < kDirectWarps
                        ? *reinterpret_cast<const float2*>(comb + (lane * G + w) * kCombPitch + 64)
                        : make_float2(-INFINITY, 0.f);
  float top = ml.x;
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, x));
  // (a warp without chunks: l and o are 0; all scores NaN: kept)
  const float mine_w = weight_of(ml.x, top);
  float den = ml.y * mine_w;
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) den += __shfl_xor_sync(kFull, den, x);
  float2 sum = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kDirectWarps; ++i) {
    const float wi = __shfl_sync(kFull, mine_w, i);
    const float2 v = reinterpret_cast<const float2*>(comb + (i * G + w) * kCombPitch)[lane];
    sum.x = fmaf(wi, v.x, sum.x);
    sum.y = fmaf(wi, v.y, sum.y);
  }
  const float inv = ctx > 0 ? 1.0f / den : 0.f;           // an empty context: zero rows
  float* dst = p.out + (static_cast<long long>(seq) * p.hq + static_cast<long long>(kvh) * G + w) * kD;
  const int e = 2 * lane;                                  // place 8 g + k in the hand-over
  dst[out_dim<F>(e >> 3, (e & 7) >> 1, 0)] = sum.x * inv;
  dst[out_dim<F>(e >> 3, (e & 7) >> 1, 1)] = sum.y * inv;
}

// --------------------------------------------------------------------- merge

constexpr int kMergeWarps = 16;
constexpr int kMergeBatch = 8;

// Entry blockIdx.x of the list of split sequences: the sequence's record in
// its first CTA, and the first record of every CTA up to its last.  `parts`
// warps a head take a share of them each, 8 records' loads in flight:
//   out = sum_r 2^(m_r - M) acc_r / sum_r 2^(m_r - M) l_r,  M = max m_r.
// 64 registers: two full CTAs an SM, so a batch of many short merges is
// resident at once.
__global__ void __launch_bounds__(kMergeWarps * 32, 2)
    window_merge_kernel(float* out, const float* ws_m, const float* ws_l, const float* ws_acc,
                        const int4* ws_split, const long long* ws_total, int hq, int ctas,
                        int parts) {
  __shared__ float pm[kMergeWarps], pl[kMergeWarps], po[kMergeWarps][kD];
  grid_dependents_launch();        // the next kernel waits for this one's memory itself
  grid_dependency_wait();
  const int4 sp = ws_split[blockIdx.x];
  if (sp.x < 0) return;
  const long long total = *ws_total;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int heads = static_cast<int>(blockDim.x) / (32 * parts);
  const int hw = warp / parts, part = warp - hw * parts;
  const int h = blockIdx.y * heads + hw;
  const bool live = h < hq;
  const int c0 = sp.z, n = sp.w - c0 + 1;
  const bool dense = total >= ctas;         // every CTA holds chunks
  const int few = static_cast<int>(total);  // used when total < ctas
  float mx = -INFINITY, den = 0.f, o0 = 0.f, o1 = 0.f;
  for (int k0 = part * kMergeBatch; live && k0 < n; k0 += parts * kMergeBatch) {
    float mv[kMergeBatch], lv[kMergeBatch], a0[kMergeBatch], a1[kMergeBatch];
    float mb = mx;
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) {
      const int k = k0 + u, c = c0 + k;
      // a CTA whose range is empty (fewer chunks than CTAs) wrote no record
      const bool has = k < n && (k == 0 || dense || few * c / ctas < few * (c + 1) / ctas);
      mv[u] = -INFINITY;
      lv[u] = a0[u] = a1[u] = 0.f;
      if (has) {
        const long long row = static_cast<long long>(k == 0 ? sp.y : 2 * c) * hq + h;
        mv[u] = ws_m[row];
        lv[u] = ws_l[row];
        a0[u] = ws_acc[row * kD + lane];
        a1[u] = ws_acc[row * kD + lane + 32];
      }
      mb = fmaxf(mb, mv[u]);
    }
    const float f = weight_of(mx, mb);             // nothing summed yet: all zero
    den *= f;
    o0 *= f;
    o1 *= f;
    mx = mb;
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) {
      const float w = weight_of(mv[u], mx);        // no record: all zero
      den = fmaf(w, lv[u], den);
      o0 = fmaf(w, a0[u], o0);
      o1 = fmaf(w, a1[u], o1);
    }
  }
  if (parts > 1) {
    if (lane == 0) {
      pm[warp] = mx;
      pl[warp] = den;
    }
    po[warp][lane] = o0;
    po[warp][lane + 32] = o1;
    __syncthreads();
    if (part != 0) return;
    mx = -INFINITY;
    for (int i = 0; i < parts; ++i) mx = fmaxf(mx, pm[warp + i]);
    den = o0 = o1 = 0.f;
    for (int i = 0; i < parts; ++i) {
      const float w = weight_of(pm[warp + i], mx);
      den = fmaf(w, pl[warp + i], den);
      o0 = fmaf(w, po[warp + i][lane], o0);
      o1 = fmaf(w, po[warp + i][lane + 32], o1);
    }
  }
  if (!live) return;
  const float inv = 1.0f / den;
  float* dst = out + (static_cast<long long>(sp.x) * hq + h) * kD;
  dst[lane] = o0 * inv;
  dst[lane + 32] = o1 * inv;
}

// --------------------------------------------------------------------- host

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult q;
    void* f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// The bf16 cache as [Hkv][NB * bs tokens][64]: one box is a 16-token chunk of
// the CTA's heads, in shared memory head after head, 16 swizzled rows each.
bool cache_map(CUtensorMap* m, const void* base, int hkv, long long tokens, int hpc) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kD), static_cast<cuuint64_t>(tokens),
                              static_cast<cuuint64_t>(hkv)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(hkv) * kD * 2, kD * 2};
  const cuuint32_t box[3] = {kD, kChunk, static_cast<cuuint32_t>(hpc)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Shared memory of a CTA of window_direct_kernel: its chunks and the hand-overs.
long long direct_smem(bool four, long long chunks, int group) {
  const long long per_warp = (chunks + kDirectWarps - 1) / kDirectWarps;
  return 1024 + kDirectWarps * (per_warp * (four ? kRecBytes : 2 * kBf16Tile) + group * kCombPitch * 4);
}

template <int F, bool kLoCols>
cudaError_t launch_direct(const CUtensorMap& tk, const CUtensorMap& tv, const Params& p, int chunks,
                          cudaStream_t stream) {
  auto kern = window_direct_kernel<F, kLoCols>;
  static PerDeviceOnce once;
  cudaError_t e = once.run([&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kDirectSmem);
  });
  if (e != cudaSuccess) return e;
  const int per_warp = (chunks + kDirectWarps - 1) / kDirectWarps;
  const uint32_t smem = static_cast<uint32_t>(direct_smem(F == k4Bit, chunks, p.group));
  return launch_pdl(kern, dim3(p.num_seqs, 1, p.hkv), dim3(kDirectWarps * 32), smem, stream, tk, tv,
                    p, per_warp);
}

template <int F, bool kLoCols, int W>
cudaError_t launch_t(const CUtensorMap& tk, const CUtensorMap& tv, const Params& p, dim3 grid,
                     uint32_t smem, cudaStream_t stream) {
  auto kern = window_decode_kernel<F, kLoCols, W>;
  static PerDeviceOnce once;
  cudaError_t e = once.run([&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, grid, dim3((p.hpc * p.wph + p.producers) * 32), smem, stream, tk, tv, p);
}

// KV heads one CTA owns: the largest divisor up to `most`.
int heads_per_cta(int num_kv_heads, int most) {
  int h = most;
  while (num_kv_heads % h != 0) --h;
  return h;
}

// The CTA's shape for a format and group size.
template <int F, bool kLoCols>
void shape(Params& p) {
  p.hpc = heads_per_cta(p.hkv, max_heads<F, kLoCols>());
  p.wph = max_warps<F, kLoCols>() / p.hpc;
  p.producers = p.wph < kMaxProducers ? p.wph : kMaxProducers;
  // bf16 takes a stage's chunks one by one: as many as make 64 KB of it, fewer
  // where a ring would hold but one such stage (8 sequences, window 16384: 84.9
  // us, 87.3 with 32 KB)
  const int nc = F == k4Bit ? chunks_per_stage<F, kLoCols>() : p.hpc > 4 ? 2 : 4;
  p.cps_log2 = nc == 4 ? 2 : nc == 2 ? 1 : 0;
}

}  // namespace

int window_max_ctas(int num_kv_heads, int sms) {
  const int c = sms / (num_kv_heads / heads_per_cta(num_kv_heads, 8));
  return c < 1 ? 1 : c;
}

// m and l [2 ctas, hq], acc [2 ctas, hq, D], split [ctas], total: each part on
// a 256-byte boundary
size_t window_workspace_bytes(int ctas, int num_q_heads) {
  const size_t rows = 2 * static_cast<size_t>(ctas) * num_q_heads;
  const size_t a = (rows * 4 + 255) / 256 * 256;
  return 2 * a + rows * kD * 4 + (static_cast<size_t>(ctas) * 16 + 255) / 256 * 256 + 256;
}

cudaError_t launch_window_decode(const WindowDecodeArgs& a, cudaStream_t stream) {
  if (a.num_seqs == 0) return cudaSuccess;
  const bool four = a.kv4 != nullptr;
  Params p;
  p.out = a.out;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.kv4 = static_cast<const uint8_t*>(a.kv4);
  p.block_tables = a.block_tables;
  p.context_lens = a.context_lens;
  p.num_seqs = a.num_seqs;
  p.hq = a.num_q_heads;
  p.hkv = a.num_kv_heads;
  p.group = a.num_q_heads / a.num_kv_heads;
  p.num_blocks = a.num_blocks;
  p.max_blocks = a.max_blocks_per_seq;
  p.cpb_log2 = 0;
  while ((kChunk << p.cpb_log2) < a.block_size) ++p.cpb_log2;
  p.window = a.window;
  p.sinks = a.window > 0 ? a.sinks : 0;
  p.scale_log2 = a.scale * kLog2e;
  p.status = a.status;
  const bool lo_cols = p.group <= 4;
  const long long tokens = static_cast<long long>(a.num_blocks) * a.block_size;
  CUtensorMap tk = {}, tv = {};
  auto maps = [&](int heads) {
    return four || (cache_map(&tk, a.k_cache, a.num_kv_heads, tokens, heads) &&
                    cache_map(&tv, a.v_cache, a.num_kv_heads, tokens, heads));
  };
  // The chunks a sequence can have: the block table's capacity, or the window's
  // and the sinks' with their edges.
  const long long capacity = static_cast<long long>(a.max_blocks_per_seq) << p.cpb_log2;
  const long long seen = p.window > 0 ? p.window / kChunk + 2LL + (p.sinks + kChunk - 1LL) / kChunk : capacity;
  const long long chunks = seen < capacity ? seen : capacity;
  if (static_cast<long long>(a.num_seqs) * p.hkv <= a.sms &&
      chunks <= (four ? kDirectChunks4 : kDirectChunks16) &&
      direct_smem(four, chunks, p.group) <= kDirectSmem) {
    if (!maps(1)) return cudaErrorInvalidValue;
    const int n = static_cast<int>(chunks);
    if (!four)
      return lo_cols ? launch_direct<kBf16, true>(tk, tv, p, n, stream)
                     : launch_direct<kBf16, false>(tk, tv, p, n, stream);
    return lo_cols ? launch_direct<k4Bit, true>(tk, tv, p, n, stream)
                   : launch_direct<k4Bit, false>(tk, tv, p, n, stream);
  }
  if (!four)
    lo_cols ? shape<kBf16, true>(p) : shape<kBf16, false>(p);
  else
    lo_cols ? shape<k4Bit, true>(p) : shape<k4Bit, false>(p);
  const int groups = p.hkv / p.hpc;
  p.ctas = a.sms / groups < 1 ? 1 : a.sms / groups;
  for (;; --p.cps_log2) {              // two stages a ring at least (bf16: by smaller stages)
    p.kv_bytes = (p.hpc << p.cps_log2) * (four ? kRecBytes : 2 * kBf16Tile);
    p.stage_bytes = align_up(p.kv_bytes + p.hpc * p.group * kD * 2, 1024);
    const uint32_t fixed = make_layout(0, p.stage_bytes, p.hpc, p.wph, p.group).total + 1024 + 16;
    const int most = static_cast<int>((kSmemLimit - fixed) / (p.stage_bytes + sizeof(StageMeta) + 16));
    p.ring = (most > 48 ? 48 : most) / p.wph;
    if (p.ring >= 2 || four || p.cps_log2 == 0) break;
  }
  p.stages = p.ring * p.wph;
  if (p.ring < 1) return cudaErrorInvalidConfiguration;
  p.seg_weight = four ? kSegWeight4 : kSegWeight16;
  const long long longest = capacity + p.seg_weight;
  p.small = a.num_seqs <= (p.hpc * p.wph + p.producers) * 32 && longest * a.num_seqs * (p.ctas + 1) < (1LL << 31);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const size_t rows = 2 * static_cast<size_t>(p.ctas) * a.num_q_heads;
  const size_t ab = (rows * 4 + 255) / 256 * 256;
  p.ws_m = reinterpret_cast<float*>(ws);
  p.ws_l = reinterpret_cast<float*>(ws + ab);
  p.ws_acc = reinterpret_cast<float*>(ws + 2 * ab);
  p.ws_split = reinterpret_cast<int4*>(ws + 2 * ab + rows * kD * 4);
  p.ws_total = reinterpret_cast<long long*>(ws + 2 * ab + rows * kD * 4 +
                                            (static_cast<size_t>(p.ctas) * 16 + 255) / 256 * 256);
  if (!maps(p.hpc)) return cudaErrorInvalidValue;
  const uint32_t smem = make_layout(p.stages, p.stage_bytes, p.hpc, p.wph, p.group).total + 1024;
  const dim3 grid(p.ctas, 1, groups);
  cudaError_t e;
  const bool wide = p.hpc == 4;         // a constant stride between a head's chunks
  if (!four)
    e = lo_cols ? launch_t<kBf16, true, 0>(tk, tv, p, grid, smem, stream)
                : launch_t<kBf16, false, 0>(tk, tv, p, grid, smem, stream);
  else if (lo_cols)
    e = wide ? launch_t<k4Bit, true, 4>(tk, tv, p, grid, smem, stream)
             : launch_t<k4Bit, true, 0>(tk, tv, p, grid, smem, stream);
  else
    e = wide ? launch_t<k4Bit, false, 4>(tk, tv, p, grid, smem, stream)
             : launch_t<k4Bit, false, 0>(tk, tv, p, grid, smem, stream);
  if (e != cudaSuccess) return e;
  // a sequence has about 1 + ctas / num_seqs records: one warp a head and
  // batch of 8, up to 16
  int parts = 1;
  while (parts < kMergeWarps && static_cast<long long>(parts) * kMergeBatch * a.num_seqs < p.ctas) parts *= 2;
  const int heads = parts < 4 ? 4 : kMergeWarps / parts;
  return launch_pdl(window_merge_kernel,
                    dim3(a.num_seqs < p.ctas ? a.num_seqs : p.ctas,
                         (a.num_q_heads + heads - 1) / heads),
                    dim3(heads * parts * 32), 0, stream, a.out, p.ws_m, p.ws_l, p.ws_acc,
                    p.ws_split, p.ws_total, a.num_q_heads, p.ctas, parts);
}

}  // namespace tvl
