// diff_decode.cu -- differential attention of one query token a sequence over the
// bf16 paged cache, with an optional sliding window and sinks.
//
// What it computes: query heads 2 i and 2 i + 1 are the two maps of pair i, KV heads
// 2 j and 2 j + 1 their keys (pair i reads pair j = i / G), V is the two V heads side
// by side, 128 wide.  Over the visible tokens
//   d = softmax(scale q_{2i} K_{2j}) V - lambda softmax(scale q_{2i+1} K_{2j+1}) V,
//   out = out_scale * w * d / sqrt(mean d^2 + eps)   (without w: out_scale * d).
//
// Bound: every visible K/V byte is read once, HBM bandwidth.  An SM is handed a
// 16-token chunk of a pair (8 KB) every 350 cycles (6.8 TB/s, 152 SMs, 1.9 GHz).  Both
// products run on mma.sync m16n8k16, tokens (Q K^T) or dimensions (P V) as the 16 rows,
// as a single token's few heads would leave a tcgen05 tile of 128 rows nearly empty.
//
// Columns.  A warp's eight columns are four query pairs: columns 0..3 their first
// map, 4..7 their second.  Each key's product has the other map's columns zero, so
// both land in one accumulator and one pass of the softmax arithmetic serves both
// maps; and P V, whose value is common to the maps, uses all eight columns.  More
// than four query pairs a KV pair take a second warp ("column group") on the same
// stage.
//
// P in two bf16 parts, 16 bits, where the output keeps 8: the difference d of the maps
// is off by 2^-16 (|o1| + lambda |o2|).  The tensor cores truncate what they add, so
// sums across chunks are added in fp32 beside them.
//
// Work split: line.cuh's.  A CTA's consumer warps are units (pair, column group)
// times `wph` rings; the warps of a unit combine at a segment's end through shared
// memory.  All waits are bounded.
//
// Measured, 32/8 heads: 8 sequences of 32k-128k tokens 189-191 us (1299 MB: HBM, 1.00 to
// 1.01 of the copy's rate); 64 of 0.5-4k 54.3 us (301 MB, 0.82: the fixed 9 us of schedule,
// first data and merge); one KV pair a CTA 61.9, two 57.2, one ring for all 56.2.  One
// sequence of 777 tokens, 8/2 heads: 5.4 us (diff_direct_kernel).
#include "diff.cuh"
#include "line.cuh"

namespace tvl {
namespace {

constexpr int kWarps = 8;                     // consumers a CTA, at most
constexpr int kThreads = (kWarps + kMaxProducers) * 32;
constexpr int kPairsPerCta = 4;
constexpr int kCols = 8;
constexpr float kMaxSum = 256.0f;             // a lane's weights under the reference maximum
// Cost of a sequence start, in chunks (64 sequences of 0.5-4k tokens: 56.6 us at 1, 54.9
// at 3, 54.4 at 6, 54.3 at 10).
constexpr int kSegWeight = 8;
constexpr int kCombPitch = kDV + 4;           // floats a column of a warp hands over: 128, m, l

struct DiffParams : Params {
  __nv_bfloat16* dout;                        // [S, pairs, kDV]
  DiffTail tail;
  int pairs;                                  // query pairs
  int cgs, units;                             // column groups a KV pair; units of a CTA
};

// A lane (g = lane / 4, t = lane % 4) holds columns 2 t and 2 t + 1: `x`, `y`.
struct State {
  uint32_t qa[4][2], qb[4][2];   // q as the column operand of the first and the second key
  float acc[8][4];               // [i][0..1]: dimension 16 i + g, [i][2..3]: 16 i + 8 + g
  float2 m, l;                   // reference maximum (log2), sum of p
};

// Query pair of column n (n & 3 of the column group), within the KV pair's G.
__device__ __forceinline__ int pair_of_column(int cg, int n) { return 4 * cg + (n & 3); }

// qbase: the KV pair's 2 G query heads
__device__ __forceinline__ void start(State& st, const DiffParams& p, const uint8_t* qbase, int cg) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int h = pair_of_column(cg, g), map = g >> 2;
  const bool live = h < p.group;
  const uint32_t* q = reinterpret_cast<const uint32_t*>(qbase + (live ? 2 * h + map : 0) * (kD * 2));
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t w = live ? q[8 * i + t + 4 * k] : 0u;
      st.qa[i][k] = map == 0 ? w : 0u;
      st.qb[i][k] = map == 0 ? 0u : w;
    }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) st.acc[i][k] = 0.f;
  st.m = make_float2(-INFINITY, -INFINITY);
  st.l = make_float2(0.f, 0.f);
}

// Moves the reference maximum to cover mx (this lane's largest scores, log2), and
// rescales what is summed so far; never down.
__device__ __forceinline__ void move_reference(State& st, float2 mx) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    mx.x = fmaxf(mx.x, __shfl_xor_sync(kFull, mx.x, o));
    mx.y = fmaxf(mx.y, __shfl_xor_sync(kFull, mx.y, o));
  }
  mx = max2(mx, st.m);
  const float2 f = make_float2(ex2(st.m.x - mx.x), ex2(st.m.y - mx.y));
  st.m = mx;
  st.l = __fmul2_rn(st.l, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    st.acc[i][0] *= f.x;
    st.acc[i][1] *= f.y;
    st.acc[i][2] *= f.x;
    st.acc[i][3] *= f.y;
  }
}

// One chunk of a pair: `chunk` is the first key's tile, the second's follows; the V
// tiles lie v_off behind.
template <bool kMasked>
__device__ __forceinline__ void process(State& st, const DiffParams& p, const uint8_t* chunk,
                                        uint32_t v_off, int tok0, int ctx) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int first = p.window > 0 && ctx > p.window ? ctx - p.window : 0;
  auto seen = [&](int tok) { return tok < ctx && (tok >= first || tok < p.sinks); };
  // --- scores: x[0] row g, x[1] row g + 8
  float2 x[2];
  {
    float c[4];
    const uint32_t base = smem_addr(chunk);
    const int row = lane & 15;                        // matrices 1 and 3: rows 8..15
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t at = base + row * 128 + (((2 * i + (lane >> 4)) ^ (row & 7)) << 4);
      uint32_t a[4], b[4];
      ldsm4(a, at);
      ldsm4(b, at + kBf16Tile);
      // four sums of 16 products (the other key adds zeros), added with rounding
      float d[4];
      mma_bf16_0(i == 0 ? c : d, a[0], a[1], a[2], a[3], st.qa[i][0], st.qa[i][1]);
      mma_bf16(i == 0 ? c : d, b[0], b[1], b[2], b[3], st.qb[i][0], st.qb[i][1]);
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
    move_reference(st, max2(x[0], x[1]));
    weights();
  }
  st.l = __fadd2_rn(st.l, sum);
  // --- weights as the column operand of P V, in two parts
  uint32_t hi[2], lo[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const uint32_t h = pack16<kBf16>(w[r]);
    const float2 back = unpack16<kBf16>(h);
    hi[r] = transpose8(h);
    lo[r] = transpose8(pack16<kBf16>(make_float2(w[r].x - back.x, w[r].y - back.y)));
  }
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
  for (int i = 0; i < 8; ++i) {
    uint32_t a[4];
    float o[4];
    ldsm4_t(a, base + (i >> 2) * kBf16Tile + tok * 128 +
                   (((2 * (i & 3) + ((lane >> 3) & 1)) ^ (tok & 7)) << 4));
    if (kMasked) {
      a[0] &= keep[0];
      a[1] &= keep[0];
      a[2] &= keep[1];
      a[3] &= keep[1];
    }
    mma_bf16_0(o, a[0], a[1], a[2], a[3], hi[0], hi[1]);
    mma_bf16(o, a[0], a[1], a[2], a[3], lo[0], lo[1]);
    add_to(st.acc[i], o);
  }
}

// Ends a warp's part of a segment.  A unit's warp 0, which has the segment's first
// stage, combines: the others with stages of it hand (m, l, o) over to it through
// shared memory, and it stores the output or the record.  handed: warp 0: bit i, the
// phase of warp i's next hand-over; else the hand-overs so far.  False: a bounded
// wait ran out.
__device__ bool finish(State& st, const DiffParams& p, uint8_t* smem, const Layout& L, int unit, int w,
                       int& handed, int flags, int seq, int record) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint64_t* cfull = reinterpret_cast<uint64_t*>(smem + L.bars) + 2 * p.stages;
  uint64_t* cempty = cfull + p.units * p.wph;
  float* comb = reinterpret_cast<float*>(smem + L.comb);
#pragma unroll
  for (int x = 4; x < 32; x <<= 1) {
    st.l.x += __shfl_xor_sync(kFull, st.l.x, x);
    st.l.y += __shfl_xor_sync(kFull, st.l.y, x);
  }
  float m[2] = {st.m.x, st.m.y}, l[2] = {st.l.x, st.l.y};
  const int pr = unit / p.cgs, cg = unit - pr * p.cgs;
  // a hand-over: column by column, 16 floats a lane g (dimensions 16 i + g, 16 i + 8 + g)
  if (w > 0) {
    const int me = w * p.units + unit;
    if (handed > 0 && !mbar_wait(&cempty[me], (handed - 1) & 1)) return false;
    ++handed;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float* dst = comb + (((w - 1) * p.units + unit) * kCols + 2 * t + j) * kCombPitch;
#pragma unroll
      for (int i = 0; i < 8; i += 2)
        reinterpret_cast<float4*>(dst)[(i >> 1) * 8 + g] =
            make_float4(st.acc[i][j], st.acc[i][2 + j], st.acc[i + 1][j], st.acc[i + 1][2 + j]);
      if (g == 0) *reinterpret_cast<float2*>(dst + kDV) = make_float2(m[j], l[j]);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&cfull[me]);
    return true;
  }
  const int parts = flags >> kPartsShift;
  for (int i = 1; i < parts; ++i) {
    const int from = i * p.units + unit;
    if (!mbar_wait(&cfull[from], handed >> i & 1)) return false;
    handed ^= 1 << i;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float* src = comb + (((i - 1) * p.units + unit) * kCols + 2 * t + j) * kCombPitch;
      const float2 ml = *reinterpret_cast<const float2*>(src + kDV);
      const float mn = fmaxf(m[j], ml.x);
      const float fa = weight_of(m[j], mn), fb = weight_of(ml.x, mn);
      m[j] = mn;
      l[j] = l[j] * fa + ml.y * fb;
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float4 v = reinterpret_cast<const float4*>(src)[(k >> 1) * 8 + g];
        st.acc[k][j] = st.acc[k][j] * fa + v.x * fb;
        st.acc[k][2 + j] = st.acc[k][2 + j] * fa + v.y * fb;
        st.acc[k + 1][j] = st.acc[k + 1][j] * fa + v.z * fb;
        st.acc[k + 1][2 + j] = st.acc[k + 1][2 + j] * fa + v.w * fb;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&cempty[from]);
  }
  const int kvp = blockIdx.z * (p.hpc / 2) + pr;
  const int map = t >> 1;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int h = pair_of_column(cg, 2 * t + j);
    const bool live = h < p.group;
    const long long pair = static_cast<long long>(kvp) * p.group + h;
    if (record >= 0) {
      if (!live) continue;
      const long long row = static_cast<long long>(record) * p.hq + 2 * pair + map;
      float* dst = p.ws_acc + row * kDV;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dst[16 * i + g] = st.acc[i][j];
        dst[16 * i + 8 + g] = st.acc[i][2 + j];
      }
      if (g == 0) {
        p.ws_m[row] = m[j];
        p.ws_l[row] = l[j];
      }
      continue;
    }
    // the pair's second map is in lane t ^ 2
    const float lam = live ? p.tail.lam[seq * p.tail.lam_stride + pair] : 0.f;
    const float f = (map == 0 ? 1.f : -lam) / l[j];
    float d[16], ss = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float o = __fmul_rn(st.acc[i >> 1][2 * (i & 1) + j], f);   // equal maps cancel exactly
      d[i] = o + __shfl_xor_sync(kFull, o, 2);
      ss = fmaf(d[i], d[i], ss);
    }
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) ss += __shfl_xor_sync(kFull, ss, x);
    const float sc = diff_factor(p.tail, ss);
    if (!live) continue;
    __nv_bfloat16* dst = p.dout + (static_cast<long long>(seq) * p.pairs + pair) * kDV;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if ((i >> 3) != map) continue;             // each of the two lanes stores half
      const int dim = 8 * i + g;
      const float wt = p.tail.weight != nullptr ? __bfloat162float(p.tail.weight[dim]) : 1.f;
      dst[dim] = __float2bfloat16_rn(d[i] * sc * wt);
    }
  }
  return true;
}

__device__ void consumer(const DiffParams& p, uint8_t* smem, const Layout& L) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int unit = warp % p.units, w = warp / p.units;
  const int pr = unit / p.cgs, cg = unit - pr * p.cgs;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L.bars);
  uint64_t* empty = full + p.stages;
  const StageMeta* meta = reinterpret_cast<const StageMeta*>(smem + L.meta);
  const uint32_t mine = 2 * pr * kBf16Tile;     // the pair's first chunk in a stage
  const uint32_t step = p.hpc * kBf16Tile;      // to its next
  const uint32_t v_off = p.kv_bytes / 2;
  State st;
  int handed = 0;
  const int ring0 = w * p.ring;                 // the warp's ring
  int stage = ring0;
  uint32_t ph = 0;
  for (;;) {
    if (!mbar_wait(&full[stage], ph)) {
      if (lane == 0) report(p.status, kDevTimeout);
      return;
    }
    const StageMeta& md = meta[stage];
    const int flags = md.flags;
    if (flags & kTerminate) return;
    const uint8_t* at = smem + static_cast<size_t>(stage) * p.stage_bytes + mine;
    if (flags & kSegFirst) start(st, p, at - mine + p.kv_bytes + 2 * pr * p.group * (kD * 2), cg);
    if (flags & kPartial) {
      // a segment's end, or a stage with slots that are not visible
      const int n = md.n, ctx = md.ctx, v0 = md.v0, ns = md.ns, delta = md.delta;
#pragma unroll 1
      for (int i = 0; i < n; ++i)
        process<true>(st, p, at + i * step, v_off, (v0 + i < ns ? v0 + i : v0 + i + delta) * kChunk, ctx);
    } else {
#pragma unroll 1
      for (int i = 0; i < 1 << p.cps_log2; ++i) process<false>(st, p, at + i * step, v_off, 0, 0);
    }
    const int seq = md.seq, record = md.record;
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[stage]);
    if (flags & kSegLast) {
      if (!finish(st, p, smem, L, unit, w, handed, flags, seq, record)) {
        if (lane == 0) report(p.status, kDevTimeout);
        return;
      }
    }
    if (++stage == ring0 + p.ring) {
      stage = ring0;
      ph ^= 1;
    }
  }
}

__host__ __device__ inline Layout diff_layout(const DiffParams& p, int stages) {
  return make_layout(stages, p.stage_bytes, p.units * p.wph, (p.wph - 1) * p.units * kCols * kCombPitch * 4);
}

__global__ void __launch_bounds__(kThreads, 1)
    diff_decode_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const DiffParams p) {
  extern __shared__ uint8_t smem_raw[];
  // 128-byte-swizzled tiles repeat every 1024 bytes
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const Layout L = diff_layout(p, p.stages);
  Schedule* sched = reinterpret_cast<Schedule*>(smem + L.sched);
  long long* tmp = reinterpret_cast<long long*>(smem + L.sched + 64);
  int* lens = reinterpret_cast<int*>(smem + L.sched + 64 + 32 * 8);
  const int tid = threadIdx.x, warp = tid >> 5;
  const int consumers = p.units * p.wph;
  if (tid == 0) {
    uint64_t* b = reinterpret_cast<uint64_t*>(smem + L.bars);
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&b[i], 1);
      mbar_init(&b[p.stages + i], p.units);
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
    producer<kBf16>(p, sc, smem, L, warp - consumers, &tm_k, &tm_v);
  } else {
    // empty contexts have no chunk and so no segment: zero rows, dealt out
    const int n = p.hpc / 2 * p.group * kDV;
    for (int s = blockIdx.x; s < p.num_seqs; s += p.ctas) {
      if (p.context_lens[s] > 0) continue;
      if (tid == 0 && blockIdx.z == 0 && p.num_seqs <= p.ctas) p.ws_split[s] = make_int4(-1, 0, 0, 0);
      __nv_bfloat16* dst = p.dout + static_cast<long long>(s) * p.pairs * kDV + static_cast<long long>(blockIdx.z) * n;
      for (int i = tid; i < n; i += consumers * 32) dst[i] = __float2bfloat16_rn(0.f);
    }
    consumer(p, smem, L);
  }
}

// -------------------------------------------------------------------- direct

// Small batches of bounded length: a cluster of kSpread CTAs does KV pair z of a
// sequence alone, in one launch.  Chunk i goes to CTA i mod kSpread, and there to warp
// i / kSpread mod 8: the warp fetches its chunks' block ids, issues their copies (all of
// them fit) and q's loads, and waits once.  A CTA adds its warps up; then CTA r takes
// the group's query pairs r, r + kSpread, ...: it reads the CTAs' sums through
// distributed shared memory.  Bound by latency (five dependent memory round trips and two
// cluster barriers): 777 tokens, 8 query heads, 5.4 us, 10.8 through the schedule and the
// merge; 2040 tokens, 3 sequences of 4 KV pairs, 6.9 and 10.7.  It wins while all clusters
// run at once (14 of them 5.8 and 10.4, 16, two waves, 10.3 and 10.5).
constexpr int kSpread = 8;
constexpr int kDirectMost = 2;                // chunks a warp: what shared memory holds

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The float at `addr` of this CTA's shared memory, in CTA `rank` of the cluster.
__device__ __forceinline__ float cluster_load(const float* addr, int rank) {
  uint32_t at;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(addr)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

constexpr uint32_t kPairChunk = 4 * kBf16Tile;        // K_0, K_1, V_0, V_1

__host__ __device__ inline uint32_t direct_smem(int per_warp, int cgs) {
  return 1024 + kWarps * per_warp * kPairChunk + (kWarps + 1) * cgs * kCols * kCombPitch * 4;
}

__global__ void __launch_bounds__(kWarps * 32, 1) __cluster_dims__(kSpread, 1, 1)
    diff_direct_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const DiffParams p, int per_warp) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[kWarps];
  __shared__ float norm[kWarps];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, t = lane & 3;
  const int rank = blockIdx.x % kSpread, seq = blockIdx.x / kSpread, kvp = blockIdx.z;
  uint8_t* mine = smem + w * per_warp * kPairChunk;
  // [warp][column group][column], then the CTA's own sums
  float* comb = reinterpret_cast<float*>(smem + kWarps * per_warp * kPairChunk);
  const int cols = p.cgs * kCols;
  float* sums = comb + kWarps * cols * kCombPitch;
  if (lane == 0) {
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
    mbar_init(&bars[w], 1);
    fence_barrier_init();
  }
  __syncwarp();
  grid_dependency_wait();
  grid_dependents_launch();
  const int ctx = load_ctx(p, seq);
  const Visible vis = visible_of(p, ctx);
  auto chunk_of = [&](int i) {               // the warp's i-th chunk as a token chunk
    const int v = rank + kSpread * (w + kWarps * i);
    return v < vis.ns ? v : v + vis.delta;
  };
  const int at = rank + kSpread * w, n = at < vis.n ? (vis.n - 1 - at) / (kSpread * kWarps) + 1 : 0;   // <= per_warp
  if (n > 0) {
    int page = 0;
    if (lane < n) page = p.block_tables[static_cast<long long>(seq) * p.max_blocks + (chunk_of(lane) >> p.cpb_log2)];
    if (lane == 0) mbar_arrive_expect_tx(&bars[w], n * kPairChunk);
    __syncwarp();
    if (lane < n) {
      if (page < 0 || page >= p.num_blocks) {
        report(p.status, TVL_DEV_BAD_BLOCK_ID);
        page = 0;
      }
      const long long chunk = (static_cast<long long>(page) << p.cpb_log2) +
                              (chunk_of(lane) & ((1 << p.cpb_log2) - 1));
      const int tok = static_cast<int>(chunk * kChunk);
      tma_load_3d(mine + lane * kPairChunk, &tm_k, 0, tok, 2 * kvp, &bars[w]);
      tma_load_3d(mine + lane * kPairChunk + 2 * kBf16Tile, &tm_v, 0, tok, 2 * kvp, &bars[w]);
    }
  }
  const uint8_t* q = reinterpret_cast<const uint8_t*>(
      p.q + (static_cast<size_t>(seq) * p.hq + 2 * static_cast<size_t>(kvp) * p.group) * kD);
  for (int cg = 0; cg < p.cgs; ++cg) {
    State st;
    start(st, p, q, cg);
    if (cg == 0 && n > 0 && !mbar_wait(&bars[w], 0) && lane == 0) report(p.status, kDevTimeout);
#pragma unroll 1
    for (int i = 0; i < n; ++i)
      process<true>(st, p, mine + i * kPairChunk, 2 * kBf16Tile, chunk_of(i) * kChunk, ctx);
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      st.l.x += __shfl_xor_sync(kFull, st.l.x, x);
      st.l.y += __shfl_xor_sync(kFull, st.l.y, x);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float* dst = comb + ((w * p.cgs + cg) * kCols + 2 * t + j) * kCombPitch;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dst[16 * i + g] = st.acc[i][j];
        dst[16 * i + 8 + g] = st.acc[i][2 + j];
      }
      if (g == 0) *reinterpret_cast<float2*>(dst + kDV) = j == 0 ? make_float2(st.m.x, st.l.x) : make_float2(st.m.y, st.l.y);
    }
  }
  __syncthreads();
  // the CTA's sums: a warp a column, four dimensions a lane
  for (int c = w; c < cols; c += kWarps) {
    float top = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kWarps; ++i) top = fmaxf(top, comb[(i * cols + c) * kCombPitch + kDV]);
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const float* src = comb + (i * cols + c) * kCombPitch;
      const float f = weight_of(src[kDV], top);        // (a warp without chunks: l and o are 0)
      const float4 v = reinterpret_cast<const float4*>(src)[lane];
      l = fmaf(f, src[kDV + 1], l);
      o = make_float4(fmaf(f, v.x, o.x), fmaf(f, v.y, o.y), fmaf(f, v.z, o.z), fmaf(f, v.w, o.w));
    }
    float* dst = sums + c * kCombPitch;
    reinterpret_cast<float4*>(dst)[lane] = o;
    if (lane == 0) *reinterpret_cast<float2*>(dst + kDV) = make_float2(top, l);
  }
  cluster_sync();
  // query pair h: its maps are columns h and h + 4 of its column group; 128 threads, a
  // dimension each (the other half of the CTA only takes part in the barriers)
  for (int h = rank; h < p.group; h += kSpread) {
    float d = 0.f;
    if (tid < kDV) {
      float o[2], l[2];
#pragma unroll
      for (int map = 0; map < 2; ++map) {
        const float* src = sums + ((h >> 2) * kCols + 4 * map + (h & 3)) * kCombPitch;
        float mv[kSpread], lv[kSpread], ov[kSpread], top = -INFINITY;
#pragma unroll
        for (int r = 0; r < kSpread; ++r) {
          mv[r] = cluster_load(src + kDV, r);
          lv[r] = cluster_load(src + kDV + 1, r);
          ov[r] = cluster_load(src + tid, r);
        }
#pragma unroll
        for (int r = 0; r < kSpread; ++r) top = fmaxf(top, mv[r]);
        o[map] = l[map] = 0.f;
#pragma unroll
        for (int r = 0; r < kSpread; ++r) {
          const float f = weight_of(mv[r], top);
          l[map] = fmaf(f, lv[r], l[map]);
          o[map] = fmaf(f, ov[r], o[map]);
        }
      }
      const long long pair = static_cast<long long>(kvp) * p.group + h;
      const float lam = p.tail.lam[seq * p.tail.lam_stride + pair];
      if (ctx > 0) d = __fmul_rn(o[0], 1.0f / l[0]) - __fmul_rn(o[1], lam / l[1]);
      float ss = d * d;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) ss += __shfl_xor_sync(kFull, ss, x);
      if (lane == 0) norm[w] = ss;
    }
    __syncthreads();
    if (tid < kDV) {
      const float sc = ctx > 0 ? diff_factor(p.tail, (norm[0] + norm[1]) + (norm[2] + norm[3])) : 0.f;
      const float wt = p.tail.weight != nullptr ? __bfloat162float(p.tail.weight[tid]) : 1.f;
      p.dout[(static_cast<long long>(seq) * p.pairs + static_cast<long long>(kvp) * p.group + h) * kDV + tid] =
          __float2bfloat16_rn(d * sc * wt);
    }
    __syncthreads();
  }
  cluster_sync();                // no CTA leaves while others read its sums
}

// --------------------------------------------------------------------- merge

constexpr int kMergeWarps = 16;
constexpr int kMergeBatch = 4;

// One map's partial results of a query pair, four dimensions a lane.
struct Sum {
  float m, l;
  float4 o;
};
__device__ __forceinline__ void rescale(Sum& s, float f) {
  s.l *= f;
  s.o = make_float4(s.o.x * f, s.o.y * f, s.o.z * f, s.o.w * f);
}
__device__ __forceinline__ void add(Sum& s, float f, float l, float4 o) {
  s.l = fmaf(f, l, s.l);
  s.o = make_float4(fmaf(f, o.x, s.o.x), fmaf(f, o.y, s.o.y), fmaf(f, o.z, s.o.z), fmaf(f, o.w, s.o.w));
}

// Entry blockIdx.x of the list of split sequences: the sequence's record in its first
// CTA, and the first record of every CTA up to its last.  `parts` warps a query pair
// take a share of them each, kMergeBatch records' loads in flight; the pair's first
// warp adds them up, takes the difference and the norm, and stores the row.
__global__ void __launch_bounds__(kMergeWarps * 32, 1)
    diff_merge_kernel(const DiffParams p, int parts) {
  __shared__ float2 pml[kMergeWarps][2];
  __shared__ float4 po[kMergeWarps][2][32];
  grid_dependents_launch();        // the next kernel waits for this one's memory itself
  grid_dependency_wait();
  const int4 sp = p.ws_split[blockIdx.x];
  if (sp.x < 0) return;
  const long long total = *p.ws_total;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = static_cast<int>(blockDim.x) / (32 * parts);
  const int pw = warp / parts, part = warp - pw * parts;
  const int pair = blockIdx.y * per + pw;
  const bool live = pair < p.pairs;
  const int c0 = sp.z, n = sp.w - c0 + 1;
  const bool dense = total >= p.ctas;       // every CTA holds chunks
  const int few = static_cast<int>(total);  // used when total < ctas
  Sum s[2];
#pragma unroll
  for (int map = 0; map < 2; ++map) s[map] = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int k0 = part * kMergeBatch; live && k0 < n; k0 += parts * kMergeBatch) {
    float mv[kMergeBatch][2], lv[kMergeBatch][2];
    float4 ov[kMergeBatch][2];
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) {
      const int k = k0 + u, c = c0 + k;
      // a CTA whose range is empty (fewer chunks than CTAs) wrote no record
      const bool has = k < n && (k == 0 || dense || few * c / p.ctas < few * (c + 1) / p.ctas);
#pragma unroll
      for (int map = 0; map < 2; ++map) {
        mv[u][map] = -INFINITY;
        lv[u][map] = 0.f;
        ov[u][map] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (has) {
          const long long row = static_cast<long long>(k == 0 ? sp.y : 2 * c) * p.hq + 2 * pair + map;
          mv[u][map] = p.ws_m[row];
          lv[u][map] = p.ws_l[row];
          ov[u][map] = reinterpret_cast<const float4*>(p.ws_acc + row * kDV)[lane];
        }
      }
    }
#pragma unroll
    for (int map = 0; map < 2; ++map) {
      float mb = s[map].m;
#pragma unroll
      for (int u = 0; u < kMergeBatch; ++u) mb = fmaxf(mb, mv[u][map]);
      rescale(s[map], weight_of(s[map].m, mb));        // nothing summed yet: all zero
      s[map].m = mb;
#pragma unroll
      for (int u = 0; u < kMergeBatch; ++u)            // no record: all zero
        add(s[map], weight_of(mv[u][map], mb), lv[u][map], ov[u][map]);
    }
  }
  if (parts > 1) {
#pragma unroll
    for (int map = 0; map < 2; ++map) {
      if (lane == 0) pml[warp][map] = make_float2(s[map].m, s[map].l);
      po[warp][map][lane] = s[map].o;
    }
    __syncthreads();
    if (part != 0) return;
#pragma unroll
    for (int map = 0; map < 2; ++map) {
      float mb = -INFINITY;
      for (int i = 0; i < parts; ++i) mb = fmaxf(mb, pml[warp + i][map].x);
      s[map] = {mb, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
      for (int i = 0; i < parts; ++i)
        add(s[map], weight_of(pml[warp + i][map].x, mb), pml[warp + i][map].y, po[warp + i][map][lane]);
    }
  }
  if (!live) return;
  const float f0 = 1.0f / s[0].l, f1 = p.tail.lam[sp.x * p.tail.lam_stride + pair] / s[1].l;
  // (the products rounded one by one: equal maps cancel exactly)
  const float d[4] = {__fmul_rn(s[0].o.x, f0) - __fmul_rn(s[1].o.x, f1),
                      __fmul_rn(s[0].o.y, f0) - __fmul_rn(s[1].o.y, f1),
                      __fmul_rn(s[0].o.z, f0) - __fmul_rn(s[1].o.z, f1),
                      __fmul_rn(s[0].o.w, f0) - __fmul_rn(s[1].o.w, f1)};
  float ss = d[0] * d[0] + d[1] * d[1] + d[2] * d[2] + d[3] * d[3];
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) ss += __shfl_xor_sync(kFull, ss, x);
  const float sc = diff_factor(p.tail, ss);
  float2 wa = make_float2(1.f, 1.f), wb = wa;
  if (p.tail.weight != nullptr) {
    const uint2 w = reinterpret_cast<const uint2*>(p.tail.weight)[lane];
    wa = bf16x2_to_float2(w.x);
    wb = bf16x2_to_float2(w.y);
  }
  __nv_bfloat16* dst = p.dout + (static_cast<long long>(sp.x) * p.pairs + pair) * kDV;
  reinterpret_cast<uint2*>(dst)[lane] =
      make_uint2(pack16<kBf16>(make_float2(d[0] * sc * wa.x, d[1] * sc * wa.y)),
                 pack16<kBf16>(make_float2(d[2] * sc * wb.x, d[3] * sc * wb.y)));
}

// --------------------------------------------------------------------- host

// KV pairs that a CTA owns.
int pairs_per_cta(int num_kv_heads) { return heads_per_cta(num_kv_heads / 2, kPairsPerCta); }

// Clusters of diff_direct_kernel that the current device runs at once (0 on an error),
// asked for once per device with the largest shared memory.
int direct_clusters() {
  static std::atomic<int> known[64];                   // 1 + the answer
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n > 0) return n - 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kSpread);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = direct_smem(kDirectMost, 2);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kSpread;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(diff_direct_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kSmemLimit - 1024) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, diff_direct_kernel, &cfg) != cudaSuccess || n < 0) {
    cudaGetLastError();
    return 0;
  }
  known[dev].store(n + 1, std::memory_order_relaxed);
  return n;
}

}  // namespace

// The most CTAs that share one KV-head group's work.
int diff_max_ctas(int num_kv_heads, int sms) {
  const int c = sms / (num_kv_heads / 2 / pairs_per_cta(num_kv_heads));
  return c < 1 ? 1 : c;
}

// m and l [2 ctas, hq], acc [2 ctas, hq, kDV], split [ctas], total: each part on a
// 256-byte boundary
size_t diff_workspace_bytes(int ctas, int num_q_heads) {
  const size_t rows = 2 * static_cast<size_t>(ctas) * num_q_heads;
  const size_t a = (rows * 4 + 255) / 256 * 256;
  return 2 * a + rows * kDV * 4 + (static_cast<size_t>(ctas) * 16 + 255) / 256 * 256 + 256;
}

cudaError_t launch_diff_decode(const DiffDecodeArgs& a, cudaStream_t stream) {
  if (a.num_seqs == 0) return cudaSuccess;
  DiffParams p = {};
  p.dout = static_cast<__nv_bfloat16*>(a.out);
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.block_tables = a.block_tables;
  p.context_lens = a.context_lens;
  p.num_seqs = a.num_seqs;
  p.hq = a.num_q_heads;
  p.hkv = a.num_kv_heads;
  p.group = a.num_q_heads / a.num_kv_heads;
  p.pairs = a.num_q_heads / 2;
  p.num_blocks = a.num_blocks;
  p.max_blocks = a.max_blocks_per_seq;
  while ((kChunk << p.cpb_log2) < a.block_size) ++p.cpb_log2;
  p.window = a.window;
  p.sinks = a.window > 0 ? a.sinks : 0;
  p.scale_log2 = a.scale * kLog2e;
  p.status = a.status;
  p.tail.lam = a.lam;
  p.tail.lam_stride = a.lam_per_token ? p.pairs : 0;
  p.tail.weight = static_cast<const __nv_bfloat16*>(a.norm_weight);
  p.tail.eps = a.norm_eps;
  p.tail.out_scale = a.out_scale;
  p.cgs = (p.group + 3) / 4;
  const long long tokens = static_cast<long long>(a.num_blocks) * a.block_size;
  const long long capacity = static_cast<long long>(a.max_blocks_per_seq) << p.cpb_log2;
  CUtensorMap tk = {}, tv = {};
  {
    // the chunks a sequence can have: the block table's capacity, or the window's and the
    // sinks' with their edges
    const long long seen = p.window > 0 ? p.window / kChunk + 2LL + (p.sinks + kChunk - 1LL) / kChunk : capacity;
    const long long chunks = seen < capacity ? seen : capacity;
    const long long per_warp = (chunks + kSpread * kWarps - 1) / (kSpread * kWarps);
    if (per_warp <= kDirectMost && static_cast<long long>(a.num_seqs) * (p.hkv / 2) <= direct_clusters()) {
      if (!cache_map(&tk, a.k_cache, a.num_kv_heads, tokens, 2) ||
          !cache_map(&tv, a.v_cache, a.num_kv_heads, tokens, 2))
        return cudaErrorInvalidValue;
      return launch_pdl(diff_direct_kernel, dim3(a.num_seqs * kSpread, 1, p.hkv / 2), dim3(kWarps * 32),
                        direct_smem(static_cast<int>(per_warp), p.cgs), stream, tk, tv, p,
                        static_cast<int>(per_warp));
    }
  }
  const int ppc = pairs_per_cta(p.hkv);
  p.hpc = 2 * ppc;
  p.units = ppc * p.cgs;
  p.wph = kWarps / p.units;
  p.producers = p.wph < kMaxProducers ? p.wph : kMaxProducers;
  const int groups = p.hkv / p.hpc;
  p.ctas = a.sms / groups < 1 ? 1 : a.sms / groups;
  p.cps_log2 = 2;
  for (;; --p.cps_log2) {              // two stages a ring at least, by smaller stages
    p.kv_bytes = (p.hpc << p.cps_log2) * 2 * kBf16Tile;
    p.stage_bytes = align_up(p.kv_bytes + p.hpc * p.group * kD * 2, 1024);
    const uint32_t fixed = diff_layout(p, 0).total + 1024 + 16;
    const int most = static_cast<int>((kSmemLimit - fixed) / (p.stage_bytes + sizeof(StageMeta) + 16));
    p.ring = (most > 48 ? 48 : most) / p.wph;
    if (p.ring >= 2 || p.cps_log2 == 0) break;
  }
  p.stages = p.ring * p.wph;
  if (p.ring < 1) return cudaErrorInvalidConfiguration;
  p.seg_weight = kSegWeight;
  const long long longest = capacity + p.seg_weight;
  p.small = a.num_seqs <= (p.units * p.wph + p.producers) * 32 && longest * a.num_seqs * (p.ctas + 1) < (1LL << 31);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const size_t rows = 2 * static_cast<size_t>(p.ctas) * a.num_q_heads;
  const size_t ab = (rows * 4 + 255) / 256 * 256;
  p.ws_m = reinterpret_cast<float*>(ws);
  p.ws_l = reinterpret_cast<float*>(ws + ab);
  p.ws_acc = reinterpret_cast<float*>(ws + 2 * ab);
  p.ws_split = reinterpret_cast<int4*>(ws + 2 * ab + rows * kDV * 4);
  p.ws_total = reinterpret_cast<long long*>(ws + 2 * ab + rows * kDV * 4 +
                                            (static_cast<size_t>(p.ctas) * 16 + 255) / 256 * 256);
  if (!cache_map(&tk, a.k_cache, a.num_kv_heads, tokens, p.hpc) ||
      !cache_map(&tv, a.v_cache, a.num_kv_heads, tokens, p.hpc))
    return cudaErrorInvalidValue;
  static PerDeviceOnce once;
  cudaError_t e = once.run([&] {
    return cudaFuncSetAttribute(diff_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
  });
  if (e != cudaSuccess) return e;
  e = launch_pdl(diff_decode_kernel, dim3(p.ctas, 1, groups), dim3((p.units * p.wph + p.producers) * 32),
                 diff_layout(p, p.stages).total + 1024, stream, tk, tv, p);
  if (e != cudaSuccess) return e;
  // a sequence has about 1 + ctas / num_seqs records: one warp a pair and batch of them
  int parts = 1;
  while (parts < kMergeWarps && static_cast<long long>(parts) * kMergeBatch * a.num_seqs < p.ctas) parts *= 2;
  const int per = parts < 4 ? 4 : kMergeWarps / parts;
  return launch_pdl(diff_merge_kernel,
                    dim3(a.num_seqs < p.ctas ? a.num_seqs : p.ctas, (p.pairs + per - 1) / per),
                    dim3(per * parts * 32), 0, stream, p, parts);
}

}  // namespace tvl
