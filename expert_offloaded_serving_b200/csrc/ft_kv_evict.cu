// ft_kv_evict: eviction from the paged cache by accumulated attention weight.
//
// Per (sequence, KV head) the entries are ordered by one 32-bit key:
//   2^31 + pos            if pos > newest - recent (recent entries stay first)
//   bits of the mass      otherwise (for mass >= 0 the order of the bits is the
//                         order of the values, and they stay below 2^31)
// and the budget's worth of largest keys survives, the lower slot first among
// equals.  k_kv_select finds the budget-th largest key by radix selection
// (11 + 11 + 10 bits: three histograms), ranks the equals at that key in the
// order of their slots, and lists the rows of the evicted slots below the budget
// and of the survivors above it, both ascending.  There are as many of each, and the
// two sets are disjoint, so k_kv_move copies the r-th survivor into the r-th freed
// slot with no order between the copies: only entries that must move are touched.
//
// Bound by latency, then memory: mass and position are read once (8 bytes an
// entry) into registers, with every load in flight before the first is used, and the
// passes of the selection run on registers; then the moved rows are read and
// written (a ragged half of 32 sequences, 8 KV heads: 16 us of selection, 31 us for 160 MB of
// moves, 5.2 TB/s).  A cluster of blocks shares one (sequence, KV head) while there are few of
// them; histograms and counts meet over distributed shared memory, every block
// reading the others', so that a pass waits for the cluster once.
#include <cooperative_groups.h>

#include "ft_kv.cuh"

namespace cg = cooperative_groups;

namespace ft {

namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;                    // of the first two passes
constexpr int kAllBins = 2 * kBins + kBins / 2;  // of all three
constexpr int kMoveThreads = 256;

struct EvictWork {
  int4* plan;     // [n_seqs * n_kv] moves, first entry of the lists, budget (-1: the sequence stays as it is), length
  int32_t* list;  // per item `length` rows: of freed slots from the front, of survivors from length / 2 on
};

__host__ __device__ inline int64_t carve(EvictWork& w, uint8_t* base, int n_seqs, int n_kv, int64_t rows) {
  int64_t at = 0;
  w.plan = reinterpret_cast<int4*>(base);
  at += pad_up((int64_t)n_seqs * n_kv * sizeof(int4), 256);
  w.list = reinterpret_cast<int32_t*>(base + at);
  at += pad_up(rows * (int64_t)sizeof(int32_t), 256);
  return at;
}

struct SelectArgs {
  KvEvictArgs a;
  EvictWork w;
  int64_t rows;  // entries of the lists
  int items;     // n_seqs * n_kv
};

struct SelectShared {
  uint32_t hist[kAllBins];   // the block's own, one run for each pass
  uint32_t total[kAllBins];  // the cluster's: each block holds an equal run of bins for all
  uint32_t warp_sum[kSelWarps];
  int len, budget;          // rank 0: of the sequence
  int newest;
  uint32_t bin, above, equal;  // the chosen bin, entries in the bins above it and in it
  uint32_t holes, movers;
  unsigned long long before;
};

// Exclusive prefix of one value a warp over the block's warps, and their sum.
__device__ __forceinline__ uint32_t warps_before(uint32_t mine, uint32_t* s, uint32_t& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (lane == 0) s[warp] = mine;
  __syncthreads();
  uint32_t before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < kSelWarps; w++) {
    if (w < warp) before += s[w];
    all += s[w];
  }
  return before;
}

// N: entries of a thread that are in registers.  ONE: that is all of them (a block's
// share of the longest possible sequence); else every pass reads them again in rounds.
template <int N, bool ONE>
__global__ void __launch_bounds__(kSelThreads, ONE && N <= 16 ? 2 : 1) k_kv_select(SelectArgs args) {
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ SelectShared sh;
  const KvView& kv = args.a.kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int blocks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int item = blockIdx.x / blocks, b = item / kv.Hkv, h = item - b * kv.Hkv;
  auto sync = [&] {
    if (blocks == 1) __syncthreads();
    else cluster.sync();
  };

  for (int i = tid; i < kAllBins; i += kSelThreads) sh.hist[i] = sh.total[i] = 0;
  if (tid == 0) {
    sh.newest = -1;
    sh.before = 0;
  }
  kv_pdl_wait();
  kv_pdl_trigger();
  // Length and budget are read once for the cluster: all its threads take the same way.
  if (rank == 0 && tid == 0) {
    sh.len = kv_length(kv, b, true);
    sh.budget = args.a.budgets[b];
    if (sh.budget < 0) set_status(kv.status, kStBadId);
  }
  sync();
  const int len = *cluster.map_shared_rank(&sh.len, 0), asked = *cluster.map_shared_rank(&sh.budget, 0);
  const int budget = asked < 0 ? len : asked;
  if (len <= budget) {
    if (rank == 0 && tid == 0) args.w.plan[item] = make_int4(0, 0, -1, 0);
    if (blocks > 1) cluster.sync();
    return;
  }
  // Where this item's lists begin: entries of the over-full sequences before it.
  {
    int64_t sum = 0;
    for (int i = tid; i < b; i += kSelThreads) {
      const int n = kv_length(kv, i), bud = args.a.budgets[i];
      if (bud >= 0 && n > bud) sum += n;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0 && sum) atomicAdd(&sh.before, (unsigned long long)sum);
  }
  // This block's slots, a multiple of 32 to each warp.
  const int share = (len + blocks - 1) / blocks, warp_share = ((share + kSelThreads - 1) / kSelThreads) * 32;
  const int begin = min(len, rank * warp_share * kSelWarps), end = min(len, begin + warp_share * kSelWarps);
  const int w_begin = min(end, begin + warp * warp_share), w_end = min(end, w_begin + warp_share);
  const int32_t* const pages = kv.table + (int64_t)b * kv.max_pages;

  // Entry i0 + 32 e + lane, for e < N: row (-1: none), position (-1: none), mass key.
  int row[N], pos[N];
  uint32_t key[N];
  auto load = [&](int i0) {
#pragma unroll
    for (int e = 0; e < N; e++) {
      const int i = i0 + 32 * e + lane;
      row[e] = i < w_end ? pages[i >> kv.page_shift] : 0;
    }
#pragma unroll
    for (int e = 0; e < N; e++) {
      const int i = i0 + 32 * e + lane;
      const bool real = i < w_end && (unsigned)row[e] < (unsigned)kv.n_pages;
      if (i < w_end && !real) set_status(kv.status, kStBadId);
      row[e] = real ? ((row[e] * kv.Hkv + h) << kv.page_shift) + (i & kv.page_mask) : -1;
      pos[e] = real ? kv.pos[row[e]] : -1;
      key[e] = real ? __float_as_uint(kv.mass[row[e]]) : 0u;  // no page: nothing there to keep
    }
#pragma unroll
    for (int e = 0; e < N; e++)
      if (!(__uint_as_float(key[e]) > 0.0f)) key[e] = 0u;
  };
  int recent_above = 0;  // positions above this one are recent
  auto rank_recent = [&] {
#pragma unroll
    for (int e = 0; e < N; e++)
      if (pos[e] > recent_above) key[e] = 0x80000000u + (uint32_t)pos[e];
  };
  auto rounds = [&](auto&& f) {  // f(first slot) with key[] ready, in the order of the slots
    if (ONE) {
      f(w_begin);
    } else {
      for (int i0 = w_begin; i0 < w_end; i0 += 32 * N) {
        load(i0);
        rank_recent();
        f(i0);
      }
    }
  };

  int newest = -1;
  for (int i0 = w_begin; i0 < w_end; i0 += 32 * N) {
    load(i0);
#pragma unroll
    for (int e = 0; e < N; e++) newest = max(newest, pos[e]);
    if (ONE) break;
  }
  if (ONE && w_begin >= w_end) {
#pragma unroll
    for (int e = 0; e < N; e++) {
      row[e] = pos[e] = -1;
      key[e] = 0u;
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) newest = max(newest, __shfl_xor_sync(0xffffffffu, newest, d));
  if (lane == 0) atomicMax(&sh.newest, newest);
  sync();
  newest = lane < blocks ? *cluster.map_shared_rank(&sh.newest, lane) : -1;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) newest = max(newest, __shfl_xor_sync(0xffffffffu, newest, d));
  recent_above = (int)max((int64_t)newest - args.a.recent, (int64_t)-1);
  if (ONE) rank_recent();
  const int64_t list0 = (int64_t)sh.before * kv.Hkv + (int64_t)h * len;

  // radix selection of the budget-th largest key
  uint32_t prefix = 0, want = (uint32_t)budget;  // entries still to be found among those with this prefix
#pragma unroll
  for (int pass = 0; pass < 3; pass++) {
    const int bits = pass == 2 ? 10 : 11, shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = 1 << bits;
    rounds([&](int i0) {
#pragma unroll
      for (int e = 0; e < N; e++)
        if (i0 + 32 * e + lane < w_end && (uint32_t)((uint64_t)key[e] >> (shift + bits)) == prefix)
          atomicAdd(&sh.hist[pass * kBins + ((key[e] >> shift) & (bins - 1))], 1u);
    });
    __syncthreads();
    // suffix sums: thread t owns bins / kSelThreads neighbouring bins, the highest bins first
    constexpr int kOwn = kBins / kSelThreads;
    const int own = bins / kSelThreads, top = bins - tid * own;  // bins top - own .. top - 1
    const int run_bits = bits - (31 - __clz(blocks));            // bins a block holds for all: 1 << run_bits
    uint32_t n[kOwn], sum = 0;
#pragma unroll
    for (int i = 0; i < kOwn; i++) n[i] = i < own ? sh.hist[pass * kBins + top - 1 - i] : 0u;
    if (blocks > 1) {
#pragma unroll
      for (int i = 0; i < kOwn; i++)
        if (n[i]) atomicAdd(cluster.map_shared_rank(&sh.total[pass * kBins + top - 1 - i], (top - 1 - i) >> run_bits), n[i]);
      cluster.sync();
#pragma unroll
      for (int i = 0; i < kOwn; i++)
        if (i < own) n[i] = *cluster.map_shared_rank(&sh.total[pass * kBins + top - 1 - i], (top - 1 - i) >> run_bits);
    }
#pragma unroll
    for (int i = 0; i < kOwn; i++) sum += n[i];
    uint32_t run = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, run, d);
      if (lane >= d) run += x;
    }
    uint32_t all;
    const uint32_t warp_total = __shfl_sync(0xffffffffu, run, 31);
    uint32_t above = warps_before(warp_total, sh.warp_sum, all) + run - sum;
#pragma unroll
    for (int i = 0; i < kOwn; i++) {
      if (i < own && above < want && above + n[i] >= want) {
        sh.bin = (uint32_t)(top - 1 - i);
        sh.above = above;
        sh.equal = n[i];
      }
      above += n[i];
    }
    if (want == 0 && tid == 0) {  // nothing survives: above every key
      sh.bin = (uint32_t)(bins - 1);
      sh.above = 0;
      sh.equal = 1;
    }
    __syncthreads();
    prefix = (prefix << bits) | sh.bin;
    want -= sh.above;
  }
  const uint32_t threshold = prefix;  // `want` of the entries with this key survive, the lowest slots

  // Ranks of the equals: blocks, then warps, then lanes.  Where all of them survive (keys
  // that differ) there is nothing to rank.
  const bool ranked = sh.equal != want;
  uint32_t tie = 0;
  if (ranked) {
    tie = lane < rank ? *cluster.map_shared_rank(&sh.hist[2 * kBins + (threshold & 1023u)], lane) : 0u;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) tie += __shfl_xor_sync(0xffffffffu, tie, d);
    uint32_t mine = 0, all;
    rounds([&](int i0) {
#pragma unroll
      for (int e = 0; e < N; e++)
        mine += __popc(__ballot_sync(0xffffffffu, i0 + 32 * e + lane < w_end && key[e] == threshold));
    });
    tie += warps_before(mine, sh.warp_sum, all);
  }
  const uint32_t below = (1u << lane) - 1u;
  // f(slot, row, is a freed slot, is a survivor to move) for every 32 entries
  auto classify = [&](auto&& f) {
    uint32_t at = tie;
    rounds([&](int i0) {
#pragma unroll
      for (int e = 0; e < N; e++) {
        const int i = i0 + 32 * e + lane;
        const bool in = i < w_end;
        bool kept = key[e] >= threshold && in;
        if (ranked) {
          const bool mine = in && key[e] == threshold;
          const uint32_t equal = __ballot_sync(0xffffffffu, mine);
          if (mine) kept = at + __popc(equal & below) < want;
          at += __popc(equal);
        }
        f(i, row[e], in && !kept && i < budget, kept && i >= budget);
      }
    });
  };
  uint32_t holes = 0, movers = 0, all_holes, all_movers;
  classify([&](int, int, bool is_hole, bool is_mover) {
    holes += is_hole;
    movers += is_mover;
  });
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    holes += __shfl_xor_sync(0xffffffffu, holes, d);
    movers += __shfl_xor_sync(0xffffffffu, movers, d);
  }
  uint32_t hole = warps_before(holes, sh.warp_sum, all_holes);
  uint32_t mover = warps_before(movers, sh.warp_sum, all_movers);
  if (tid == 0) {
    sh.holes = all_holes;
    sh.movers = all_movers;
  }
  sync();
  uint32_t moves = 0;
  {
    uint32_t nh = 0, nm = 0;
    if (lane < blocks) {
      nh = *cluster.map_shared_rank(&sh.holes, lane);
      nm = *cluster.map_shared_rank(&sh.movers, lane);
    }
    moves = nh;
    if (lane >= rank) nh = nm = 0;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      nh += __shfl_xor_sync(0xffffffffu, nh, d);
      nm += __shfl_xor_sync(0xffffffffu, nm, d);
      moves += __shfl_xor_sync(0xffffffffu, moves, d);
    }
    hole += nh;
    mover += nm;
  }
  // the lists; a page that two sequences share could make them longer than the pool
  const bool fits = list0 + len <= args.rows;
  if (!fits && tid == 0) set_status(kv.status, kStBadId);
  if (fits) {
    int32_t* const freed = args.w.list + list0;
    int32_t* const from = freed + (len >> 1);
    classify([&](int, int at_row, bool is_hole, bool is_mover) {
      const uint32_t hb = __ballot_sync(0xffffffffu, is_hole), mb = __ballot_sync(0xffffffffu, is_mover);
      if (is_hole) freed[hole + __popc(hb & below)] = at_row;
      if (is_mover) from[mover + __popc(mb & below)] = at_row;
      hole += __popc(hb);
      mover += __popc(mb);
    });
  }
  if (rank == 0 && tid == 0)
    args.w.plan[item] = make_int4(fits ? (int)moves : 0, (int)list0, fits ? budget : -1, len);
  if (blocks > 1) cluster.sync();  // no block leaves while another reads its shared memory
}

// The r-th survivor's key and value rows, mass and position into the r-th freed
// slot.  A group of lanes takes a row, 16 bytes a lane; all items' moves in one order
// are dealt out to the groups of the grid.
template <int RB>
__global__ void __launch_bounds__(kMoveThreads) k_kv_move(SelectArgs args) {
  constexpr int kLanes = RB / 16 > 16 ? 32 : RB / 16 > 8 ? 16 : RB / 16 > 4 ? 8 : 4;  // of a row
  constexpr int kGroups = kMoveThreads / kLanes;
  constexpr int kDeep = 4;  // moves a group has in flight
  __shared__ int64_t s_sum[kMoveThreads + 1];
  __shared__ int64_t s_warp[kMoveThreads / 32];
  const KvView& kv = args.a.kv;
  const int tid = threadIdx.x;
  kv_pdl_trigger();
  kv_pdl_wait();
  const int per = (args.items + kMoveThreads - 1) / kMoveThreads;
  {
    int64_t sum = 0;
    for (int i = tid * per; i < min(args.items, (tid + 1) * per); i++) {
      const int4 plan = args.w.plan[i];
      sum += plan.x;
      if (blockIdx.x == 0 && plan.z >= 0 && i % kv.Hkv == 0) kv.lengths[i / kv.Hkv] = plan.z;
    }
    int64_t run = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, run, d);
      if ((tid & 31) >= d) run += x;
    }
    if ((tid & 31) == 31) s_warp[tid >> 5] = run;
    __syncthreads();
    for (int w = 0; w < tid >> 5; w++) run += s_warp[w];
    s_sum[tid + 1] = run;
    if (tid == 0) s_sum[0] = 0;
    __syncthreads();
  }
  const int64_t total = s_sum[kMoveThreads];
  const int group = blockIdx.x * kGroups + tid / kLanes, lane = tid % kLanes;
  const int64_t step = (int64_t)gridDim.x * kGroups;
  for (int64_t f0 = group; f0 < total; f0 += step * kDeep) {
    int to[kDeep], src[kDeep];
    uint4 kd[kDeep], vd[kDeep];
    float mass[kDeep];
    int pos[kDeep];
#pragma unroll
    for (int d = 0; d < kDeep; d++) {
      const int64_t f = f0 + d * step;
      to[d] = src[d] = -1;
      if (f < total) {
        int lo = 0, hi = kMoveThreads;  // s_sum[lo] <= f < s_sum[hi]
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const int m = (lo + hi) >> 1;
          if (s_sum[m] <= f) lo = m;
          else hi = m;
        }
        int64_t r = f - s_sum[lo];
        int item = lo * per;
        int4 plan = args.w.plan[item];
        while (r >= plan.x) {
          r -= plan.x;
          plan = args.w.plan[++item];
        }
        const int32_t* const list = args.w.list + (int64_t)(uint32_t)plan.y + r;
        to[d] = list[0];
        src[d] = list[plan.w >> 1];
      }
    }
#pragma unroll
    for (int d = 0; d < kDeep; d++) {
      if (src[d] < 0 || to[d] < 0) {  // a page that is missing
        to[d] = -1;
        continue;
      }
      if (lane * 16 < RB) {
        kd[d] = *reinterpret_cast<const uint4*>(kv.k + (int64_t)src[d] * RB + lane * 16);
        vd[d] = *reinterpret_cast<const uint4*>(kv.v + (int64_t)src[d] * RB + lane * 16);
      }
      if (lane == 0) {
        mass[d] = kv.mass[src[d]];
        pos[d] = kv.pos[src[d]];
      }
    }
#pragma unroll
    for (int d = 0; d < kDeep; d++) {
      if (to[d] < 0) continue;
      if (lane * 16 < RB) {
        *reinterpret_cast<uint4*>(kv.k + (int64_t)to[d] * RB + lane * 16) = kd[d];
        *reinterpret_cast<uint4*>(kv.v + (int64_t)to[d] * RB + lane * 16) = vd[d];
      }
      if (lane == 0) {
        kv.mass[to[d]] = mass[d];
        kv.pos[to[d]] = pos[d];
      }
    }
  }
}

template <int N, bool ONE>
cudaError_t select(const SelectArgs& a, int blocks, int device, cudaStream_t s) {
  auto kern = k_kv_select<N, ONE>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = kv_attribute_once(done, device, kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.items * blocks));
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)blocks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

int64_t kv_evict_workspace(const ft_kv_cache& c) {
  EvictWork w;
  return carve(w, nullptr, c.n_seqs, c.n_kv_heads, c.n_pages * c.n_kv_heads * c.page_size);
}

cudaError_t launch_kv_evict(const KvEvictArgs& args, int row_bytes, int device, int sms, cudaStream_t s) {
  const KvView& kv = args.kv;
  SelectArgs a;
  a.a = args;
  a.rows = (int64_t)kv.n_pages * kv.Hkv << kv.page_shift;
  carve(a.w, args.work, kv.n_seqs, kv.Hkv, a.rows);
  a.items = kv.n_seqs * kv.Hkv;
  // Blocks of a cluster: one takes 4,096 entries in 8 a thread; more share longer sequences
  // while the items alone do not fill the GPU.  A pass costs a cluster 1.7 to 3 us, one block
  // alone 1.2 (64 items of 2,112 entries: 12.9 us alone, 15.4 in pairs), and what a thread
  // reads beyond that costs more (two sequences of 131,000: 42 us in 16 blocks, 89 in 8).
  int blocks = 1;
  while (blocks < 16 && kv.cap > 4096 * blocks && a.items * blocks * 2 <= sms) blocks *= 2;
  // Entries of a thread, by the longest sequence the table has room for (lengths are known on the device
  // alone): all of them in registers where they are 32 at most.  20 serve a context of 131,072 entries and a page
  // to spare in 16 blocks (17 a thread): two such sequences 41.8 us, 46.6 with 32 in that place.  A table much wider than
  // its sequences pays for it by reading mass and position again in every pass: 8 sequences of 2,112 entries, 8 KV
  // heads, 13.1 us in a table for 2,128, 32.9 in one for 131,072.
  const int share = (kv.cap + blocks - 1) / blocks, each = (share + kSelThreads - 1) / kSelThreads;
  cudaError_t e = each <= 4    ? select<4, true>(a, blocks, device, s)
                  : each <= 8  ? select<8, true>(a, blocks, device, s)
                  : each <= 16 ? select<16, true>(a, blocks, device, s)
                  : each <= 20 ? select<20, true>(a, blocks, device, s)
                  : each <= 32 ? select<32, true>(a, blocks, device, s)
                               : select<16, false>(a, blocks, device, s);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(sms * 4));  // all resident: 64 registers a thread
  switch (row_bytes) {
    case 64: return kv_launch_after(k_kv_move<64>, grid, kMoveThreads, 0, s, a);
    case 96: return kv_launch_after(k_kv_move<96>, grid, kMoveThreads, 0, s, a);
    case 128: return kv_launch_after(k_kv_move<128>, grid, kMoveThreads, 0, s, a);
    case 192: return kv_launch_after(k_kv_move<192>, grid, kMoveThreads, 0, s, a);
    case 256: return kv_launch_after(k_kv_move<256>, grid, kMoveThreads, 0, s, a);
    case 384: return kv_launch_after(k_kv_move<384>, grid, kMoveThreads, 0, s, a);
    default: return kv_launch_after(k_kv_move<512>, grid, kMoveThreads, 0, s, a);
  }
}

}  // namespace ft
