// ft_kv_evict: eviction from the paged cache by accumulated attention weight.
//
// Per (sequence, KV head) the entries are ordered by one 32-bit key:
//   2^31 + pos            if pos > newest - recent (recent entries stay first)
//   bits of the mass      otherwise (for mass >= 0 the order of the bits is the
//                         order of the values, and they stay below 2^31)
// and the budget's worth of largest keys survives, the lower slot first among
// equals.  k_kv_select finds the budget-th largest key by radix selection
// (11 + 11 + 10 bits: three histograms), ranks the equals at that key in the order of their
// slots, and lists the evicted slots below the budget and the survivors above
// it, both ascending.  There are as many of each, and the two sets are disjoint, so
// k_kv_move copies the r-th survivor into the r-th freed slot with no order
// between the copies: only entries that must move are touched.
//
// Bound by memory: mass and position once (8 bytes an entry), then the moved
// rows read and written.  A cluster of blocks shares one (sequence, KV head):
// keys stay in shared memory for the passes behind the first, histograms and
// prefix sums meet over distributed shared memory.
#include <cooperative_groups.h>

#include "ft_kv.cuh"

namespace cg = cooperative_groups;

namespace ft {

namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kKeyWords = 40 * 1024;   // keys a block keeps in shared memory (160 KB)
constexpr int kMoveThreads = 256;

struct EvictWork {
  int4* plan;     // [n_seqs * n_kv] moves, first entry of the lists, budget (-1: the sequence stays as it is), length
  int32_t* list;  // per item `length` entries: freed slots from the front, survivors from length / 2 on
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
  int64_t rows;   // entries of the lists
  int keep_keys;  // keys a block keeps in shared memory
  int per_item;   // blocks of k_kv_move for an item
};

struct SelectShared {
  uint32_t hist[kBins];
  uint32_t total[kBins];   // rank 0: the cluster's histogram
  uint32_t warp_sum[kSelWarps];
  int newest;
  uint32_t bin, above;     // rank 0: the chosen bin, entries in the bins above it
  uint32_t ties, holes, movers;
  int64_t before;
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

__global__ void __launch_bounds__(kSelThreads, 1) k_kv_select(SelectArgs args) {
  cg::cluster_group cluster = cg::this_cluster();
  extern __shared__ __align__(16) uint32_t s_keys[];  // keys, then a bit an entry: it survives
  __shared__ SelectShared sh;
  const KvView& kv = args.a.kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int blocks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int item = blockIdx.x / blocks, b = item / kv.Hkv, h = item - b * kv.Hkv;

  kv_pdl_trigger();
  const int len = kv_length(kv, b, true);
  int budget = args.a.budgets[b];
  if (budget < 0) {
    if (tid == 0) set_status(kv.status, kStBadId);
    budget = len;
  }
  if (len <= budget) {  // the same answer in every block of the cluster
    if (rank == 0 && tid == 0) args.w.plan[item] = make_int4(0, 0, -1, 0);
    return;
  }
  // Where this item's lists begin: entries of the over-full sequences before it.
  if (tid == 0) sh.before = 0;
  __syncthreads();
  {
    int64_t sum = 0;
    for (int i = tid; i < b; i += kSelThreads) {
      const int n = kv_length(kv, i), bud = args.a.budgets[i];
      if (bud >= 0 && n > bud) sum += n;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0 && sum) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.before), (unsigned long long)sum);
  }
  // This block's slots, a multiple of 32 to each warp.
  const int share = (len + blocks - 1) / blocks, warp_share = ((share + kSelThreads - 1) / kSelThreads) * 32;
  const int begin = min(len, rank * warp_share * kSelWarps), end = min(len, begin + warp_share * kSelWarps);
  const int w_begin = min(end, begin + warp * warp_share), w_end = min(end, w_begin + warp_share);
  const bool cached = warp_share * kSelWarps <= args.keep_keys;
  uint32_t* const s_bits = s_keys + args.keep_keys;

  // newest position of the head
  if (tid == 0) sh.newest = -1;
  __syncthreads();
  const int64_t list0 = sh.before * kv.Hkv + (int64_t)h * len;
  int newest = -1;
  for (int i = w_begin + lane; i < w_end; i += 32) {
    const int row = kv_row(kv, b, h, i);
    if (row >= 0) newest = max(newest, kv.pos[row]);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) newest = max(newest, __shfl_xor_sync(0xffffffffu, newest, d));
  if (lane == 0) atomicMax(&sh.newest, newest);
  cluster.sync();
  newest = -1;
  for (int r = 0; r < blocks; r++) newest = max(newest, *cluster.map_shared_rank(&sh.newest, r));

  auto make_key = [&](int i) -> uint32_t {
    const int row = kv_row(kv, b, h, i);
    if (row < 0) return 0u;  // no page: nothing there to keep
    const int pos = kv.pos[row];
    if (pos >= 0 && (int64_t)pos > (int64_t)newest - args.a.recent) return 0x80000000u + (uint32_t)pos;
    const float m = kv.mass[row];
    return m > 0.0f ? __float_as_uint(m) : 0u;
  };
  auto key_at = [&](int i) -> uint32_t { return cached ? s_keys[i - begin] : make_key(i); };

  // radix selection of the budget-th largest key
  uint32_t prefix = 0, want = (uint32_t)budget;  // entries still to be found among those with this prefix
  int shift = 21;
  uint32_t local_ties = 0;
  for (int pass = 0; pass < 3; pass++) {
    const int bits = pass == 2 ? 10 : 11;
    for (int i = tid; i < kBins; i += kSelThreads) sh.hist[i] = 0;
    __syncthreads();
    for (int i0 = w_begin; i0 < w_end; i0 += 32) {
      const int i = i0 + lane;
      if (i < w_end) {
        const uint32_t key = pass == 0 ? make_key(i) : key_at(i);
        if (pass == 0 && cached) s_keys[i - begin] = key;
        const uint64_t hi = (uint64_t)key >> (shift + bits);
        if (hi == prefix) atomicAdd(&sh.hist[(key >> shift) & ((1u << bits) - 1)], 1u);
      }
    }
    cluster.sync();
    // every block adds its share of the bins over the cluster into rank 0's total
    const int bins = 1 << bits, each = (bins + blocks - 1) / blocks;
    uint32_t* const total = cluster.map_shared_rank(sh.total, 0);
    for (int i = rank * each + tid; i < min(bins, (rank + 1) * each); i += kSelThreads) {
      uint32_t sum = 0;
      for (int r = 0; r < blocks; r++) sum += *cluster.map_shared_rank(&sh.hist[i], r);
      total[i] = sum;
    }
    cluster.sync();
    if (rank == 0) {
      // suffix sums: thread t owns bins/kSelThreads neighbouring bins, the highest bins first
      const int own = bins / kSelThreads, top = bins - tid * own;  // bins top-own .. top-1
      uint32_t sum = 0;
      for (int i = 0; i < own; i++) sum += sh.total[top - 1 - i];
      uint32_t run = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, run, d);
        if (lane >= d) run += x;
      }
      uint32_t all;
      const uint32_t warp_total = __shfl_sync(0xffffffffu, run, 31);
      uint32_t above = warps_before(warp_total, sh.warp_sum, all) + run - sum;
      for (int i = 0; i < own; i++) {
        const uint32_t n = sh.total[top - 1 - i];
        if (above < want && above + n >= want) {
          sh.bin = (uint32_t)(top - 1 - i);
          sh.above = above;
        }
        above += n;
      }
      if (want == 0 && tid == 0) {  // nothing survives: above every key
        sh.bin = (uint32_t)(bins - 1);
        sh.above = 0;
      }
    }
    cluster.sync();
    const uint32_t bin = *cluster.map_shared_rank(&sh.bin, 0);
    want -= *cluster.map_shared_rank(&sh.above, 0);
    local_ties = sh.hist[bin];
    prefix = (prefix << bits) | bin;
    shift -= pass == 0 ? 11 : 10;
    cluster.sync();  // rank 0's words and the histograms have been read
  }
  const uint32_t threshold = prefix;  // `want` of the entries with this key survive, the lowest slots

  // ranks of the equals: blocks, then warps, then lanes
  if (tid == 0) sh.ties = local_ties;
  cluster.sync();
  uint32_t tie = 0;
  for (int r = 0; r < rank; r++) tie += *cluster.map_shared_rank(&sh.ties, r);
  {
    uint32_t mine = 0;
    for (int i0 = w_begin; i0 < w_end; i0 += 32) {
      const int i = i0 + lane;
      mine += __popc(__ballot_sync(0xffffffffu, i < w_end && key_at(i) == threshold));
    }
    uint32_t all;
    tie += warps_before(mine, sh.warp_sum, all);
  }
  const uint32_t tie0 = tie;
  uint32_t holes = 0, movers = 0;
  for (int i0 = w_begin; i0 < w_end; i0 += 32) {
    const int i = i0 + lane;
    const bool in = i < w_end;
    const uint32_t key = in ? key_at(i) : 0u;
    const uint32_t equal = __ballot_sync(0xffffffffu, in && key == threshold);
    const uint32_t at = tie + __popc(equal & ((1u << lane) - 1));
    const bool kept = in && (key > threshold || (key == threshold && at < want));
    tie += __popc(equal);
    const uint32_t keeps = __ballot_sync(0xffffffffu, kept);
    if (cached && lane == 0) s_bits[(i0 - begin) >> 5] = keeps;
    holes += __popc(__ballot_sync(0xffffffffu, in && !kept && i < budget));
    movers += __popc(__ballot_sync(0xffffffffu, kept && i >= budget));
  }
  uint32_t all_holes, all_movers;
  uint32_t hole = warps_before(holes, sh.warp_sum, all_holes);
  uint32_t mover = warps_before(movers, sh.warp_sum, all_movers);
  if (tid == 0) {
    sh.holes = all_holes;
    sh.movers = all_movers;
  }
  cluster.sync();
  uint32_t moves = 0;
  for (int r = 0; r < blocks; r++) {
    const uint32_t nh = *cluster.map_shared_rank(&sh.holes, r), nm = *cluster.map_shared_rank(&sh.movers, r);
    if (r < rank) {
      hole += nh;
      mover += nm;
    }
    moves += nh;
  }
  // the lists; a page that two sequences share could make them longer than the pool
  const bool fits = list0 + len <= args.rows;
  if (!fits && tid == 0) set_status(kv.status, kStBadId);
  if (fits) {
    int32_t* const freed = args.w.list + list0;
    int32_t* const from = freed + (len >> 1);
    uint32_t t = tie0;
    for (int i0 = w_begin; i0 < w_end; i0 += 32) {
      const int i = i0 + lane;
      const bool in = i < w_end;
      bool kept;
      if (cached) {
        kept = (s_bits[(i0 - begin) >> 5] >> lane) & 1u;
      } else {
        const uint32_t key = in ? key_at(i) : 0u;
        const uint32_t equal = __ballot_sync(0xffffffffu, in && key == threshold);
        kept = in && (key > threshold || (key == threshold && t + __popc(equal & ((1u << lane) - 1)) < want));
        t += __popc(equal);
      }
      const bool is_hole = in && !kept && i < budget, is_mover = kept && i >= budget;
      const uint32_t hb = __ballot_sync(0xffffffffu, is_hole), mb = __ballot_sync(0xffffffffu, is_mover);
      if (is_hole) freed[hole + __popc(hb & ((1u << lane) - 1))] = i;
      if (is_mover) from[mover + __popc(mb & ((1u << lane) - 1))] = i;
      hole += __popc(hb);
      mover += __popc(mb);
    }
  }
  if (rank == 0 && tid == 0)
    args.w.plan[item] = make_int4(fits ? (int)moves : 0, (int)list0, fits ? budget : -1, len);
  cluster.sync();  // no block leaves while another reads its shared memory
}

// The r-th survivor's key and value rows, mass and position into the r-th freed
// slot.  A group of lanes takes a row, 16 bytes a lane.
template <int RB>
__global__ void __launch_bounds__(kMoveThreads) k_kv_move(SelectArgs args) {
  constexpr int kLanes = RB / 16 > 16 ? 32 : RB / 16 > 8 ? 16 : RB / 16 > 4 ? 8 : 4;  // of a row
  constexpr int kGroups = kMoveThreads / kLanes;
  constexpr int kDeep = 4;  // moves a group has in flight
  const KvView& kv = args.a.kv;
  const int per_item = args.per_item;
  kv_pdl_wait();
  const int item = blockIdx.x / per_item, part = blockIdx.x - item * per_item;
  const int b = item / kv.Hkv, h = item - b * kv.Hkv;
  const int4 plan = args.w.plan[item];
  if (plan.z < 0) return;
  if (part == 0 && h == 0 && threadIdx.x == 0) kv.lengths[b] = plan.z;
  const int32_t* const freed = args.w.list + (int64_t)(uint32_t)plan.y;
  const int32_t* const from = freed + (plan.w >> 1);
  const int group = part * kGroups + threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int step = per_item * kGroups;
  for (int r0 = group; r0 < plan.x; r0 += step * kDeep) {
    int to[kDeep], src[kDeep];
    uint4 kd[kDeep], vd[kDeep];
    float mass[kDeep];
    int pos[kDeep];
#pragma unroll
    for (int d = 0; d < kDeep; d++) {
      const int r = r0 + d * step;
      to[d] = src[d] = -1;
      if (r < plan.x) {
        to[d] = kv_row(kv, b, h, freed[r]);
        src[d] = kv_row(kv, b, h, from[r]);
        if (src[d] < 0) to[d] = -1;
        if (to[d] < 0) src[d] = -1;
      }
    }
#pragma unroll
    for (int d = 0; d < kDeep; d++) {
      if (src[d] < 0) continue;
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

}  // namespace

int64_t kv_evict_workspace(const ft_kv_cache& c) {
  EvictWork w;
  return carve(w, nullptr, c.n_seqs, c.n_kv_heads, c.n_pages * c.n_kv_heads * c.page_size);
}

cudaError_t launch_kv_evict(const KvEvictArgs& args, int row_bytes, int sms, cudaStream_t s) {
  const KvView& kv = args.kv;
  SelectArgs a;
  a.a = args;
  a.rows = (int64_t)kv.n_pages * kv.Hkv << kv.page_shift;
  carve(a.w, args.work, kv.n_seqs, kv.Hkv, a.rows);
  const int items = kv.n_seqs * kv.Hkv;
  // Blocks of a cluster: one block takes 4,096 entries in 8 a thread; more
  // blocks share longer sequences while the items alone do not fill the GPU.
  int blocks = 1;
  while (blocks < 8 && kv.cap > 4096 * blocks && items * blocks < sms) blocks *= 2;
  // Two thousand threads an SM for the moves, shared out evenly: lengths are not
  // known here, and a block without moves leaves at once.
  a.per_item = (sms * 8 + items - 1) / items;
  // A block keeps its keys where its share of the longest sequence fits.
  const int share = (kv.cap + blocks - 1) / blocks;
  const int64_t need = (int64_t)((share + kSelThreads - 1) / kSelThreads) * kSelThreads;
  a.keep_keys = need <= kKeyWords ? (int)need : kKeyWords;
  const size_t smem = (size_t)(a.keep_keys + a.keep_keys / 32) * sizeof(uint32_t);
  cudaError_t e = cudaFuncSetAttribute(k_kv_select, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(items * blocks));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)blocks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, k_kv_select, a)) != cudaSuccess) return e;
  const dim3 grid((unsigned)(items * a.per_item));
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
