// ft_kv_attention: attention of one new token a sequence over its paged
// entries, split over the entries of the whole batch and joined.
//
// Mathematics: one pass over the entries with the running maximum m and sum l
// of a softmax.  For a tile of entries, with s = q.k in units of log2(e):
//   m' = max(m, max s), p = 2^(s - m'), l' = l 2^(m - m') + sum p,
//   O' = O 2^(m - m') + p V;  at the end out = O / l, lse = ln 2 (m + log2 l).
// Two parts of one row join the same way: weights 2^(m_i - max m).
//
// What bounds it: every cached byte is read once and meets G query heads, 4 G flops
// for 4 bytes of a BF16 entry.  At the measured copy rate an SM gets 22 bytes a
// clock, so 16 heads are 90 multiply-adds a clock an SM: far below what mma.sync
// does, a multiple of what the fp32 pipe could do next to the softmax.  So the
// products run on mma.sync, the entries as the 16 rows of a tile and 8 or 16 query
// heads of one KV head as its columns, and everything else serves the stream of
// loads: a tile of keys or values is one TMA copy into the ring of the warp that
// uses it.
//
// Split: the unit is a tile of 16 or 32 entries of one (sequence, KV head).  All tiles
// of the batch, in that order, are cut into equal contiguous chunks, one a warp; a warp
// streams its chunk through its own ring and meets no barrier with other warps.  With more
// than 16 query heads a KV head, a chunk goes to one warp for each group of 16: they
// begin together, so memory is read once and L2 serves the rest (32 sequences of 16,000 entries, 32
// heads over one of 128: 71 us, 75 with the groups one after the other).  A row (the tiles of one
// KV head) that lies inside one chunk is finished there; the parts of the others go to the
// workspace (fp32) and k_kv_join adds them in the order of the chunks.  Lengths are read on the device:
// ragged batches and idle rows are balanced by construction, a captured graph stays
// valid when lengths grow, and the split depends on nothing but the lengths and the
// number of SMs.
//
// With FT_KV_MASS the scores go to the workspace as they come (G fp32 values an entry, next to
// its 4 D or 2 D bytes), and k_kv_join turns them into weights once the row's lse
// is known.
//
// Measured (one B200, a graph of passes): 1 x 131,071 entries, 64 query and 8 KV heads of 128, BF16
// 92 us (5.8 TB/s; the slowest SMs end at 86, the mean one at 77: the share of the
// memory's rate that an SM gets differs by 13 %); 64 sequences of 300 to 16,000 entries
// 165 us (6.0 TB/s, 6.2 in the split); 48 of 500 to 12,000 in E4M3, 64 heads over 4 of 128, 57.6 us weighed
// and 38.2 not; 37 entries 6.4 us, two launches and four trips to memory.
#include "ft_gemm.h"
#include "ft_kv.cuh"
#include "ft_tc.cuh"

namespace ft {

namespace {

constexpr int kRows = 16;        // query heads of a group, which one warp takes

// The ring of a warp for entries of RB bytes a side: a stage holds a tile of keys
// and one of values as TMA leaves them, boxes of kBox bytes x the tile's rows whose
// 16-byte pieces are swizzled (ldmatrix then reads 8 rows from 8 different
// groups of banks).
//
// Tile and warps by what was measured: 32 entries halve the instructions around the
// products, up to rows of 256 bytes (131,072 entries of 256 bytes 93 us, 16 entries a tile 96).
// There 4 warps x 3 stages match 6 x 2 on long rows (93 and 92 us) and win on 64 sequences of 200
// entries (12.4 against 15.3); rows of 128 bytes want 8 warps (a ragged weighed batch of 48, 64 heads over 4
// of 128 57.6 us, 60.9 with 6, 65.1 with 12; 16 x 8,000 entries of the same heads 34.9, 41.3 and 38.9), rows of 96 too (64 sequences
// of 300 to 9,000 entries, 16 heads over one: 18.4, 21.2 with 12), rows of 64 want 16 (16 x 8,000
// entries, 8 heads with a KV head each: 31.1, 35.2 with 8; with one for all 14.9 and 11.6); beyond 256
// the registers of O leave room for 4.
//
// Registers: heads of 256 in E4M3 with more than 8 query heads a KV head hold 192 of O and q alone and spill
// 676 bytes a thread (12 sequences of 1,000 to 24,000 entries, 32 heads over 2: 49.6 us on a floor of 16); BF16 heads of
// 256 and E4M3 heads of 192 and 64 with as many spill 16 to 48.
constexpr int tile_of(int row_bytes) { return row_bytes <= 256 ? 32 : 16; }
constexpr int warps_of(int row_bytes) { return row_bytes >= 256 ? 4 : row_bytes == 64 ? 16 : 8; }
template <int RB>
struct Ring {
  static constexpr int kTile = tile_of(RB);  // entries
  static constexpr int kBox = RB % 128 == 0 ? 128 : RB % 64 == 0 ? 64 : 32;
  static constexpr int kBoxes = RB / kBox;
  static constexpr int kBoxBytes = kTile * kBox;
  static constexpr int kSide = kTile * RB;
  static constexpr int kStage = 2 * kSide;
  static constexpr int kWarps = warps_of(RB);
  static constexpr int kFit = 220 * 1024 / (kWarps * kStage);
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static constexpr int kBytes = kWarps * kStages * kStage + 1024;  // the swizzle goes by address: aligned to its period
};


// What warp j leaves for block j of k_kv_join: chunk j / groups, for the query heads of group j % groups.
struct __align__(16) Chunk {
  int b, h, first, len;   // sequence and KV head of its first tile, that row's first tile in the batch and its entries
  int tiles, size;        // its tiles (0: none), tiles of a chunk in this launch
  int go_b, go_h;         // the row that goes on past its end (go_b -1: none)
  int go_j0, go_parts;    // the chunk that row begins on, the chunks it lies on
  int pad[2];
};
struct AttnWork {
  Chunk* chunks;
  float2* ml;        // [warps][2][8 or 16] m and l of a part (log2 units); side 0: a row that came in, 1: one that goes on
  float* o;          // [warps][2][8 or 16][D]
  float* lse2;       // [n_seqs][Hq] lse of whole rows in log2 units (mass)
  float* scores;     // [groups][tiles][entries of a tile][score_rows] scores in log2 units (mass)
  int64_t tiles;     // that `scores` holds
};

__host__ __device__ inline int64_t up256(int64_t n) { return (n + 255) & ~(int64_t)255; }

// Scores kept of an entry, for G query heads a KV head: as many of the 8 or 16 heads of a warp as a power of two covers.
__host__ __device__ inline int score_rows(int G) { return G > 8 ? 16 : G > 4 ? 8 : G > 2 ? 4 : G; }

// Query heads of a KV head go in groups of 16.
__host__ __device__ inline int groups_of(int G) { return (G + kRows - 1) / kRows; }

// Scores of the tiles that sequences of their own pages can have: every row of the pool, and a last tile each.
inline int64_t carve(AttnWork& w, uint8_t* base, int D, int row_bytes, int n_seqs, int Hq, int Hkv, int64_t rows, bool mass) {
  const int G = Hq / Hkv, tile = tile_of(row_bytes), kept = G > 8 ? 16 : 8;  // heads of a warp
  const int64_t warps = kKvMaxSms * warps_of(row_bytes);
  int64_t at = 0;
  w.chunks = reinterpret_cast<Chunk*>(base + at);
  at += up256(warps * (int64_t)sizeof(Chunk));
  w.ml = reinterpret_cast<float2*>(base + at);
  at += up256(warps * 2 * kept * (int64_t)sizeof(float2));
  w.o = reinterpret_cast<float*>(base + at);
  at += up256(warps * 2 * kept * D * (int64_t)sizeof(float));
  w.lse2 = reinterpret_cast<float*>(base + at);
  w.scores = nullptr;
  w.tiles = 0;
  if (!mass) return at;
  at += up256((int64_t)n_seqs * Hq * sizeof(float));
  w.scores = reinterpret_cast<float*>(base + at);
  w.tiles = rows / tile + (int64_t)n_seqs * Hkv;
  at += up256(w.tiles * groups_of(G) * tile * score_rows(G) * (int64_t)sizeof(float));
  return at;
}

struct SplitArgs {
  CUtensorMap k_map, v_map;  // pools as kBox bytes x rows x kBoxes; a box has box_rows, and all kBoxes where that is a tile's rows
  KvAttnArgs a;
  AttnWork w;
  int groups;      // of 16 query heads, a KV head
  float per_part;  // 1 / (rows x kMaxParts)
  int box_shift;  // box_rows = 1 << box_shift: a tile's rows, or a page's where pages are smaller
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// Wait of a whole warp for phase `parity`; false after `limit` nanoseconds.  Votes decide, so that
// its lanes always go the same way: after the wait they meet in products, shuffles and
// votes that need every one of them.  A phase that one lane has seen stays complete until the warp
// itself loads the stage again.  The timer is read once the wait has already taken many polls.
__device__ __forceinline__ bool wait_full(uint64_t* bar, uint32_t parity, uint64_t limit = tc::kWaitNs) {
  const uint32_t at = smem_u32(bar);
  uint64_t since = 0;
  for (uint32_t n = 1;; n++) {
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(at), "r"(parity)
                 : "memory");
    if (__all_sync(0xffffffffu, ok)) return true;
    if ((n & 255) == 0) {
      const uint64_t now = tc::gtime();
      if (since == 0) since = now;
      if (__any_sync(0xffffffffu, now - since > limit)) return false;
    }
  }
}

// The wait alone (ft_debug_kv_wait): warp 0 of a block waits on a barrier at which warp 1 arrives
// after arrive_ns and a nanosecond for each block (never, if negative).
__global__ void __launch_bounds__(64) k_kv_wait(uint64_t limit_ns, int64_t arrive_ns, int32_t* lanes) {
  __shared__ __align__(8) uint64_t s_bar;
  if (threadIdx.x == 0) tc::mbar_init(&s_bar, 1);
  __syncthreads();
  if (threadIdx.x < 32) {
    const bool there = wait_full(&s_bar, 0, limit_ns);
    const int n = __syncthreads_count(there);
    if (threadIdx.x == 0) lanes[blockIdx.x] = n;
  } else {
    if (threadIdx.x == 32 && arrive_ns >= 0) {
      const uint64_t t0 = tc::gtime();
      while (tc::gtime() - t0 < (uint64_t)arrive_ns + blockIdx.x) __nanosleep(20);
      asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&s_bar)) : "memory");
    }
    __syncwarp();
    __syncthreads_count(false);
  }
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}

// c += A(16 x 16) B(16 x 8), fp32 accumulators.
template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  if (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// 8 x 8 values of 16 bits, transposed over the warp.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Four E4M3 bytes as two f16x2 (bytes 0, 1 and bytes 2, 3), exact.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  const __half2 b = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A place in the batch's order of tiles: sequence, KV head, tile of the row.
struct Place {
  int b, h, t, len, nt;
};

template <int TILE>
__device__ __forceinline__ int tiles_of(int len) {
  return (len + TILE - 1) / TILE;
}

template <int TILE>
__device__ __forceinline__ void next_sequence(const KvView& kv, Place& p) {
  do {
    p.len = ++p.b < kv.n_seqs ? kv_length(kv, p.b) : 1;
  } while (p.len == 0);
  p.b = min(p.b, kv.n_seqs - 1);  // past the end only if somebody changes the lengths meanwhile
  p.nt = tiles_of<TILE>(p.len);
}

template <int TILE>
__device__ __forceinline__ void advance(const KvView& kv, Place& p) {
  if (++p.t < p.nt) return;
  p.t = 0;
  if (++p.h < kv.Hkv) return;
  p.h = 0;
  next_sequence<TILE>(kv, p);
}

constexpr float kNegInf = -__builtin_huge_valf();

// Parts a row of mean length is cut into while a warp has fewer than 4 tiles: a warp for
// every tile of a short row is quickest (each further tile of a warp costs what the
// join of one more part does not), but one row's hundreds of parts are not (4,000
// entries, two KV heads of 256: 250 parts 17.3 us, 84 parts 12.7).
constexpr int kMaxParts = 64;
inline float part_share(int n_seqs, int n_kv) { return 1.0f / ((float)n_seqs * (float)n_kv * kMaxParts); }

// Tiles of a chunk: an equal share (all of them lie on the chunks there are), more for short rows.
__host__ __device__ inline int chunk_tiles(int total, int chunks, float per_part) {
  const int equal = (int)(((uint32_t)total + (uint32_t)chunks - 1u) / (uint32_t)chunks);
  const int fewer = (int)((float)total * per_part);
  const int least = fewer < 4 ? fewer : 4;
  const int n = equal > least ? equal : least;
  return n > 1 ? n : 1;
}

// A running maximum is replaced once a score passes it by this much (a factor of
// 256): any reference would do for the sums, and most tiles then need neither
// the maximum over the warp's lanes nor the rescaling of O.
//
// Over an E4M3 cache p meets v as f16, in two parts of 11 bits, and below 2^-14 f16 has fewer
// bits, below 2^-25 none.  So the reference is taken kLift lower there: the largest p is
// 2^7 to 2^15, still within f16 (a maximum that fp32 cannot lower by 7 only leaves p smaller), and what
// is lost of a weight is 2^-22 of itself or 2^-32 of the largest, whichever is more.  The second part
// costs 0 to 3 % (rows of 64 bytes with 16 heads a warp and heads of 256 with as many 11 %); one
// part alone is 8.5e-4 from what fp32 gives, both 1e-4 and less.
constexpr float kSlack = 8.0f;
constexpr float kLift = 7.0f;

// D: head_dim.  E4M3: the cache's format.  NB: blocks of 8 query heads of a
// warp.  MASS: scores go to the workspace.
template <int D, bool E4M3, int NB, bool MASS>
__global__ void __launch_bounds__(Ring<D * (E4M3 ? 1 : 2)>::kWarps * 32, 1) k_kv_split(const __grid_constant__ SplitArgs args) {
  constexpr int RB = D * (E4M3 ? 1 : 2);
  using R = Ring<RB>;
  constexpr int TILE = R::kTile, NT = TILE / 16;       // entries of a tile, steps of 16
  constexpr int kThreads = R::kWarps * 32;
  constexpr int kPieces = RB / 16, kBoxPieces = R::kBox / 16;  // 16-byte pieces of a row, of its part in a box
  constexpr int KC = NT * NB >= 4 ? 1 : 4 / (NT * NB);
  constexpr uint32_t kFull = TILE == 32 ? 0xffffffffu : 0xffffu;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t s_full[R::kWarps * R::kStages];
  __shared__ uint32_t s_there[R::kWarps * R::kStages];  // entries of a stage's tile that exist, a bit each
  __shared__ int s_sum[kThreads + 1];
  __shared__ int s_warp[R::kWarps];

  const KvView& kv = args.a.kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  uint64_t* const full = s_full + warp * R::kStages;
  if (lane < R::kStages) tc::mbar_init(full + lane, 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncwarp();  // lane 0 arrives at barriers that other lanes made
  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&args.k_map) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&args.v_map) : "memory");
  }
  kv_pdl_wait();
  kv_pdl_trigger();
  const int j = warp * gridDim.x + blockIdx.x;  // neighbours in the batch sit on different SMs
  const int groups = NB == 1 ? 1 : args.groups;
  const int warps = (int)gridDim.x * R::kWarps, chunks = warps / groups;
  const int c = j / groups, gi = j - c * groups;  // the warp's chunk and group; c can be `chunks`: nothing there
  // The tiles of the batch are counted, cut, and the chunk's first one is looked up: its
  // sequence, and that one's first tile in the batch.
  Place cons;
  int base, total, chunk, lo, hi;
  auto cut = [&] {
    chunk = chunk_tiles(total, chunks, args.per_part);
    lo = (int)min((int64_t)c * chunk, (int64_t)total);
    hi = min(lo + chunk, total);
  };
  if (kv.n_seqs <= 128) {  // every warp by itself, four sequences a lane
    int len[4], upto[4];  // tiles up to and with the lane's sequence
    total = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int b = i * 32 + lane;
      len[i] = b < kv.n_seqs ? kv_length(kv, b, blockIdx.x == 0 && warp == 0) : 0;
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
      upto[i] = total;
      if (i * 32 >= kv.n_seqs) continue;
      int run = tiles_of<TILE>(len[i]) * kv.Hkv;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, run, d);
        if (lane >= d) run += x;
      }
      upto[i] += run;
      total = __shfl_sync(0xffffffffu, upto[i], 31);
    }
    cut();
    cons.b = cons.len = base = 0;
#pragma unroll
    for (int i = 3; i >= 0; i--) {
      // sequences of these 32 whose tiles all lie before the chunk; one holds `lo` if not all do
      const int before = __popc(__ballot_sync(0xffffffffu, upto[i] <= lo));
      if (i * 32 >= kv.n_seqs || before == 32) continue;
      cons.b = i * 32 + before;
      cons.len = __shfl_sync(0xffffffffu, len[i], before);
      base = __shfl_sync(0xffffffffu, upto[i], before) - tiles_of<TILE>(cons.len) * kv.Hkv;
    }
  } else {  // the block together: a run of `per` sequences a thread
    const int per = (kv.n_seqs + kThreads - 1) / kThreads;
    int sum = 0;
    for (int i = 0; i < per; i++) {
      const int b = tid * per + i;
      if (b < kv.n_seqs) sum += tiles_of<TILE>(kv_length(kv, b, blockIdx.x == 0)) * kv.Hkv;
    }
    int run = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, run, d);
      if (lane >= d) run += x;
    }
    if (lane == 31) s_warp[warp] = run;
    __syncthreads();
    for (int w = 0; w < warp; w++) run += s_warp[w];
    s_sum[tid + 1] = run;
    if (tid == 0) s_sum[0] = 0;
    __syncthreads();
    total = s_sum[kThreads];
    cut();
    int l = 0, h = kThreads;  // s_sum[l] <= lo < s_sum[h]
    while (h - l > 1) {
      const int m = (l + h) >> 1;
      if (s_sum[m] <= lo) l = m;
      else h = m;
    }
    base = s_sum[l];
    cons.b = l * per;
    cons.len = 0;
    for (; lo < hi && cons.b < kv.n_seqs; cons.b++) {
      cons.len = kv_length(kv, cons.b);
      const int n = tiles_of<TILE>(cons.len) * kv.Hkv;
      if (lo < base + n) break;
      base += n;
    }
    if (cons.b >= kv.n_seqs || cons.len == 0) {  // only if somebody changes the lengths meanwhile
      cons.b = kv.n_seqs - 1;
      cons.len = 1;
      base = lo;
    }
  }
  // Idle rows, from the last warps on, which have no tiles in a small batch: out 0, lse -inf.
  auto idle_rows = [&] {
    for (int b = warps - 1 - j; b < kv.n_seqs; b += warps) {
      if (kv_length(kv, b) != 0) continue;
      uint4* o = reinterpret_cast<uint4*>(args.a.out + (int64_t)b * kv.Hq * D);
      for (int i = lane; i < kv.Hq * D / 8; i += 32) o[i] = make_uint4(0u, 0u, 0u, 0u);
      if (args.a.lse)
        for (int i = lane; i < kv.Hq; i += 32) args.a.lse[(int64_t)b * kv.Hq + i] = kNegInf;
    }
  };
  if (lo >= hi) {
    idle_rows();
    if (lane == 0) args.w.chunks[j] = Chunk{-1, 0, 0, 0, 0, chunk, -1, 0, 0, 0, {0, 0}};
    return;
  }
  cons.nt = tiles_of<TILE>(cons.len);
  cons.h = (lo - base) / cons.nt;
  cons.t = (lo - base) - cons.h * cons.nt;
  int row_first = lo - cons.t;  // first tile of the present row in the batch's order
  Chunk left{cons.b, cons.h, row_first, cons.len, hi - lo, chunk, -1, 0, 0, 0, {0, 0}};

  uint8_t* const ring = smem + ((1024u - (smem_u32(smem) & 1023u)) & 1023u) + warp * (R::kStages * R::kStage);
  const uint32_t ring32 = smem_u32(ring);
  uint32_t* const there_of = s_there + warp * R::kStages;

  // ---- producer: the tile's rows, a box (of one page) for each of the first lanes ----
  Place prod = cons;
  const int box_shift = args.box_shift, box_bytes = RB << box_shift;
  auto box_row = [&](const Place& p) {  // first row of the lane's box, -1 where there is none
    const int slot = p.t * TILE + (lane << box_shift);
    return lane < (TILE >> box_shift) && slot < p.len ? kv_row(kv, p.b, p.h, slot) : -1;
  };
  int row_next = box_row(prod), left_next = prod.len - prod.t * TILE;
  int to_load = hi - lo;
  auto load = [&](int stage) {
    if (to_load <= 0) return;
    to_load--;
    const int row = row_next, left = left_next;
    if (to_load > 0) {
      advance<TILE>(kv, prod);
      row_next = box_row(prod);
      left_next = prod.len - prod.t * TILE;
    }
    const uint32_t boxes = __ballot_sync(0xffffffffu, row >= 0);
    const uint32_t there = __ballot_sync(0xffffffffu, lane < TILE && lane < left && ((boxes >> (lane >> box_shift)) & 1u));
    if (lane == 0) {
      there_of[stage] = there;
      tc::mbar_expect(full + stage, (uint32_t)(__popc(boxes) * box_bytes * 2));
    }
    __syncwarp();
    if (row >= 0) {
      uint8_t* const at = ring + stage * R::kStage + ((lane << box_shift) * R::kBox);
      const int each = (1 << box_shift) == TILE ? R::kBoxes : 1;
#pragma unroll 1
      for (int i = 0; i < R::kBoxes; i += each) {
        tc::tma_3d(at + i * R::kBoxBytes, &args.k_map, 0, row, i, full + stage);
        tc::tma_3d(at + R::kSide + i * R::kBoxBytes, &args.v_map, 0, row, i, full + stage);
      }
    }
  };

  // ---- consumer ----
  // S^T = K Q^T: 16 entries x 8 heads, O^T = V^T P^T: 16 dims x 8 heads.  A lane
  // (g, j) of the mma layout has the heads 2j and 2j+1 of each block, the entries g
  // and g + 8 of S^T; P^T becomes the second product's operand by two transposes of
  // 8 x 8.
  const int g = lane >> 2, j2 = (lane & 3) * 2;
  uint32_t q[D / 16][NB][2];
  float o[D / 16][NB][4];
  float m[NB][2], l[NB][2], qs[NB][2];
  const int n_rows = min(kRows, kv.G - gi * kRows);
  int head0 = 0;

  auto begin_row = [&](int b, int h) {
    head0 = h * kv.G + gi * kRows;
    const float unit = args.a.scale * 1.4426950408889634f * kv.k_scale;
#pragma unroll
    for (int nb = 0; nb < NB; nb++) {
      // Columns without a head repeat the first one: add_mass takes their weights out by an lse of +inf,
      // and the scores of a q of zero would be NaN against an infinite key whatever the heads' own are.
      const uint16_t* src = args.a.q + (int64_t)b * args.a.q_stride + (int64_t)(head0 + (g + 8 * nb < n_rows ? g + 8 * nb : 0)) * D;
#pragma unroll
      for (int i = 0; i < 2; i++) {
        m[nb][i] = kNegInf;
        l[nb][i] = 0.0f;
        qs[nb][i] = unit;
      }
#pragma unroll
      for (int ks = 0; ks < D / 16; ks++) {
        // E4M3: the 16 contraction steps of an mma take the dims 4i, 4i+1 (first
        // half) and 4i+2, 4i+3 (second half) of each lane i of a quad: the order in
        // which ldmatrix hands out the bytes of a key.
        const uint2 x = E4M3 ? *reinterpret_cast<const uint2*>(src + ks * 16 + 2 * j2)
                             : make_uint2(*reinterpret_cast<const uint32_t*>(src + ks * 16 + j2),
                                          *reinterpret_cast<const uint32_t*>(src + ks * 16 + 8 + j2));
        q[ks][nb][0] = x.x;
        q[ks][nb][1] = x.y;
      }
    }
#pragma unroll
    for (int n = 0; n < D / 16; n++)
#pragma unroll
      for (int nb = 0; nb < NB; nb++)
#pragma unroll
        for (int i = 0; i < 4; i++) o[n][nb][i] = 0.0f;
  };

  // For an E4M3 cache q becomes f16 with a power-of-two factor that puts the head's
  // largest magnitude into [2^14, 2^15): exact for bf16 values down to 2^-28 of it.
  auto encode_row = [&] {
#pragma unroll
    for (int nb = 0; nb < NB; nb++) {
      float top = 0.0f;
#pragma unroll
      for (int ks = 0; ks < D / 16; ks++)
#pragma unroll
        for (int i = 0; i < 2; i++)
          top = fmaxf(top, fmaxf(fabsf(bf16_lo(q[ks][nb][i])), fabsf(bf16_hi(q[ks][nb][i]))));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = min((int)(__float_as_uint(top) >> 23), 254);  // biased exponent; next to an infinity the others have to fit all the same
      const bool usual = e > 14;
      const float up = usual ? __uint_as_float((uint32_t)(127 + 14 + 127 - e) << 23) : 1.0f;
      const float down = usual ? __uint_as_float((uint32_t)(e - 14) << 23) : 1.0f;
#pragma unroll
      for (int i = 0; i < 2; i++) qs[nb][i] *= __shfl_sync(0xffffffffu, down, (j2 + i) * 4);
#pragma unroll
      for (int ks = 0; ks < D / 16; ks++)
#pragma unroll
        for (int i = 0; i < 2; i++)
          q[ks][nb][i] = f16x2(bf16_lo(q[ks][nb][i]) * up, bf16_hi(q[ks][nb][i]) * up);
    }
  };

  // Rows g and g + 8 of the n-th block of O^T are the dims 16n + g and 16n + g + 8
  // (BF16), 16n + 2g and 16n + 2g + 1 (E4M3).
  auto end_row = [&](int b, bool whole, int side) {
#pragma unroll
    for (int nb = 0; nb < NB; nb++)
#pragma unroll
      for (int i = 0; i < 2; i++) {
        float sum = l[nb][i];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int row = 8 * nb + j2 + i;
        if (row >= n_rows) continue;
        if (whole) {
          const float inv = sum == 0.0f ? 0.0f : kv.v_scale / sum;
          uint16_t* out = args.a.out + ((int64_t)b * kv.Hq + head0 + row) * D;
#pragma unroll
          for (int n = 0; n < D / 16; n++) {
            const uint32_t y = bf16x2(o[n][nb][i] * inv, o[n][nb][2 + i] * inv);
            if (E4M3) {
              *reinterpret_cast<uint32_t*>(out + n * 16 + 2 * g) = y;
            } else {
              out[n * 16 + g] = (uint16_t)y;
              out[n * 16 + g + 8] = (uint16_t)(y >> 16);
            }
          }
          if (g == 0) {
            const float lse2 = sum == 0.0f ? kNegInf : m[nb][i] + log2f(sum);
            if (args.a.lse) args.a.lse[(int64_t)b * kv.Hq + head0 + row] = lse2 * 0.6931471805599453f;
            if (MASS) args.w.lse2[(int64_t)b * kv.Hq + head0 + row] = lse2;
          }
        } else {
          const int64_t at = ((int64_t)j * 2 + side) * (8 * NB) + row;
          if (g == 0) args.w.ml[at] = make_float2(m[nb][i], sum);
          float* po = args.w.o + at * D;
#pragma unroll
          for (int n = 0; n < D / 16; n++) {
            if (E4M3) {
              *reinterpret_cast<float2*>(po + n * 16 + 2 * g) = make_float2(o[n][nb][i], o[n][nb][2 + i]);
            } else {
              po[n * 16 + g] = o[n][nb][i];
              po[n * 16 + g + 8] = o[n][nb][2 + i];
            }
          }
        }
      }
  };

  // ldmatrix addresses: lanes 0-7, 8-15, 16-23 and 24-31 point at the rows of the four
  // 8 x 8 matrices, by halves of the entries first, or (values of a BF16 cache) of the
  // dims.  The swizzle flips the low bits of a 16-byte piece's number by the row's.
  constexpr uint32_t kFlip = R::kBox == 128 ? 7 : R::kBox == 64 ? 3 : 1, kFlipShift = R::kBox == 128 ? 0 : R::kBox == 64 ? 1 : 2;
  const uint32_t row_e = lane & 15, col_e = lane >> 4, row_d = (lane & 7) + ((lane >> 4) << 3), col_d = (lane >> 3) & 1;
  const uint32_t by_entry = row_e * R::kBox + ((col_e ^ ((row_e >> kFlipShift) & kFlip)) << 4);
  const uint32_t by_dim = row_d * R::kBox + ((col_d ^ ((row_d >> kFlipShift) & kFlip)) << 4);
  // pieces c (even) and c + 1 of the 16 entries from 16t on
  auto piece = [&](uint32_t base, int t, int c) {
    return (base ^ (uint32_t)((c % kBoxPieces) << 4)) + (uint32_t)((c / kBoxPieces) * R::kBoxBytes + t * 16 * R::kBox);
  };

  int stage = 0;
  uint32_t phase = 0;
  bool broken = false;
  bool fresh = true;  // a row begins with this tile
  begin_row(cons.b, cons.h);  // q is on its way before the tiles fill the memory's queues
#pragma unroll 1
  for (int s = 0; s < R::kStages - 1; s++) load(s);
#pragma unroll 1
  for (int at = lo; at < hi; at++) {
    if (E4M3 && fresh) encode_row();
    {
      const int ahead = stage + R::kStages - 1;
      load(ahead >= R::kStages ? ahead - R::kStages : ahead);
    }
    if (!wait_full(full + stage, phase)) {
      set_status(kv.status, kStTimeout);
      broken = true;
      break;
    }
    const uint32_t k_at = ring32 + stage * R::kStage, v_at = k_at + R::kSide;
    const uint32_t there = there_of[stage];
    if (there != kFull) {
      // Values that no sequence wrote could be NaN, which no weight of zero makes zero.
      uint8_t* const v_box = ring + stage * R::kStage + R::kSide + lane * 16;
#pragma unroll
      for (int i = 0; i < TILE * kPieces / 32; i++)  // pieces in the order in which they lie: by box, entry, piece
        if (!((there >> ((i * 32 + lane) / kBoxPieces % TILE)) & 1u)) *reinterpret_cast<uint4*>(v_box + i * 512) = make_uint4(0u, 0u, 0u, 0u);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before a copy comes here again
      __syncwarp();
    }

    // The steps of a score go to KC sums in turn: products that wait for one another are few.
    float part[KC][NT][NB][4];
#pragma unroll
    for (int c = 0; c < KC; c++)
#pragma unroll
      for (int t = 0; t < NT; t++)
#pragma unroll
        for (int nb = 0; nb < NB; nb++)
#pragma unroll
          for (int i = 0; i < 4; i++) part[c][t][nb][i] = 0.0f;
    if (!E4M3) {
#pragma unroll
      for (int ks = 0; ks < D / 16; ks++)
#pragma unroll
        for (int t = 0; t < NT; t++) {
          uint32_t a[4];
          ldsm4(a, k_at + piece(by_entry, t, 2 * ks));
#pragma unroll
          for (int nb = 0; nb < NB; nb++) mma<false>(part[ks % KC][t][nb], a, q[ks][nb]);
        }
    } else {
#pragma unroll
      for (int k2 = 0; k2 < D / 32; k2++)
#pragma unroll
        for (int t = 0; t < NT; t++) {
          uint32_t x[4];  // entries 0-7 and 8-15 of 16 dims, then of the next 16
          ldsm4(x, k_at + piece(by_entry, t, 2 * k2));
#pragma unroll
          for (int u = 0; u < 2; u++) {
            uint32_t a[4];
            e4m3x4_to_f16(x[2 * u], a[0], a[2]);
            e4m3x4_to_f16(x[2 * u + 1], a[1], a[3]);
#pragma unroll
            for (int nb = 0; nb < NB; nb++) mma<true>(part[(2 * k2 + u) % KC][t][nb], a, q[2 * k2 + u][nb]);
          }
        }
    }

    float s[NT][NB][4];
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
      for (int nb = 0; nb < NB; nb++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          s[t][nb][i] = part[0][t][nb][i];
#pragma unroll
          for (int c = 1; c < KC; c++) s[t][nb][i] += part[c][t][nb][i];
        }

    // softmax step.  s[t][nb][2e + i]: entry 16t + 8e + g, head 8nb + j2 + i.
    float top[NB][2];
    bool over = false;
#pragma unroll
    for (int nb = 0; nb < NB; nb++)
#pragma unroll
      for (int i = 0; i < 2; i++) {
        float x = kNegInf;
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
          for (int e = 0; e < 2; e++) {
            const bool gone = there != kFull && !((there >> (16 * t + 8 * e + g)) & 1u);
            s[t][nb][2 * e + i] = gone ? kNegInf : s[t][nb][2 * e + i] * qs[nb][i];
            x = fmaxf(x, s[t][nb][2 * e + i]);
          }
        top[nb][i] = x;
        over |= x - m[nb][i] > kSlack + (E4M3 ? kLift : 0.0f);  // the difference is exact where the two are near
      }
    if (MASS && at < args.w.tiles) {
      const int kept = NB == 2 ? 16 : score_rows(kv.G);  // of an entry
      float* sc = args.w.scores + ((gi * args.w.tiles + at) * TILE + g) * kept + j2;
#pragma unroll
      for (int t = 0; t < NT; t++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          float* const to = sc + (16 * t + 8 * e) * kept;
          if (NB == 1 && kept == 1) {
            if (j2 == 0) *to = s[t][0][2 * e];
            continue;
          }
          if (NB == 1 && j2 >= kept) continue;
#pragma unroll
          for (int nb = 0; nb < NB; nb++)
            *reinterpret_cast<float2*>(to + 8 * nb) = make_float2(s[t][nb][2 * e], s[t][nb][2 * e + 1]);
        }
    }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int nb = 0; nb < NB; nb++)
#pragma unroll
        for (int i = 0; i < 2; i++) {
          float x = top[nb][i];
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          x = fmaxf(E4M3 ? x - kLift : x, m[nb][i]);
          const float down = x == m[nb][i] ? 1.0f : exp2_fast(m[nb][i] - x);
          m[nb][i] = x;
          l[nb][i] *= down;
#pragma unroll
          for (int n = 0; n < D / 16; n++) {
            o[n][nb][i] *= down;
            o[n][nb][2 + i] *= down;
          }
        }
    }
    uint32_t hi_p[NT][NB][2], lo_p[NT][NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; nb++) {
      const float z0 = m[nb][0] == kNegInf ? 0.0f : m[nb][0];  // a row without a score yet: 2^(-inf) = 0
      const float z1 = m[nb][1] == kNegInf ? 0.0f : m[nb][1];
#pragma unroll
      for (int t = 0; t < NT; t++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          const float x = exp2_fast(s[t][nb][2 * e] - z0), y = exp2_fast(s[t][nb][2 * e + 1] - z1);
          l[nb][0] += x;
          l[nb][1] += y;
          // f16 keeps 11 bits of p, bf16 8: the rest goes through a second product
          if (E4M3) {
            const uint32_t u = f16x2(x, y);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
            hi_p[t][nb][e] = transposed(u);
            lo_p[t][nb][e] = transposed(f16x2(x - f.x, y - f.y));
          } else {
            const uint32_t u = bf16x2(x, y);
            hi_p[t][nb][e] = transposed(u);
            lo_p[t][nb][e] = transposed(bf16x2(x - bf16_lo(u), y - bf16_hi(u)));
          }
        }
    }

    if (!E4M3) {
#pragma unroll
      for (int n = 0; n < D / 16; n++)
#pragma unroll
        for (int t = 0; t < NT; t++) {
          uint32_t a[4];
          ldsm4t(a, v_at + piece(by_dim, t, 2 * n));
#pragma unroll
          for (int nb = 0; nb < NB; nb++) {
            mma<false>(o[n][nb], a, hi_p[t][nb]);
            mma<false>(o[n][nb], a, lo_p[t][nb]);
          }
        }
    } else {
#pragma unroll
      for (int n = 0; n < D / 32; n++)
#pragma unroll
        for (int t = 0; t < NT; t++) {
          uint32_t x[4];  // entries 0-7 and 8-15 of 16 dims, then of the next 16
          ldsm4t(x, v_at + piece(by_entry, t, 2 * n));
#pragma unroll
          for (int u = 0; u < 2; u++) {
            uint32_t a[4];
            e4m3x4_to_f16(__byte_perm(x[2 * u], 0, 0x3120), a[0], a[1]);
            e4m3x4_to_f16(__byte_perm(x[2 * u + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
            for (int nb = 0; nb < NB; nb++) {
              mma<true>(o[2 * n + u][nb], a, hi_p[t][nb]);
              mma<true>(o[2 * n + u][nb], a, lo_p[t][nb]);
            }
          }
        }
    }
    __syncwarp();  // the stage may be loaded again
    if (++stage == R::kStages) {
      stage = 0;
      phase ^= 1u;
    }

    const bool last = cons.t + 1 == cons.nt;
    if (last || at + 1 == hi) {
      end_row(cons.b, last && row_first >= lo, row_first >= lo ? 1 : 0);
      if (!last) {
        left.go_b = cons.b;
        left.go_h = cons.h;
        left.go_j0 = row_first / chunk;
        left.go_parts = (row_first + cons.nt - 1) / chunk - left.go_j0 + 1;
      }
      row_first += cons.nt;
      if (at + 1 < hi) {
        advance<TILE>(kv, cons);
        begin_row(cons.b, cons.h);
      }
      fresh = true;
    } else {
      cons.t++;
      fresh = false;
    }
  }
  if (broken) {  // the copies still under way land before the block leaves
    for (int i = 1; i < R::kStages; i++) {
      if (++stage == R::kStages) {
        stage = 0;
        phase ^= 1u;
      }
      wait_full(full + stage, phase);
    }
    left.tiles = 0;
    left.go_b = -1;
  }
  if (lane == 0) args.w.chunks[j] = left;
  idle_rows();
  if (MASS && lane == 0 && hi > args.w.tiles) set_status(kv.status, kStBadId);
}

// ---------------------------------------------------------------------------
// join: block j serves the row that goes on past the end of warp j's chunk, for that
// warp's group of heads.  The P parts of a row lie on the chunks j0 .. j0+P-1, so P - 1
// blocks of a group share it: a row in many parts has many blocks.  Part p lies on chunk
// j0 + p, side 1 (the row begins) for p = 0, else side 0.
//
// With MASS the blocks of a chunk, one for each group, then add the weights of its
// entries: 2^(score - lse) over the query heads of their KV head.  Every warp of both goes its own way: one
// trip to memory for what it joins.
// ---------------------------------------------------------------------------
struct JoinArgs {
  KvAttnArgs a;
  AttnWork w;
  int groups;
};

// Warps of a block of k_kv_join: 32 an SM in all, as many blocks as the split has warps.  Measured
// against half and double: 37 entries 6.4 us with 8 (4: 6.8, 16: 6.4), a weighed E4M3 batch 57.6
// with 4 (2: 65.0, 8: 61.3).
constexpr int join_warps(int row_bytes) { return 32 / warps_of(row_bytes); }

// What a sum with reference x counts for under the reference `both` >= x.
__device__ __forceinline__ float rescale(float x, float both) { return x == both ? 1.0f : exp2_fast(x - both); }

template <int D, int NB, int WARPS>
__device__ __forceinline__ void join_row(const JoinArgs& args, const Chunk& c) {
  const KvView& kv = args.a.kv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = NB == 1 ? 1 : args.groups;
  const int at = (int)blockIdx.x / groups, gi = (int)blockIdx.x - at * groups;
  const int n_rows = min(kRows, kv.G - gi * kRows);
  const int64_t head0 = (int64_t)c.go_b * kv.Hq + c.go_h * kv.G + gi * kRows;
  const int parts = c.go_parts, blocks = parts - 1, mine = at - c.go_j0;
  // Units of four dims of a row.  `split` lanes share a unit's parts while
  // there are more threads than units.
  const int units = n_rows * (D / 4), threads = blocks * WARPS * 32;
  int split = 1;
  while (split < 32 && split * 2 <= parts && units * split * 2 <= threads) split *= 2;
  const int width = 32 / split;
  // Warps by block, then by turn: the first blocks to start share an SM, and a row of few units in many
  // parts (100,000 E4M3 entries and one head of 128: 31 us, 17 so) would all be gathered by that one.
  for (int u0 = (warp * blocks + mine) * width; u0 < units; u0 += blocks * WARPS * width) {
    const int u = min(u0 + lane % width, units - 1), row = u / (D / 4), d4 = u - row * (D / 4);
    float top = kNegInf, sum = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](float m, float l, float4 x) {
      const float both = fmaxf(top, m), a = rescale(top, both), b = rescale(m, both);
      top = both;
      sum = sum * a + l * b;
      acc.x = acc.x * a + x.x * b;
      acc.y = acc.y * a + x.y * b;
      acc.z = acc.z * a + x.z * b;
      acc.w = acc.w * a + x.w * b;
    };
#pragma unroll 8
    for (int p = lane / width; p < parts; p += split) {
      const int64_t at = (((int64_t)(c.go_j0 + p) * groups + gi) * 2 + (p == 0 ? 1 : 0)) * (8 * NB) + row;
      const float2 ml = args.w.ml[at];
      add(ml.x, ml.y, *reinterpret_cast<const float4*>(args.w.o + at * D + d4 * 4));
    }
    for (int d = width; d < 32; d <<= 1) {
      const float m = __shfl_xor_sync(0xffffffffu, top, d), l = __shfl_xor_sync(0xffffffffu, sum, d);
      const float4 x = make_float4(__shfl_xor_sync(0xffffffffu, acc.x, d), __shfl_xor_sync(0xffffffffu, acc.y, d),
                                   __shfl_xor_sync(0xffffffffu, acc.z, d), __shfl_xor_sync(0xffffffffu, acc.w, d));
      add(m, l, x);
    }
    if (lane >= width || u0 + lane >= units) continue;
    const float inv = sum == 0.0f ? 0.0f : kv.v_scale / sum;
    *reinterpret_cast<uint2*>(args.a.out + (head0 + row) * D + d4 * 4) =
        make_uint2(bf16x2(acc.x * inv, acc.y * inv), bf16x2(acc.z * inv, acc.w * inv));
    if (d4 == 0 && args.a.lse)
      args.a.lse[head0 + row] = sum == 0.0f ? kNegInf : (top + log2f(sum)) * 0.6931471805599453f;
  }
}

// A row in more parts than this has its lse found by the block together, not by each warp for itself:
// 100,000 E4M3 entries and 16 heads of 128 35 us, 78 by warps alone; 11 ragged rows of up to 14,000
// entries, 48 heads over two of 256 48.4 (from 32 parts on 49.8, from 64 on 54.8).  Few parts cost less by warps (13 rows
// of up to 171 entries 18.4 us so, 19.6 with the block's way in the kernel at all).
constexpr int kManyParts = 16;
constexpr int kMaxGroups = 64;  // n_heads / n_kv_heads is at most 1024

template <int V>
struct Floats;
template <>
struct Floats<1> {
  using type = float;
};
template <>
struct Floats<2> {
  using type = float2;
};
template <>
struct Floats<4> {
  using type = float4;
};

// The warp's share of a chunk's tiles, cut over the warps of all blocks of the chunk.  L lanes
// hold an entry's KEPT scores, V query heads each; 32 / L entries go at a time, and after L
// of them each lane has the sum of one entry.
template <int TILE, int KEPT, int WARPS>
__device__ __forceinline__ void add_mass(const JoinArgs& args, const Chunk& c) {
  constexpr int ROWS = KEPT == 16 ? 16 : 8, V = KEPT < 4 ? KEPT : 4, L = KEPT / V, E = 32 / L;
  constexpr int RUNS = L == 1 ? 4 : 2;  // of 32 entries, their loads in flight together
  using Vec = typename Floats<V>::type;
  union Scores {
    Vec vec;
    float v[V];
  };
  const KvView& kv = args.a.kv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % L, set = lane / L;
  const int groups = KEPT < 16 ? 1 : args.groups;
  const int here = (int)blockIdx.x / groups, turn = ((int)blockIdx.x - here * groups) * WARPS + warp;
  const int share = (c.tiles + WARPS * groups - 1) / (WARPS * groups);
  const int chunk0 = here * c.size, lo = chunk0 + min(c.tiles, turn * share), hi = min(chunk0 + c.tiles, lo + share);

  // m and l of the lane's heads over the parts q, q + step, ... of a row, and over all lanes with these heads.
  auto sum_parts = [&](int j0, int parts, int gi, int q, int step, float2 (&ml)[V]) {
    auto part = [&](int q, float2 (&ml)[V]) {
      const float2* at = args.w.ml + (((int64_t)(j0 + q) * groups + gi) * 2 + (q == 0 ? 1 : 0)) * ROWS + sub * V;
      if constexpr (V == 4) {
        const float4 u = reinterpret_cast<const float4*>(at)[0], v = reinterpret_cast<const float4*>(at)[1];
        ml[0] = make_float2(u.x, u.y), ml[1] = make_float2(u.z, u.w);
        ml[2] = make_float2(v.x, v.y), ml[3] = make_float2(v.z, v.w);
      } else {
#pragma unroll
        for (int i = 0; i < V; i++) ml[i] = at[i];
      }
    };
    part(min(q, parts - 1), ml);
    if (q >= parts) {
#pragma unroll
      for (int i = 0; i < V; i++) ml[i].y = 0.0f;
    }
    for (q += step; q < parts; q += step) {
      float2 y[V];
      part(q, y);
#pragma unroll
      for (int i = 0; i < V; i++) {
        const float both = fmaxf(ml[i].x, y[i].x);
        ml[i].y = ml[i].y * rescale(ml[i].x, both) + y[i].y * rescale(y[i].x, both);
        ml[i].x = both;
      }
    }
#pragma unroll
    for (int i = 0; i < V; i++) {
      float top = ml[i].x;
#pragma unroll
      for (int d = L; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      float sum = ml[i].y * rescale(ml[i].x, top);
#pragma unroll
      for (int d = L; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      ml[i] = make_float2(top, sum);
    }
  };
  // Rows in many parts: the block's warps share them.  They can only be the chunk's first row and the one that goes on.
  __shared__ float2 s_part[WARPS][ROWS];
  __shared__ float s_lse[2][KEPT < 16 ? 1 : kMaxGroups][ROWS];
  const int first_j0 = c.first / c.size, first_nt = tiles_of<TILE>(c.len);
  const int first_parts = (c.first + first_nt - 1) / c.size - first_j0 + 1;
  const bool other = c.go_b >= 0 && c.first + first_nt <= chunk0 + c.tiles;  // the row that goes on is not the first
  for (int side = 0; side < 2; side++) {
    const int j0 = side ? c.go_j0 : first_j0, parts = side ? (other ? c.go_parts : 0) : first_parts;
    for (int gi = 0; parts > kManyParts && gi < groups; gi++) {
      float2 ml[V];
      sum_parts(j0, parts, gi, warp * E + set, WARPS * E, ml);
      if (set == 0) {
#pragma unroll
        for (int i = 0; i < V; i++) s_part[warp][sub * V + i] = ml[i];
      }
      __syncthreads();
      if (threadIdx.x < KEPT) {
        float top = kNegInf, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; w++) top = fmaxf(top, s_part[w][threadIdx.x].x);
#pragma unroll
        for (int w = 0; w < WARPS; w++) sum += s_part[w][threadIdx.x].y * rescale(s_part[w][threadIdx.x].x, top);
        const bool real = threadIdx.x < kv.G - gi * kRows;
        s_lse[side][gi][threadIdx.x] = real && sum != 0.0f ? top + __log2f(sum) : kNegInf;
      }
      __syncthreads();
    }
  }

  if (lo >= hi) return;
  Place p{c.b, c.h, 0, c.len, tiles_of<TILE>(c.len)};
  for (int first = c.first; first < hi;) {
    const int j0 = first / c.size, parts = (first + p.nt - 1) / c.size - j0 + 1;
    const int e0 = (max(lo, first) - first) * TILE, e1 = min((min(hi, first + p.nt) - first) * TILE, p.len);
    const int last = (int)min((int64_t)e1, (args.w.tiles - first) * TILE);  // entries whose scores were kept
    for (int gi = 0; first + p.nt > lo && gi < groups; gi++) {
      const int n_rows = min(kRows, kv.G - gi * kRows);
      const float* const scores = args.w.scores + (gi * args.w.tiles + first) * TILE * KEPT + sub * V;
      Scores x[RUNS][L];
      int row[RUNS];
      auto load = [&](int e) {  // the lane keeps the sum of entry sub * E + set of each run
#pragma unroll
        for (int r = 0; r < RUNS; r++)
#pragma unroll
          for (int k = 0; k < L; k++) {
            const int at = e + 32 * r + k * E + set;
#pragma unroll
            for (int i = 0; i < V; i++) x[r][k].v[i] = kNegInf;
            if (at < last) x[r][k].vec = *reinterpret_cast<const Vec*>(scores + (int64_t)at * KEPT);
          }
#pragma unroll
        for (int r = 0; r < RUNS; r++) {
          const int own = e + 32 * r + sub * E + set;
          row[r] = own < last ? kv_row(kv, p.b, p.h, own) : -1;
        }
      };
      if (e0 < last) load(e0);
      float z[V];  // lse of the lane's heads; +inf takes a head (without weights, or none) out
      if (parts == 1) {
#pragma unroll
        for (int i = 0; i < V; i++)
          z[i] = sub * V + i < n_rows ? args.w.lse2[(int64_t)p.b * kv.Hq + p.h * kv.G + gi * kRows + sub * V + i] : kNegInf;
      } else if (parts > kManyParts) {
#pragma unroll
        for (int i = 0; i < V; i++) z[i] = s_lse[first == c.first ? 0 : 1][gi][sub * V + i];
      } else {
        float2 ml[V];
        sum_parts(j0, parts, gi, set, E, ml);
#pragma unroll
        for (int i = 0; i < V; i++) z[i] = sub * V + i < n_rows && ml[i].y != 0.0f ? ml[i].x + __log2f(ml[i].y) : kNegInf;
      }
#pragma unroll
      for (int i = 0; i < V; i++)
        if (z[i] == kNegInf) z[i] = -kNegInf;
#pragma unroll 1
      for (int e = e0; e < last;) {
        float old[RUNS];
#pragma unroll
        for (int r = 0; r < RUNS; r++) old[r] = row[r] >= 0 ? kv.mass[row[r]] : 0.0f;
#pragma unroll
        for (int r = 0; r < RUNS; r++) {
          float mine = 0.0f;
#pragma unroll
          for (int k = 0; k < L; k++) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; i++) sum += exp2_fast(x[r][k].v[i] - z[i]);
#pragma unroll
            for (int d = 1; d < L; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            if (sub == k) mine = sum;
          }
          if (row[r] >= 0) kv.mass[row[r]] = old[r] + mine;
        }
        e += 32 * RUNS;
        if (e < last) load(e);
      }
    }
    first += p.nt;
    if (first < hi) {
      p.t = p.nt - 1;
      advance<TILE>(kv, p);
    }
  }
}

// KEPT: scores of an entry (0: without FT_KV_MASS).
template <int D, int TILE, int NB, int KEPT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 32 / WARPS) k_kv_join(JoinArgs args) {
  kv_pdl_trigger();
  kv_pdl_wait();
  const Chunk c = args.w.chunks[blockIdx.x];
  if (c.go_b >= 0) join_row<D, NB, WARPS>(args, c);
  if constexpr (KEPT > 0) {
    if (c.tiles > 0) add_mass<TILE, KEPT, WARPS>(args, c);
  }
}

template <int D, bool E4M3, int NB, bool MASS>
cudaError_t run(SplitArgs& a, int device, int sms, cudaStream_t s) {
  using R = Ring<D * (E4M3 ? 1 : 2)>;
  static_assert(R::kStages >= 2, "a ring of at least two stages fits");
  const KvView& kv = a.a.kv;
  const uint64_t rows = (uint64_t)kv.n_pages * kv.Hkv << kv.page_shift;
  a.box_shift = R::kTile == 32 ? 5 : 4;
  if (kv.page_shift < a.box_shift) a.box_shift = kv.page_shift;
  a.per_part = part_share(kv.n_seqs, kv.Hkv);
  const uint32_t deep = (1 << a.box_shift) == R::kTile ? R::kBoxes : 1;
  if (encode_tmap_rows(&a.k_map, kv.k, D * (E4M3 ? 1 : 2), rows, R::kBox, 1u << a.box_shift, deep) != FT_OK ||
      encode_tmap_rows(&a.v_map, kv.v, D * (E4M3 ? 1 : 2), rows, R::kBox, 1u << a.box_shift, deep) != FT_OK)
    return cudaErrorInvalidValue;
  auto kern = k_kv_split<D, E4M3, NB, MASS>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = kv_attribute_once(done, device, kern, cudaFuncAttributeMaxDynamicSharedMemorySize, R::kBytes);
  if (e != cudaSuccess) return e;
  if ((e = kv_launch_after(kern, dim3((unsigned)sms), R::kWarps * 32, R::kBytes, s, a)) != cudaSuccess) return e;
  const JoinArgs ja{a.a, a.w, a.groups};
  constexpr int JW = join_warps(D * (E4M3 ? 1 : 2)), T = R::kTile;
  const dim3 chunks((unsigned)(sms * R::kWarps));
  auto join = [&](void (*kern)(const JoinArgs)) { return kv_launch_after(kern, chunks, JW * 32, 0, s, ja); };
  if constexpr (!MASS) return join(k_kv_join<D, T, NB, 0, JW>);
  else if constexpr (NB == 2) return join(k_kv_join<D, T, 2, 16, JW>);
  else
    switch (score_rows(kv.G)) {
      case 1: return join(k_kv_join<D, T, 1, 1, JW>);
      case 2: return join(k_kv_join<D, T, 1, 2, JW>);
      case 4: return join(k_kv_join<D, T, 1, 4, JW>);
      default: return join(k_kv_join<D, T, 1, 8, JW>);
    }
}

template <int D, bool E4M3>
cudaError_t run_d(SplitArgs& a, int device, int sms, cudaStream_t s) {
  if (a.a.kv.G > 8) return a.a.mass ? run<D, E4M3, 2, true>(a, device, sms, s) : run<D, E4M3, 2, false>(a, device, sms, s);
  return a.a.mass ? run<D, E4M3, 1, true>(a, device, sms, s) : run<D, E4M3, 1, false>(a, device, sms, s);
}

}  // namespace

cudaError_t launch_kv_wait(int blocks, uint64_t limit_ns, int64_t arrive_ns, int32_t* lanes, cudaStream_t s) {
  k_kv_wait<<<blocks, 64, 0, s>>>(limit_ns, arrive_ns, lanes);
  return cudaGetLastError();
}

void kv_geometry(const ft_kv_cache& c, int total, int sms, int64_t out[4]) {
  const int row_bytes = c.head_dim * (c.format == FT_KV_E4M3 ? 1 : 2);
  const int chunks = (sms < kKvMaxSms ? sms : kKvMaxSms) * warps_of(row_bytes) / groups_of(c.n_heads / c.n_kv_heads);
  out[0] = tile_of(row_bytes);
  out[1] = chunk_tiles(total, chunks, part_share(c.n_seqs, c.n_kv_heads));
  out[2] = (total + out[1] - 1) / out[1];
  out[3] = chunks;
}

int64_t kv_attn_workspace(const ft_kv_cache& c) {
  AttnWork w;
  return carve(w, nullptr, c.head_dim, c.head_dim * (c.format == FT_KV_E4M3 ? 1 : 2), c.n_seqs, c.n_heads, c.n_kv_heads,
               c.n_pages * c.n_kv_heads * c.page_size, c.mass != nullptr);
}

cudaError_t launch_kv_attention(const KvAttnArgs& args, bool e4m3, int device, int sms, cudaStream_t s) {
  SplitArgs a;
  a.a = args;
  a.groups = groups_of(args.kv.G);
  const KvView& kv = args.kv;
  carve(a.w, args.work, kv.D, kv.D * (e4m3 ? 1 : 2), kv.n_seqs, kv.Hq, kv.Hkv,
        (int64_t)kv.n_pages * kv.Hkv << kv.page_shift, args.mass);
  sms = sms < kKvMaxSms ? sms : kKvMaxSms;
  switch (kv.D) {
    case 64: return e4m3 ? run_d<64, true>(a, device, sms, s) : run_d<64, false>(a, device, sms, s);
    case 96: return e4m3 ? run_d<96, true>(a, device, sms, s) : run_d<96, false>(a, device, sms, s);
    case 128: return e4m3 ? run_d<128, true>(a, device, sms, s) : run_d<128, false>(a, device, sms, s);
    case 192: return e4m3 ? run_d<192, true>(a, device, sms, s) : run_d<192, false>(a, device, sms, s);
    default: return e4m3 ? run_d<256, true>(a, device, sms, s) : run_d<256, false>(a, device, sms, s);
  }
}

}  // namespace ft
