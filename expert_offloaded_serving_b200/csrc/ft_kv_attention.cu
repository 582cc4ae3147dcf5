// ft_kv_attention: attention of one new token a sequence over its paged
// entries, split over the entries of the whole batch and joined.
//
// Mathematics: one pass over the entries with the running maximum m and sum l
// of a softmax.  For a tile of entries, with s = q.k in units of log2(e):
//   m' = max(m, max s), p = 2^(s - m'), l' = l 2^(m - m') + sum p,
//   O' = O 2^(m - m') + p V;  at the end out = O / l, lse = ln 2 (m + log2 l).
// Two parts of one row join the same way: weights 2^(m_i - max m).
//
// What bounds it: every cached byte is read once and meets G query heads,
// 4 G flops for 4 bytes of a BF16 entry.  At the measured copy rate an SM gets
// 22 bytes a clock, so 16 heads are 90 multiply-adds a clock an SM: far below what
// mma.sync does, a multiple of what the fp32 pipe could do next to the softmax.
// So the products run on mma.sync with the heads of one KV head as the 16
// rows of the tile (idle rows cost nothing that is short), and everything
// else serves the stream of loads.
//
// Split: the unit is a tile of 16 entries of one (sequence, KV head, group of
// 16 query heads).  All tiles of the batch, in that order, are cut into
// equal contiguous chunks, one a warp; a warp streams its chunk through its own
// ring of cp.async stages in shared memory and meets no barrier with other
// warps.  A row (the tiles of one item) that lies inside one chunk is
// finished there; the parts of the others go to the workspace (fp32) and
// k_kv_join adds them in the order of the chunks.  Lengths are read on the
// device: ragged batches and idle rows are balanced by construction, a
// captured graph stays valid when lengths grow, and the split depends on
// nothing but the lengths and the number of SMs.
//
// With FT_KV_MASS the scores go to the workspace as they come (G fp32 values
// an entry, next to 4 D bytes of it), and k_kv_mass turns them into weights
// once the row's lse is known.
#include "ft_kv.cuh"

namespace ft {

namespace {

constexpr int kTile = 16;        // entries of a tile
constexpr int kRows = 16;        // query heads of an item: rows of the mma tile
constexpr int kMaxWarps = 8;     // warps of a block at most
constexpr int kMaxChunks = kKvMaxSms * kMaxWarps;
constexpr int kRingBytes = 212 * 1024;  // shared memory of a block's rings at most

// The ring of a warp for entries of RB bytes a side: a stage holds 16 keys and 16
// values, rows 16 bytes apart from a multiple of 128 (ldmatrix then reads 8 rows
// from 8 different groups of banks), and the 16 row numbers.
template <int RB>
struct Ring {
  static constexpr int kStride = RB + 16;
  static constexpr int kSide = kTile * kStride;
  static constexpr int kStage = 2 * kSide + kTile * 4;
  static constexpr int kWarps = 2 * kSide > 12000 ? 4 : 8;
  static constexpr int kFit = kRingBytes / (kWarps * kStage);
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static constexpr int kBytes = kWarps * kStages * kStage;
};

// What k_kv_split leaves for the kernels behind it.
struct Going {  // the row that goes on past the end of a chunk
  int b, hh;      // sequence (-1: none) and item of it
  int j0, parts;  // the chunk it begins on, the chunks it lies on
};
struct AttnWork {
  Going* going;      // [chunks]
  int4* start;       // [chunks] where the chunk begins: sequence (-1: empty chunk), item, tile of the item, tiles of the chunk
  float2* ml;        // [chunks][2][16] m and l of a part (log2 units); part 0: a row that came in, 1: one that goes on
  float* o;          // [chunks][2][16][D]
  float* lse2;       // [n_seqs][Hq] lse in log2 units (mass)
  float* scores;     // [rows / page][G][page] scores in log2 units (mass)
};

__host__ __device__ inline int64_t up256(int64_t n) { return (n + 255) & ~(int64_t)255; }

__host__ __device__ inline int64_t carve(AttnWork& w, uint8_t* base, int D, int n_seqs, int Hq, int64_t rows, int G) {
  int64_t at = 0;
  w.going = reinterpret_cast<Going*>(base + at);
  at += up256((int64_t)kMaxChunks * sizeof(Going));
  w.start = reinterpret_cast<int4*>(base + at);
  at += up256((int64_t)kMaxChunks * sizeof(int4));
  w.ml = reinterpret_cast<float2*>(base + at);
  at += up256((int64_t)kMaxChunks * 2 * kRows * sizeof(float2));
  w.o = reinterpret_cast<float*>(base + at);
  at += up256((int64_t)kMaxChunks * 2 * kRows * D * sizeof(float));
  w.lse2 = reinterpret_cast<float*>(base + at);
  at += up256((int64_t)n_seqs * Hq * sizeof(float));
  w.scores = reinterpret_cast<float*>(base + at);
  at += up256(rows * G * (int64_t)sizeof(float));
  return at;
}

struct SplitArgs {
  KvAttnArgs a;
  AttnWork w;
  int groups;  // items of a KV head: groups of 16 query heads
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
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
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two E4M3 bytes (low half of v) as f16x2, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  uint32_t h;
  asm("{ .reg .b16 b; cvt.u16.u32 b, %1; cvt.rn.f16x2.e4m3x2 %0, b; }" : "=r"(h) : "r"(v));
  return h;
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

// A place in the batch's order of tiles: sequence, item of the sequence, tile of the item.
struct Place {
  int b, hh, t, len, nt;
};

__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

__device__ __forceinline__ void next_sequence(const KvView& kv, Place& p) {
  do {
    p.b++;
    p.len = p.b < kv.n_seqs ? kv_length(kv, p.b) : 1;
  } while (p.len == 0);
  p.nt = tiles_of(p.len);
}

__device__ __forceinline__ void advance(const KvView& kv, Place& p, int items) {
  if (++p.t < p.nt) return;
  p.t = 0;
  if (++p.hh < items) return;
  p.hh = 0;
  next_sequence(kv, p);
}

constexpr float kNegInf = -__builtin_huge_valf();

// D: head_dim.  E4M3: the cache's format.  WIDE: more than 8 query heads in an
// item (else rows 8 to 15 of the tile are idle and their registers are not kept).
// MASS: scores go to the workspace.
template <int D, bool E4M3, bool WIDE, bool MASS>
__global__ void __launch_bounds__(Ring<D * (E4M3 ? 1 : 2)>::kWarps * 32, 1) k_kv_split(SplitArgs args) {
  constexpr int RB = D * (E4M3 ? 1 : 2);
  using R = Ring<RB>;
  constexpr int kThreads = R::kWarps * 32;
  constexpr int kChunksRow = RB / 16;                  // 16-byte pieces of a row
  constexpr int kCopies = kTile * kChunksRow / 32;     // cp.async a lane and side
  constexpr int NR = WIDE ? 2 : 1;                     // rows of the tile a lane keeps
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_sum[kThreads + 1];

  const KvView& kv = args.a.kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int items = kv.Hkv * args.groups;

  kv_pdl_trigger();
  // Tiles of the batch and where each thread's share of the sequences begins.
  const int per = (kv.n_seqs + kThreads - 1) / kThreads;
  {
    int sum = 0;
    for (int i = 0; i < per; i++) {
      const int b = tid * per + i;
      if (b < kv.n_seqs) sum += tiles_of(kv_length(kv, b, blockIdx.x == 0)) * items;
    }
    int run = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, run, d);
      if (lane >= d) run += x;
    }
    __shared__ int s_warp[R::kWarps];
    if (lane == 31) s_warp[warp] = run;
    __syncthreads();
    for (int w = 0; w < warp; w++) run += s_warp[w];
    s_sum[tid + 1] = run;
    if (tid == 0) s_sum[0] = 0;
    __syncthreads();
  }
  // Idle rows: out 0, lse -inf.
  for (int b = blockIdx.x; b < kv.n_seqs; b += gridDim.x) {
    if (kv_length(kv, b) != 0) continue;
    uint32_t* o = reinterpret_cast<uint32_t*>(args.a.out + (int64_t)b * kv.Hq * D);
    for (int i = tid; i < kv.Hq * D / 2; i += kThreads) o[i] = 0u;
    if (args.a.lse)
      for (int i = tid; i < kv.Hq; i += kThreads) args.a.lse[(int64_t)b * kv.Hq + i] = kNegInf;
  }

  const int total = s_sum[kThreads];
  const int chunk = max(1, (total + (int)gridDim.x * R::kWarps - 1) / ((int)gridDim.x * R::kWarps));
  const int j = warp * gridDim.x + blockIdx.x;  // neighbours in the batch sit on different SMs
  const int lo = (int)min((int64_t)j * chunk, (int64_t)total), hi = min(lo + chunk, total);
  if (lo >= hi) {
    if (lane == 0) {
      args.w.going[j] = Going{-1, 0, 0, 0};
      if (MASS) args.w.start[j] = make_int4(-1, 0, 0, 0);
    }
    return;
  }

  // The place of tile `lo`: the thread share that holds it, then its sequences.
  Place cons;
  int base;  // first tile of sequence cons.b
  {
    int l = 0, h = kThreads;  // s_sum[l] <= lo < s_sum[h]
    while (h - l > 1) {
      const int m = (l + h) >> 1;
      if (s_sum[m] <= lo) l = m;
      else h = m;
    }
    base = s_sum[l];
    cons.b = l * per;
    for (;; cons.b++) {
      cons.len = kv_length(kv, cons.b);
      cons.nt = tiles_of(cons.len);
      if (lo < base + cons.nt * items) break;
      base += cons.nt * items;
    }
    cons.hh = (lo - base) / cons.nt;
    cons.t = (lo - base) - cons.hh * cons.nt;
  }
  if (MASS && lane == 0) args.w.start[j] = make_int4(cons.b, cons.hh, cons.t, hi - lo);

  uint8_t* const ring = smem + warp * (R::kStages * R::kStage);
  const uint32_t ring32 = smem_u32(ring);

  // ---- producer: rows of a tile, then their copies ----
  Place prod = cons;
  auto tile_row = [&](const Place& p) {  // lanes 0..15: row of entry lane of the tile, -1 past the end
    const int slot = p.t * kTile + (lane & 15);
    return slot < p.len && p.b < kv.n_seqs ? kv_row(kv, p.b, p.hh / args.groups, slot) : -1;
  };
  int row_next = tile_row(prod);
  int to_load = hi - lo;
  auto load = [&](int stage) {
    if (to_load > 0) {
      to_load--;
      const int row = row_next;
      if (to_load > 0) {
        advance(kv, prod, items);
        row_next = tile_row(prod);
      }
      const uint32_t k_at = ring32 + stage * R::kStage, v_at = k_at + R::kSide;
      if (lane < kTile) *reinterpret_cast<int*>(ring + stage * R::kStage + 2 * R::kSide + lane * 4) = row;
#pragma unroll
      for (int i = 0; i < kCopies; i++) {
        const int c = i * 32 + lane, r = c / kChunksRow, col = c - r * kChunksRow;
        const int from = __shfl_sync(0xffffffffu, row, r);
        const bool real = from >= 0;
        const int64_t off = (int64_t)(real ? from : 0) * RB + col * 16;
        cp16(k_at + r * R::kStride + col * 16, kv.k + off, real);
        cp16(v_at + r * R::kStride + col * 16, kv.v + off, real);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < R::kStages - 1; s++) load(s);

  // ---- consumer ----
  const int g = lane >> 2, j2 = (lane & 3) * 2;  // the mma layout's row and first column
  uint32_t qf[D / 16][4];
  float o[D / 8][4];
  float m[NR], l[NR], qs[NR];
  int n_rows = 0, head0 = 0;

  auto begin_row = [&](int b, int hh) {
    const int h = hh / args.groups, gi = hh - h * args.groups;
    head0 = h * kv.G + gi * kRows;
    n_rows = min(kRows, kv.G - gi * kRows);
    const float unit = args.a.scale * 1.4426950408889634f * kv.k_scale;
#pragma unroll
    for (int r = 0; r < 2; r++) {
      if (r >= NR) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ks++) qf[ks][1] = qf[ks][3] = 0u;
        continue;
      }
      const bool real = g + 8 * r < n_rows;
      const uint16_t* q = args.a.q + (int64_t)b * args.a.q_stride + (int64_t)(head0 + (real ? g + 8 * r : 0)) * D;
      m[r] = kNegInf;
      l[r] = 0.0f;
      qs[r] = unit;
      if (!E4M3) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ks++) {
          qf[ks][r] = real ? *reinterpret_cast<const uint32_t*>(q + ks * 16 + j2) : 0u;
          qf[ks][2 + r] = real ? *reinterpret_cast<const uint32_t*>(q + ks * 16 + 8 + j2) : 0u;
        }
      } else {
        // The 16 contraction steps of an mma take the dims 4i, 4i+1 (first half)
        // and 4i+2, 4i+3 (second half) of each lane i of a quad: the order in which
        // ldmatrix hands out the bytes of a key.  q joins them as f16 with a
        // power-of-two factor that puts the head's largest magnitude into
        // [2^14, 2^15): exact for bf16 values down to 2^-28 of it.
        uint2 raw[D / 16];
        float top = 0.0f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ks++) {
          raw[ks] = real ? *reinterpret_cast<const uint2*>(q + ks * 16 + 2 * j2) : make_uint2(0u, 0u);
          top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16_lo(raw[ks].x)), fabsf(bf16_hi(raw[ks].x))),
                                 fmaxf(fabsf(bf16_lo(raw[ks].y)), fabsf(bf16_hi(raw[ks].y)))));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = (int)(__float_as_uint(top) >> 23);  // biased exponent; 0 and 255: as it is
        const bool usual = e > 14 && e < 255;
        const float up = usual ? __uint_as_float((uint32_t)(127 + 14 + 127 - e) << 23) : 1.0f;
        qs[r] = usual ? unit * __uint_as_float((uint32_t)(e - 14) << 23) : unit;
#pragma unroll
        for (int ks = 0; ks < D / 16; ks++) {
          qf[ks][r] = f16x2(bf16_lo(raw[ks].x) * up, bf16_hi(raw[ks].x) * up);
          qf[ks][2 + r] = f16x2(bf16_lo(raw[ks].y) * up, bf16_hi(raw[ks].y) * up);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < D / 8; n++)
#pragma unroll
      for (int i = 0; i < 4; i++) o[n][i] = 0.0f;
  };

  // Element (row r of the lane, n-tile, side) of O sits at these dims: BF16
  // n-tile n covers dims 8n .. 8n+7; E4M3 n-tiles 2c and 2c+1 cover the even
  // and odd dims of the 16 from 16c on.
  auto end_row = [&](int b, bool whole, int part) {
#pragma unroll
    for (int r = 0; r < NR; r++) {
      float sum = l[r];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const int row = g + 8 * r;
      if (row >= n_rows) continue;
      if (whole) {
        const float inv = sum == 0.0f ? 0.0f : kv.v_scale / sum;
        uint16_t* out = args.a.out + ((int64_t)b * kv.Hq + head0 + row) * D;
        if (!E4M3) {
#pragma unroll
          for (int n = 0; n < D / 8; n++)
            *reinterpret_cast<uint32_t*>(out + n * 8 + j2) = bf16x2(o[n][2 * r] * inv, o[n][2 * r + 1] * inv);
        } else {
#pragma unroll
          for (int c = 0; c < D / 16; c++)
            *reinterpret_cast<uint2*>(out + c * 16 + 2 * j2) =
                make_uint2(bf16x2(o[2 * c][2 * r] * inv, o[2 * c + 1][2 * r] * inv),
                           bf16x2(o[2 * c][2 * r + 1] * inv, o[2 * c + 1][2 * r + 1] * inv));
        }
        if ((lane & 3) == 0) {
          const float lse2 = sum == 0.0f ? kNegInf : m[r] + log2f(sum);
          if (args.a.lse) args.a.lse[(int64_t)b * kv.Hq + head0 + row] = lse2 * 0.6931471805599453f;
          if (MASS) args.w.lse2[(int64_t)b * kv.Hq + head0 + row] = lse2;
        }
      } else {
        const int64_t at = ((int64_t)j * 2 + part) * kRows + row;
        if ((lane & 3) == 0) args.w.ml[at] = make_float2(m[r], sum);
        float* po = args.w.o + at * D;
        if (!E4M3) {
#pragma unroll
          for (int n = 0; n < D / 8; n++)
            *reinterpret_cast<float2*>(po + n * 8 + j2) = make_float2(o[n][2 * r], o[n][2 * r + 1]);
        } else {
#pragma unroll
          for (int c = 0; c < D / 16; c++)
            *reinterpret_cast<float4*>(po + c * 16 + 2 * j2) =
                make_float4(o[2 * c][2 * r], o[2 * c + 1][2 * r], o[2 * c][2 * r + 1], o[2 * c + 1][2 * r + 1]);
        }
      }
    }
  };

  const uint32_t k_lane = E4M3 ? (lane & 15) * R::kStride + (lane >> 4) * 16
                               : ((lane & 7) + ((lane >> 4) << 3)) * R::kStride + ((lane >> 3) & 1) * 16;
  const uint32_t v_lane = (lane & 15) * R::kStride + (lane >> 4) * 16;

  begin_row(cons.b, cons.hh);
  int row_first = base + cons.hh * cons.nt;  // first tile of the row in the batch's order
  Going going{-1, 0, 0, 0};
  int stage = 0;
  for (int at = lo; at < hi; at++) {
    {
      const int ahead = stage + R::kStages - 1;
      load(ahead >= R::kStages ? ahead - R::kStages : ahead);
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(R::kStages - 1) : "memory");
    __syncwarp();
    const uint32_t k_at = ring32 + stage * R::kStage, v_at = k_at + R::kSide;
    const int* rows = reinterpret_cast<const int*>(ring + stage * R::kStage + 2 * R::kSide);
    const int2 ra = *reinterpret_cast<const int2*>(rows + j2), rb = *reinterpret_cast<const int2*>(rows + 8 + j2);
    const int row_of[4] = {ra.x, ra.y, rb.x, rb.y};  // entries j2, j2+1, 8+j2, 9+j2 of the tile

    float s[2][4] = {};
    if (!E4M3) {
#pragma unroll
      for (int ks = 0; ks < D / 16; ks++) {
        uint32_t b[4];
        ldsm4(b, k_at + k_lane + ks * 32);
        mma<false>(s[0], qf[ks], b[0], b[1]);
        mma<false>(s[1], qf[ks], b[2], b[3]);
      }
    } else {
#pragma unroll
      for (int k2 = 0; k2 < D / 32; k2++) {
        uint32_t b[4];  // entries 0-7 and 8-15 of 16 dims, then of the next 16
        ldsm4(b, k_at + k_lane + k2 * 32);
#pragma unroll
        for (int u = 0; u < 2; u++) {
          mma<true>(s[0], qf[2 * k2 + u], e4m3x2_to_f16x2(b[2 * u]), e4m3x2_to_f16x2(b[2 * u] >> 16));
          mma<true>(s[1], qf[2 * k2 + u], e4m3x2_to_f16x2(b[2 * u + 1]), e4m3x2_to_f16x2(b[2 * u + 1] >> 16));
        }
      }
    }

    // softmax step; lane rows g (and g + 8), four entries each
    float p[NR][4];
    bool moved = false;
    float m_new[NR];
#pragma unroll
    for (int r = 0; r < NR; r++) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const float x = s[i >> 1][2 * r + (i & 1)] * qs[r];
        p[r][i] = row_of[i] < 0 ? kNegInf : x;
      }
      if (MASS && g + 8 * r < n_rows) {
        const int head = head0 - (cons.hh / args.groups) * kv.G + g + 8 * r;
#pragma unroll
        for (int i = 0; i < 4; i++)
          if (row_of[i] >= 0)
            args.w.scores[(((int64_t)(row_of[i] >> kv.page_shift) * kv.G + head) << kv.page_shift) +
                          (row_of[i] & kv.page_mask)] = p[r][i];
      }
      float top = fmaxf(fmaxf(p[r][0], p[r][1]), fmaxf(p[r][2], p[r][3]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      m_new[r] = fmaxf(m[r], top);
      moved |= m_new[r] != m[r];
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int r = 0; r < NR; r++) {
        const float down = m_new[r] == m[r] ? 1.0f : exp2_fast(m[r] - m_new[r]);
        l[r] *= down;
#pragma unroll
        for (int n = 0; n < D / 8; n++) {
          o[n][2 * r] *= down;
          o[n][2 * r + 1] *= down;
        }
        m[r] = m_new[r];
      }
    }
    uint32_t hi_p[4], lo_p[4];
#pragma unroll
    for (int r = 0; r < NR; r++) {
      const float zero = m[r] == kNegInf ? 0.0f : m[r];  // a row without a score yet: 2^(-inf) = 0
#pragma unroll
      for (int i = 0; i < 4; i++) p[r][i] = exp2_fast(p[r][i] - zero);
      l[r] += (p[r][0] + p[r][1]) + (p[r][2] + p[r][3]);
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const float x = p[r][2 * i], y = p[r][2 * i + 1];
        if (E4M3) {
          hi_p[2 * i + r] = f16x2(x, y);
        } else {  // bf16 keeps 8 bits of p: the rest goes through a second product
          const uint32_t u = bf16x2(x, y);
          hi_p[2 * i + r] = u;
          lo_p[2 * i + r] = bf16x2(x - bf16_lo(u), y - bf16_hi(u));
        }
      }
    }
    if (NR == 1) hi_p[1] = hi_p[3] = lo_p[1] = lo_p[3] = 0u;

    if (!E4M3) {
#pragma unroll
      for (int n = 0; n < D / 16; n++) {
        uint32_t b[4];
        ldsm4t(b, v_at + v_lane + n * 32);
        mma<false>(o[2 * n], hi_p, b[0], b[1]);
        mma<false>(o[2 * n + 1], hi_p, b[2], b[3]);
        mma<false>(o[2 * n], lo_p, b[0], b[1]);
        mma<false>(o[2 * n + 1], lo_p, b[2], b[3]);
      }
    } else {
#pragma unroll
      for (int n = 0; n < D / 32; n++) {
        uint32_t b[4];  // entries 0-7 and 8-15 of 16 dims, then of the next 16
        ldsm4t(b, v_at + v_lane + n * 32);
#pragma unroll
        for (int u = 0; u < 2; u++) {
          const uint32_t x = __byte_perm(b[2 * u], 0, 0x3120), y = __byte_perm(b[2 * u + 1], 0, 0x3120);
          mma<true>(o[4 * n + 2 * u], hi_p, e4m3x2_to_f16x2(x), e4m3x2_to_f16x2(y));
          mma<true>(o[4 * n + 2 * u + 1], hi_p, e4m3x2_to_f16x2(x >> 16), e4m3x2_to_f16x2(y >> 16));
        }
      }
    }
    __syncwarp();  // the stage may be loaded again
    stage = stage + 1 == R::kStages ? 0 : stage + 1;

    const bool last = cons.t + 1 == cons.nt;
    if (last || at + 1 == hi) {
      const bool whole = last && row_first >= lo;
      end_row(cons.b, whole, row_first >= lo ? 1 : 0);
      if (!last) {
        const int j0 = row_first / chunk;
        going = Going{cons.b, cons.hh, j0, (row_first + cons.nt - 1) / chunk - j0 + 1};
      }
      row_first += cons.nt;
      if (at + 1 < hi) {
        advance(kv, cons, items);
        begin_row(cons.b, cons.hh);
      }
    } else {
      cons.t++;
    }
  }
  if (lane == 0) args.w.going[j] = going;
}

// ---------------------------------------------------------------------------
// join: block j serves the row that goes on past the end of chunk j.  The P
// parts of a row lie on the chunks j0 .. j0+P-1, so P - 1 blocks share its
// units (one query head x 32 dims): a row in many parts has many blocks.
// ---------------------------------------------------------------------------
struct JoinArgs {
  KvAttnArgs a;
  AttnWork w;
  int groups;
  int D;
  bool mass;
};

constexpr int kJoinWarps = 8;

__device__ __forceinline__ float part_weight(float m, float top) { return m == kNegInf ? 0.0f : exp2_fast(m - top); }

__global__ void __launch_bounds__(kJoinWarps * 32) k_kv_join(JoinArgs args) {
  __shared__ float s_acc[kJoinWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const KvView& kv = args.a.kv;
  kv_pdl_trigger();
  kv_pdl_wait();
  const Going gg = args.w.going[blockIdx.x];
  if (gg.b < 0) return;
  const int h = gg.hh / args.groups, gi = gg.hh - h * args.groups;
  const int n_rows = min(kRows, kv.G - gi * kRows), head0 = h * kv.G + gi * kRows;
  const int dims = args.D >> 5, units = n_rows * dims;
  const int parts = gg.parts, blocks = parts - 1, mine = (int)blockIdx.x - gg.j0;
  // Several units for this block: a warp each.  Else its warps share a unit's parts.
  const bool shared = units <= blocks * 4;
  for (int u = shared ? mine : mine + blocks * warp; u < units; u += shared ? blocks : blocks * kJoinWarps) {
    const int row = u / dims, dim = (u - row * dims) * 32 + lane;
    // part p lies on chunk j0 + p: side 1 (the row begins) for p = 0, else side 0
    auto slot = [&](int p) { return ((int64_t)(gg.j0 + p) * 2 + (p == 0 ? 1 : 0)) * kRows + row; };
    float top = kNegInf;
    for (int p = lane; p < parts; p += 32) top = fmaxf(top, args.w.ml[slot(p)].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    float sum = 0.0f;
    for (int p = lane; p < parts; p += 32) {
      const float2 ml = args.w.ml[slot(p)];
      sum += ml.x == kNegInf ? ml.y : ml.y * exp2_fast(ml.x - top);  // no score: l is 0, or NaN
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    float acc = 0.0f;
#pragma unroll 4
    for (int p = shared ? warp : 0; p < parts; p += shared ? kJoinWarps : 1) {
      const int64_t at = slot(p);
      acc += part_weight(args.w.ml[at].x, top) * args.w.o[at * args.D + dim];
    }
    if (shared) {
      s_acc[warp][lane] = acc;
      __syncthreads();
      if (warp == 0) {
        acc = 0.0f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; w++) acc += s_acc[w][lane];
      }
      __syncthreads();
      if (warp != 0) continue;
    }
    const int64_t head = (int64_t)gg.b * kv.Hq + head0 + row;
    const __nv_bfloat16 y = __float2bfloat16_rn(sum == 0.0f ? 0.0f : acc * (kv.v_scale / sum));
    args.a.out[head * args.D + dim] = *reinterpret_cast<const uint16_t*>(&y);
    if (dim == 0) {
      const float lse2 = sum == 0.0f ? kNegInf : top + log2f(sum);
      if (args.a.lse) args.a.lse[head] = lse2 * 0.6931471805599453f;
      if (args.mass) args.w.lse2[head] = lse2;
    }
  }
}

// ---------------------------------------------------------------------------
// mass: block j walks chunk j's tiles again, two a warp (a half warp each), and
// adds 2^(score - lse) over the query heads of the KV head.
// ---------------------------------------------------------------------------
constexpr int kMassThreads = 128;

__global__ void __launch_bounds__(kMassThreads) k_kv_mass(JoinArgs args) {
  const KvView& kv = args.a.kv;
  kv_pdl_wait();
  const int4 st = args.w.start[blockIdx.x];
  if (st.x < 0) return;
  const int items = kv.Hkv * args.groups;
  Place p{st.x, st.y, st.z, kv_length(kv, st.x), 0};
  p.nt = tiles_of(p.len);
  const int e = threadIdx.x & 15;
  int skip = threadIdx.x >> 4;
  for (int i = skip; i < st.w; i += kMassThreads / 16, skip = kMassThreads / 16) {
    p.t += skip;
    while (p.t >= p.nt) {
      p.t -= p.nt;
      if (++p.hh == items) {
        p.hh = 0;
        next_sequence(kv, p);
      }
    }
    const int h = p.hh / args.groups;
    const int slot = p.t * kTile + e;
    if (p.hh != h * args.groups || slot >= p.len) continue;  // the first group adds all heads of h
    const int row = kv_row(kv, p.b, h, slot);
    if (row < 0) continue;
    const float* sc = args.w.scores + (((int64_t)(row >> kv.page_shift) * kv.G) << kv.page_shift) + (row & kv.page_mask);
    const float* lse2 = args.w.lse2 + (int64_t)p.b * kv.Hq + h * kv.G;
    float sum = 0.0f;
#pragma unroll 8
    for (int g = 0; g < kv.G; g++) {
      const float z = lse2[g];
      sum += z == kNegInf ? 0.0f : exp2_fast(sc[(int64_t)g << kv.page_shift] - z);
    }
    kv.mass[row] += sum;
  }
}

template <int D, bool E4M3, bool WIDE, bool MASS>
cudaError_t run(const SplitArgs& a, int sms, cudaStream_t s) {
  using R = Ring<D * (E4M3 ? 1 : 2)>;
  static_assert(R::kStages >= 2 && R::kWarps <= kMaxWarps, "a ring of at least two stages fits");
  auto kern = k_kv_split<D, E4M3, WIDE, MASS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, R::kBytes);
  if (e != cudaSuccess) return e;
  kern<<<sms, R::kWarps * 32, R::kBytes, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const JoinArgs ja{a.a, a.w, a.groups, D, MASS};
  const dim3 chunks((unsigned)(sms * R::kWarps));
  if ((e = kv_launch_after(k_kv_join, chunks, kJoinWarps * 32, 0, s, ja)) != cudaSuccess) return e;
  return MASS ? kv_launch_after(k_kv_mass, chunks, kMassThreads, 0, s, ja) : cudaSuccess;
}

template <int D, bool E4M3>
cudaError_t run_d(const SplitArgs& a, int sms, cudaStream_t s) {
  if (a.a.kv.G > 8) return a.a.mass ? run<D, E4M3, true, true>(a, sms, s) : run<D, E4M3, true, false>(a, sms, s);
  return a.a.mass ? run<D, E4M3, false, true>(a, sms, s) : run<D, E4M3, false, false>(a, sms, s);
}

}  // namespace

int64_t kv_attn_workspace(const ft_kv_cache& c) {
  AttnWork w;
  return carve(w, nullptr, c.head_dim, c.n_seqs, c.n_heads, c.mass ? c.n_pages * c.n_kv_heads * c.page_size : 0,
               c.n_heads / c.n_kv_heads);
}

cudaError_t launch_kv_attention(const KvAttnArgs& args, bool e4m3, int sms, cudaStream_t s) {
  SplitArgs a;
  a.a = args;
  a.groups = (args.kv.G + kRows - 1) / kRows;
  const KvView& kv = args.kv;
  carve(a.w, args.work, kv.D, kv.n_seqs, kv.Hq, 0, kv.G);
  sms = sms < kKvMaxSms ? sms : kKvMaxSms;
  switch (kv.D) {
    case 64: return e4m3 ? run_d<64, true>(a, sms, s) : run_d<64, false>(a, sms, s);
    case 96: return e4m3 ? run_d<96, true>(a, sms, s) : run_d<96, false>(a, sms, s);
    case 128: return e4m3 ? run_d<128, true>(a, sms, s) : run_d<128, false>(a, sms, s);
    case 192: return e4m3 ? run_d<192, true>(a, sms, s) : run_d<192, false>(a, sms, s);
    default: return e4m3 ? run_d<256, true>(a, sms, s) : run_d<256, false>(a, sms, s);
  }
}

}  // namespace ft
