// ft_kv_append: rotary positions with several axes on new queries and keys,
// and the write of keys and values into the paged cache, in one pass.
//
// Pair i of a head turns by angle[t][i] = positions[axis[i]][t] * inv_freq[i]:
//   (x1, x2) -> (x1 cos - x2 sin, x2 cos + x1 sin).
// A position near 2^31 leaves a 32-bit angle no correct bit, so the product
// is fp64 and is brought into [-pi, pi] there; sine and cosine of the rest
// are fp32.  The heads of a token share its angles, so a block computes them
// once into shared memory and its threads then walk the token's heads, one
// 16-byte load of each side of a pair at a time.
//
// Bound by memory: every input is read once and every output written once
// ((4 Hq + 4 Hkv) D bytes and the cache rows a token); a single token is bound by the
// latency of its chain of loads (length, page, position, row).
#include <cuda_fp8.h>

#include "ft_kv.cuh"

namespace ft {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 4;   // tokens of a group
constexpr int kLone = 14;       // blocks of one token an SM has at most
constexpr int kMaxHalf = 128;   // rot_dim / 2 at most

struct Vec8 {
  float v[8];
};

__device__ __forceinline__ Vec8 load8(const uint16_t* p) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  Vec8 r;
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    r.v[2 * i] = __uint_as_float(u[i] << 16);
    r.v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
  return r;
}

__device__ __forceinline__ void store8(uint16_t* p, const Vec8& x) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x.v[2 * i], x.v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

// E4M3(x * inv), inv the rounded reciprocal of the scale: within a unit in the last
// place of the quotient, so the stored byte is the nearest one to it but for
// quotients that close to the middle between two.
__device__ __forceinline__ void store8_e4m3(uint8_t* p, const Vec8& x, float inv) {
  uint32_t u[2];
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const float* s = x.v + 4 * i;
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(s[0] * inv, s[1] * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(s[2] * inv, s[3] * inv), __NV_SATFINITE, __NV_E4M3);
    u[i] = lo | (hi << 16);
  }
  *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
}

__device__ __forceinline__ void load_floats(float (&v)[8], const float* s) {
  const float4 a = *reinterpret_cast<const float4*>(s), b = *reinterpret_cast<const float4*>(s + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ void prefetch_row(const uint16_t* p, int n) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(n * 2) : "memory");
}

// The last of the sequences whose new tokens begin at or before t, by the whole warp: 32
// places of the ascending cu_new are compared at a time.
__device__ __forceinline__ int find_sequence(const int32_t* cu_new, int n_seqs, int64_t t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, span = n_seqs;
  while (span > 1) {
    const int step = (span + 31) / 32, at = lane * step;
    const uint32_t before = __ballot_sync(0xffffffffu, at < span && cu_new[lo + at] <= t);
    const int k = before ? 31 - __clz(before) : 0;
    lo += k * step;
    span = min(step, span - k * step);
  }
  return lo;
}

// The rows of the block's tokens t0 .. t0 + nt - 1 for KV head 0 (-1: skipped), one in each of
// the first lanes of a warp.
__device__ __forceinline__ int find_row(const KvAppendArgs& a, int64_t t0, int nt) {
  const KvView& kv = a.kv;
  const int lane = threadIdx.x & 31;
  const int64_t t = t0 + lane;
  bool live = lane < nt;
  int b = (int)t, after = 1;  // new tokens of the sequence from this one on
  if (a.cu_new) {
    const int first = find_sequence(a.cu_new, kv.n_seqs, t0);
    const int begin = a.cu_new[0], end = a.cu_new[kv.n_seqs];
    b = first;
    int next = a.cu_new[b + 1];
    live = live && t >= begin && t < end;
    if (live && t >= next) {  // a later sequence: cu_new[lo] <= t < cu_new[hi]
      int lo = b, hi = kv.n_seqs;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu_new[mid] <= t) lo = mid;
        else hi = mid;
      }
      b = lo;
      next = a.cu_new[b + 1];
    }
    after = (int)(next - t);
  }
  if (!live) return -1;
  const int n = kv_length(kv, b, true);
  if (n == 0 && !a.cu_new) return -1;  // idle row
  const int slot = n - after;
  if (after <= 0 || slot < 0) {
    set_status(kv.status, kStBadId);
    return -1;
  }
  return kv_row(kv, b, 0, slot);
}

// A thread's place among the pieces (n a head) of the heads (m a token) of a block's
// tokens, and the step to its next one: no division on the way.
struct Walk {
  int token, head, piece;
  int n, m, step_heads, step_pieces;
  __device__ Walk(int first, int step, int pieces, int heads) : n(pieces), m(heads) {
    head = first / n;
    piece = first - head * n;
    token = head / m;
    head -= token * m;
    step_heads = step / n;
    step_pieces = step - step_heads * n;
  }
  __device__ void next() {
    piece += step_pieces;
    head += step_heads;
    if (piece >= n) {
      piece -= n;
      head++;
    }
    while (head >= m) {
      head -= m;
      token++;
    }
  }
};

// A block takes `group` tokens; their data are on their way into L2 while rows and angles
// are found.  blockIdx.y shares out a token's pieces where there are few tokens.
template <bool E4M3, bool ADJ>
__global__ void __launch_bounds__(kThreads, 6) k_kv_append(KvAppendArgs a, int group) {
  __shared__ __align__(16) float s_cos[kMaxTokens * kMaxHalf], s_sin[kMaxTokens * kMaxHalf];
  __shared__ int s_row[kMaxTokens];  // row of KV head 0, or -1
  __shared__ int s_bad[kMaxTokens];  // a position or axis is
  __shared__ const uint16_t* s_src[kMaxTokens][3];  // q, k and v rows
  const KvView& kv = a.kv;
  const int tid = threadIdx.x, D = kv.D, half = a.rot >> 1;
  const float k_inv = 1.0f / kv.k_scale, v_inv = 1.0f / kv.v_scale;
  const int first = blockIdx.y * kThreads + tid, step = gridDim.y * kThreads;
  // Queries and keys: a head is per_head pieces, 16 elements (8 of each side of 8
  // pairs) or 8 elements that stay together.
  const int piece = D >> 3, turning = ADJ ? a.rot >> 3 : a.rot >> 4;
  const int per_head = ADJ ? piece : turning + (piece - (a.rot >> 3));
  const int heads_q = a.q ? kv.Hq : 0;
  const Walk qk(first, step, per_head, heads_q + kv.Hkv), values(first, step, piece, kv.Hkv);
  // Angles: thread (u, f) takes frequency f of the tokens u, u + rows, ...
  const int rows = half > 0 ? kThreads / half : 0, u = half > 0 ? tid / half : 0, f = tid - u * half;
  if (tid < kMaxTokens) s_bad[tid] = 0;
  kv_pdl_wait();
  kv_pdl_trigger();
  int ax = -1;
  double freq = 0.0;
  if (u < rows) {
    ax = a.axis[f];
    freq = a.inv_freq[f];
    if ((unsigned)ax >= (unsigned)a.n_axes) ax = -1;
  }

  const int64_t t0 = (int64_t)blockIdx.x * group;
  const int nt = (int)min((int64_t)group, a.T - t0);
  __syncthreads();
  if (tid < nt) {
    const int64_t t = t0 + tid;
    const uint16_t* const src[3] = {a.q + t * a.q_stride, a.k + t * a.k_stride, a.v + t * a.v_stride};
    if (a.q) prefetch_row(src[0], kv.Hq * D);
    prefetch_row(src[1], kv.Hkv * D);
    prefetch_row(src[2], kv.Hkv * D);
#pragma unroll
    for (int i = 0; i < 3; i++) s_src[tid][i] = src[i];
  }
  if (u < rows) {
    const int32_t* const at = a.positions + (int64_t)max(ax, 0) * a.T + t0;
#pragma unroll 1
    for (int tt = u; tt < nt; tt += rows) {
      const int p = ax >= 0 ? at[tt] : -1;
      if (p < 0) s_bad[tt] = 1;
      const double turn = (double)p * freq;
      const double rest = fma(rint(turn * 0.15915494309189533577), -6.2831853071795864769, turn);
      sincosf((float)rest, &s_sin[tt * kMaxHalf + f], &s_cos[tt * kMaxHalf + f]);
    }
  }
  if (tid >= kThreads - 32) {  // the last warp has the fewest angles
    const int row = find_row(a, t0, nt), mine = tid - (kThreads - 32);
    if (mine < nt) {
      s_row[mine] = row;
      if (a.positions && a.positions[t0 + mine] < 0) s_bad[mine] = 1;
    }
  }
  __syncthreads();
  auto row_of = [&](int token) { return s_bad[token] ? -1 : s_row[token]; };
  uint16_t* const q_dst = a.q_out + t0 * kv.Hq * D;
#pragma unroll 1
  for (Walk w = qk; w.token < nt; w.next()) {
    const int row0 = row_of(w.token);
    if (row0 < 0) continue;
    const bool is_q = w.head < heads_q;
    const int h = is_q ? w.head : w.head - heads_q, c = w.piece;
    const int lo = ADJ || c < turning ? c * 8 : a.rot + (c - turning) * 8;
    const uint16_t* src = s_src[w.token][is_q ? 0 : 1] + h * D + lo;
    // where it goes: q_out, or the row of the pool
    uint8_t* const dst = is_q ? reinterpret_cast<uint8_t*>(q_dst + ((w.token * kv.Hq + h) * D + lo))
                              : kv.k + ((int64_t)(row0 + (h << kv.page_shift)) * D + lo) * (E4M3 ? 1 : 2);
    auto store = [&](const Vec8& y, int at) {
      if (E4M3 && !is_q) store8_e4m3(dst + at, y, k_inv);
      else store8(reinterpret_cast<uint16_t*>(dst) + at, y);
    };
    Vec8 x = load8(src);
    if (!ADJ && c < turning) {
      const Vec8 x2 = load8(src + half);
      float co[8], si[8];
      load_floats(co, s_cos + w.token * kMaxHalf + lo);
      load_floats(si, s_sin + w.token * kMaxHalf + lo);
      Vec8 y2;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float y1 = x.v[j] * co[j] - x2.v[j] * si[j];
        y2.v[j] = x2.v[j] * co[j] + x.v[j] * si[j];
        x.v[j] = y1;
      }
      store(y2, half);
    } else if (ADJ && c < turning) {
      const float4 co = *reinterpret_cast<const float4*>(s_cos + w.token * kMaxHalf + c * 4);
      const float4 si = *reinterpret_cast<const float4*>(s_sin + w.token * kMaxHalf + c * 4);
      const float cs[4] = {co.x, co.y, co.z, co.w}, sn[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const float x1 = x.v[2 * j], x2 = x.v[2 * j + 1];
        x.v[2 * j] = x1 * cs[j] - x2 * sn[j];
        x.v[2 * j + 1] = x2 * cs[j] + x1 * sn[j];
      }
    }
    store(x, 0);
  }
  // Values: stored as they are.
#pragma unroll 1
  for (Walk w = values; w.token < nt; w.next()) {
    const int row0 = row_of(w.token);
    if (row0 < 0) continue;
    const int at = w.piece * 8, row = row0 + (w.head << kv.page_shift);
    const uint16_t* src = s_src[w.token][2] + w.head * D + at;
    if (E4M3) store8_e4m3(kv.v + (int64_t)row * D + at, load8(src), v_inv);
    else *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(kv.v) + (int64_t)row * D + at) = *reinterpret_cast<const uint4*>(src);
  }
  if (blockIdx.y == 0) {
    if (tid < nt && s_row[tid] >= 0 && s_bad[tid]) set_status(kv.status, kStBadId);
    for (int i = tid; (kv.mass || kv.pos) && i < nt * kv.Hkv; i += kThreads) {
      const int token = i / kv.Hkv, row0 = row_of(token);
      if (row0 < 0) continue;
      const int row = row0 + ((i - token * kv.Hkv) << kv.page_shift);
      if (kv.mass) kv.mass[row] = 0.0f;
      if (kv.pos) kv.pos[row] = a.positions[t0 + token];
    }
  }
}

template <bool E4M3, bool ADJ>
cudaError_t run(const KvAppendArgs& a, dim3 grid, int group, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_kv_append<E4M3, ADJ>, a, group);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, bool e4m3, bool adjacent, int sms, cudaStream_t s) {
  // Few tokens: one a block, and several blocks a token while those leave SMs idle: the
  // latency of one token's chain counts then.  Beyond kLone blocks an SM (a little over two waves) up to 4
  // tokens share a block, whose 256 threads have their angles in one go: 8,191 tokens, 32 + 8 heads of
  // 128, 37.8 us with 14 (7: 40.3, 28: 48.8), 3,000 tokens 20.4 (16.1 and 20.3), 16,384 tokens 71.5 (71.7 and 67.7).
  const int64_t lone = (int64_t)sms * kLone;
  const int group = (int)(a.T <= lone ? 1 : a.T >= lone * kMaxTokens ? kMaxTokens : a.T / lone);
  const int64_t groups = (a.T + group - 1) / group;
  const int64_t pieces = (int64_t)((a.q ? a.kv.Hq : 0) + 2 * a.kv.Hkv) * (a.kv.D >> 3);
  int share = 1;
  while (share < 8 && a.T * share * 2 <= sms && pieces > (int64_t)kThreads * share) share *= 2;
  const dim3 grid((unsigned)groups, (unsigned)share);
  if (e4m3) return adjacent ? run<true, true>(a, grid, group, s) : run<true, false>(a, grid, group, s);
  return adjacent ? run<false, true>(a, grid, group, s) : run<false, false>(a, grid, group, s);
}

}  // namespace ft
