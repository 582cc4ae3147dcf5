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
constexpr int kMaxTokens = 8;   // tokens of a block
constexpr int kMaxHalf = 128;   // rot_dim / 2 at most

struct Vec8 {
  float v[8];
};

__device__ __forceinline__ Vec8 load8(const uint16_t* p) {
  const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
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

// E4M3(x / scale): a true division, so that the stored byte is the nearest one
// to the quotient in fp32.
__device__ __forceinline__ void store8_e4m3(uint8_t* p, const Vec8& x, float scale) {
  uint32_t u[2];
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const float* s = x.v + 4 * i;
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(s[0] / scale, s[1] / scale), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(s[2] / scale, s[3] / scale), __NV_SATFINITE, __NV_E4M3);
    u[i] = lo | (hi << 16);
  }
  *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
}

template <bool E4M3>
__device__ __forceinline__ void store_cache(uint8_t* pool, int row, int D, int at, const Vec8& x, float scale) {
  if (E4M3) store8_e4m3(pool + (int64_t)row * D + at, x, scale);
  else store8(reinterpret_cast<uint16_t*>(pool) + (int64_t)row * D + at, x);
}

// The sequence of new token t and its slot; false for a token that is skipped.
__device__ __forceinline__ bool locate(const KvAppendArgs& a, int64_t t, int& b, int& slot) {
  const KvView& kv = a.kv;
  int after = 1;  // new tokens of the sequence from this one on
  if (a.cu_new) {
    int lo = 0, hi = kv.n_seqs;  // cu_new[lo] <= t < cu_new[hi] once t is below cu_new[n_seqs]
    if (t >= a.cu_new[hi] || t < a.cu_new[0]) return false;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu_new[mid] <= t) lo = mid;
      else hi = mid;
    }
    b = lo;
    after = (int)(a.cu_new[hi] - t);
  } else {
    b = (int)t;
  }
  const int n = kv_length(kv, b, true);
  if (n == 0 && !a.cu_new) return false;  // idle row
  slot = n - after;
  if (after <= 0 || slot < 0) {
    set_status(kv.status, kStBadId);
    return false;
  }
  return true;
}

template <bool E4M3, bool ADJ>
__global__ void __launch_bounds__(kThreads) k_kv_append(KvAppendArgs a, int per_block) {
  __shared__ float s_cos[kMaxTokens * kMaxHalf], s_sin[kMaxTokens * kMaxHalf];
  __shared__ int s_row[kMaxTokens];  // row of KV head 0, or -1
  __shared__ int s_bad[kMaxTokens];
  const KvView& kv = a.kv;
  const int64_t t0 = (int64_t)blockIdx.x * per_block;
  const int nt = (int)min((int64_t)per_block, a.T - t0);
  const int tid = threadIdx.x;
  const int half = a.rot >> 1;

  if (tid < nt) {
    int b = 0, slot = 0, row = -1;
    if (locate(a, t0 + tid, b, slot)) row = kv_row(kv, b, 0, slot);
    s_row[tid] = row;
    s_bad[tid] = 0;
  }
  __syncthreads();
  for (int i = tid; i < nt * half; i += kThreads) {
    const int tt = i / half, f = i - tt * half;
    if (s_row[tt] < 0) continue;
    const int ax = __ldg(a.axis + f);
    int p = -1;
    if ((unsigned)ax < (unsigned)a.n_axes) p = __ldg(a.positions + (int64_t)ax * a.T + t0 + tt);
    if (p < 0) {
      s_bad[tt] = 1;
      continue;
    }
    const double turn = (double)p * __ldg(a.inv_freq + f);
    const double rest = fma(rint(turn * 0.15915494309189533577), -6.2831853071795864769, turn);
    sincosf((float)rest, &s_sin[tt * kMaxHalf + f], &s_cos[tt * kMaxHalf + f]);
  }
  if (tid < nt && s_row[tid] >= 0 && a.positions && __ldg(a.positions + t0 + tid) < 0) s_bad[tid] = 1;
  __syncthreads();
  if (tid < nt && s_bad[tid]) {
    set_status(kv.status, kStBadId);
    s_row[tid] = -1;
  }
  __syncthreads();

  // A head is per_head pieces: 16 elements (8 of each side of 8 pairs) or 8
  // elements that stay together.
  const int D = kv.D, piece = D >> 3;
  const int turning = ADJ ? a.rot >> 3 : a.rot >> 4;
  const int per_head = ADJ ? piece : turning + (piece - (a.rot >> 3));
  const int nq = a.q ? kv.Hq * per_head : 0;
  const int nk = kv.Hkv * per_head;
  const int per_token = nq + nk + kv.Hkv * piece;
  for (int w = tid; w < nt * per_token; w += kThreads) {
    const int tt = w / per_token;
    const int64_t t = t0 + tt;
    const int row0 = s_row[tt];
    if (row0 < 0) continue;
    int i = w - tt * per_token;
    if (i >= nq + nk) {  // a value: stored as it is
      i -= nq + nk;
      const int h = i / piece, at = (i - h * piece) * 8;
      const Vec8 x = load8(a.v + t * a.v_stride + h * D + at);
      store_cache<E4M3>(kv.v, row0 + (h << kv.page_shift), D, at, x, kv.v_scale);
      continue;
    }
    const bool is_q = i < nq;
    if (!is_q) i -= nq;
    const int h = i / per_head, c = i - h * per_head;
    const uint16_t* src = is_q ? a.q + t * a.q_stride + (int64_t)h * D : a.k + t * a.k_stride + (int64_t)h * D;
    uint16_t* const q_dst = a.q_out + (t * kv.Hq + h) * D;
    const int row = row0 + (h << kv.page_shift);
    const float* cs = s_cos + tt * kMaxHalf;
    const float* sn = s_sin + tt * kMaxHalf;
    if (c < turning && !ADJ) {
      const int lo = c * 8, hi = half + lo;
      const Vec8 x1 = load8(src + lo), x2 = load8(src + hi);
      Vec8 y1, y2;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float co = cs[lo + j], si = sn[lo + j];
        y1.v[j] = x1.v[j] * co - x2.v[j] * si;
        y2.v[j] = x2.v[j] * co + x1.v[j] * si;
      }
      if (is_q) {
        store8(q_dst + lo, y1);
        store8(q_dst + hi, y2);
      } else {
        store_cache<E4M3>(kv.k, row, D, lo, y1, kv.k_scale);
        store_cache<E4M3>(kv.k, row, D, hi, y2, kv.k_scale);
      }
    } else {
      const int at = ADJ ? c * 8 : a.rot + (c - turning) * 8;
      Vec8 x = load8(src + at);
      if (ADJ && c < turning) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const float co = cs[c * 4 + j], si = sn[c * 4 + j], x1 = x.v[2 * j], x2 = x.v[2 * j + 1];
          x.v[2 * j] = x1 * co - x2 * si;
          x.v[2 * j + 1] = x2 * co + x1 * si;
        }
      }
      if (is_q) store8(q_dst + at, x);
      else store_cache<E4M3>(kv.k, row, D, at, x, kv.k_scale);
    }
  }
  if (kv.mass || kv.pos) {
    for (int w = tid; w < nt * kv.Hkv; w += kThreads) {
      const int tt = w / kv.Hkv, h = w - tt * kv.Hkv;
      if (s_row[tt] < 0) continue;
      const int row = s_row[tt] + (h << kv.page_shift);
      if (kv.mass) kv.mass[row] = 0.0f;
      if (kv.pos) kv.pos[row] = __ldg(a.positions + t0 + tt);
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, bool e4m3, bool adjacent, cudaStream_t s) {
  // One token a block while there are fewer tokens than the GPU holds blocks
  // of this size (148 SMs x 8): the latency of one token's chain counts then.
  // Beyond, up to 8 tokens share a block, whose 256 threads compute the
  // angles of 2 to 8 of them at a time.
  const int64_t resident = 148 * 8;
  const int per_block = (int)(a.T <= resident ? 1 : a.T >= resident * kMaxTokens ? kMaxTokens : a.T / resident);
  const unsigned grid = (unsigned)((a.T + per_block - 1) / per_block);
  if (e4m3) {
    if (adjacent) k_kv_append<true, true><<<grid, kThreads, 0, s>>>(a, per_block);
    else k_kv_append<true, false><<<grid, kThreads, 0, s>>>(a, per_block);
  } else {
    if (adjacent) k_kv_append<false, true><<<grid, kThreads, 0, s>>>(a, per_block);
    else k_kv_append<false, false><<<grid, kThreads, 0, s>>>(a, per_block);
  }
  return cudaGetLastError();
}

}  // namespace ft
