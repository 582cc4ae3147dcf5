// Host calls of the paged key-value cache (ft_kv_* of ft_moe.h): argument
// checks, then the launches of ft_kv_append.cu, ft_kv_attention.cu and
// ft_kv_evict.cu.  They keep no state: a cache is plain data of the caller.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "ft_kv.cuh"
#include "ft_runtime.h"

namespace {

ft_status refuse(ft_status st, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  ft::set_last_error(buf);
  return st;
}

ft_status cu(const char* what, cudaError_t e) {
  return e == cudaSuccess ? FT_OK : refuse(FT_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

#define KV_TRY(expr)                \
  do {                              \
    const ft_status st_ = (expr);   \
    if (st_ != FT_OK) return st_;   \
  } while (0)

int element_size(const ft_kv_cache& c) { return c.format == FT_KV_E4M3 ? 1 : 2; }

ft_status check_shape(const ft_kv_cache* c) {
  if (!c) return refuse(FT_ERR_INVALID, "cache is NULL");
  const int D = c->head_dim;
  if (D != 64 && D != 96 && D != 128 && D != 192 && D != 256)
    return refuse(FT_ERR_INVALID, "head_dim %d is not 64, 96, 128, 192 or 256", D);
  if (c->n_kv_heads <= 0 || c->n_heads <= 0 || c->n_heads % c->n_kv_heads || c->n_heads > 65536)
    return refuse(FT_ERR_INVALID, "n_heads %d is not a positive multiple of n_kv_heads %d, at most 65536", c->n_heads,
                  c->n_kv_heads);
  if (c->n_heads / c->n_kv_heads > 1024)
    return refuse(FT_ERR_INVALID, "n_heads / n_kv_heads %d is above 1024", c->n_heads / c->n_kv_heads);
  if (c->page_size < 8 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
    return refuse(FT_ERR_INVALID, "page_size %d is not a power of two from 8 to 1024", c->page_size);
  if (c->n_seqs < 0 || c->n_seqs > ft::kKvMaxSeqs)
    return refuse(FT_ERR_INVALID, "n_seqs %d not in [0, %d]", c->n_seqs, ft::kKvMaxSeqs);
  if (c->max_pages < 1 || (int64_t)c->max_pages * c->page_size > (1 << 30))
    return refuse(FT_ERR_INVALID, "max_pages %d: a sequence holds 1 page to 2^30 entries", c->max_pages);
  const int64_t rows_a_page = (int64_t)c->n_kv_heads * c->page_size;
  if (c->n_pages < 1 || c->n_pages >= ((int64_t)1 << 31) / rows_a_page)
    return refuse(FT_ERR_INVALID, "n_pages %lld: the pools hold 1 page to 2^31 - 1 rows", (long long)c->n_pages);
  const int64_t tiles = ((int64_t)c->max_pages * c->page_size + 15) / 16;
  if ((double)c->n_seqs * (double)tiles * (double)c->n_kv_heads >= 1073741824.0)
    return refuse(FT_ERR_INVALID, "n_seqs x max_pages x n_kv_heads is too large: below 2^30 tiles of 16 entries");
  if (c->format != FT_KV_BF16 && c->format != FT_KV_E4M3)
    return refuse(FT_ERR_INVALID, "format %d is not FT_KV_BF16 or FT_KV_E4M3", c->format);
  if (!(c->k_scale > 0) || !(c->v_scale > 0) || !std::isfinite(c->k_scale) || !std::isfinite(c->v_scale))
    return refuse(FT_ERR_INVALID, "k_scale and v_scale must be positive and finite");
  if (!std::isfinite(1.0f / c->k_scale) || !std::isfinite(1.0f / c->v_scale))
    return refuse(FT_ERR_INVALID, "k_scale or v_scale is 2^-128 or less: its reciprocal is not finite");
  if (c->format == FT_KV_BF16 && (c->k_scale != 1.0f || c->v_scale != 1.0f))
    return refuse(FT_ERR_INVALID, "k_scale and v_scale of a BF16 cache are 1");
  return FT_OK;
}

bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

ft_status check_cache(const ft_kv_cache* c) {
  KV_TRY(check_shape(c));
  if (c->n_seqs == 0) return FT_OK;
  if (!c->k || !c->v || !c->block_table || !c->lengths) return refuse(FT_ERR_INVALID, "NULL pool, block_table or lengths");
  if (!ft::aligned16(c->k) || !ft::aligned16(c->v))
    return refuse(FT_ERR_INVALID, "k and v pools must start on a 16-byte boundary");
  if (!aligned(c->mass, 4) || !aligned(c->pos, 4) || !aligned(c->block_table, 4) || !aligned(c->lengths, 4) ||
      !aligned(c->status, 4))
    return refuse(FT_ERR_INVALID, "mass, pos, block_table, lengths and status must start on a 4-byte boundary");
  return FT_OK;
}

// [p, p + bytes) and [q, q + more) have a byte in common.
bool overlap(const void* p, int64_t bytes, const void* q, int64_t more) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return p && q && a < b + (uintptr_t)more && b < a + (uintptr_t)bytes;
}

// Rows of q, k or v: `rows` of them `stride` elements apart, `width` elements each.
ft_status check_rows(const char* name, const void* p, int64_t rows, int64_t stride, int64_t width) {
  if (!ft::aligned16(p) || stride % 8)
    return refuse(FT_ERR_INVALID, "%s must start on a 16-byte boundary, its stride be a multiple of 8", name);
  if (stride < 0 || stride > ((int64_t)1 << 31) || (rows > 1 && stride < width && stride != 0))
    return refuse(FT_ERR_INVALID, "stride %lld of %s: 0, or its %lld elements a row to 2^31", (long long)stride, name,
                  (long long)width);
  return FT_OK;
}

int64_t rows_bytes(int64_t rows, int64_t stride, int64_t width) { return rows > 0 ? ((rows - 1) * stride + width) * 2 : 0; }

// Every pointer names memory of the current device (or of no GPU at all, managed):
// a kernel given host memory or a peer's would fault or read over the link.
struct Pointers {
  int device = -1;
  ft_status begin() { return cu("cudaGetDevice", cudaGetDevice(&device)); }
  ft_status on(const char* name, const void* p) {
    if (!p) return FT_OK;
    cudaPointerAttributes at;
    KV_TRY(cu("cudaPointerGetAttributes", cudaPointerGetAttributes(&at, p)));
    if (at.type == cudaMemoryTypeManaged) return FT_OK;
    if (at.type != cudaMemoryTypeDevice) return refuse(FT_ERR_INVALID, "%s is not device memory", name);
    if (at.device != device)
      return refuse(FT_ERR_INVALID, "%s is on device %d, the current device is %d", name, at.device, device);
    return FT_OK;
  }
  ft_status cache(const ft_kv_cache& c) {
    KV_TRY(begin());
    KV_TRY(on("k", c.k));
    KV_TRY(on("v", c.v));
    KV_TRY(on("mass", c.mass));
    KV_TRY(on("pos", c.pos));
    KV_TRY(on("block_table", c.block_table));
    KV_TRY(on("lengths", c.lengths));
    return on("status", c.status);
  }
};

ft_status sm_count(int device, int& sms) {
  return cu("cudaDeviceGetAttribute", cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device));
}

ft::KvView view(const ft_kv_cache& c) {
  ft::KvView v;
  v.D = c.head_dim;
  v.Hq = c.n_heads;
  v.Hkv = c.n_kv_heads;
  v.G = c.n_heads / c.n_kv_heads;
  v.page_shift = __builtin_ctz((unsigned)c.page_size);
  v.page_mask = c.page_size - 1;
  v.n_seqs = c.n_seqs;
  v.max_pages = c.max_pages;
  v.n_pages = (int)c.n_pages;
  v.cap = c.max_pages * c.page_size;
  v.k_scale = c.k_scale;
  v.v_scale = c.v_scale;
  v.k = (uint8_t*)c.k;
  v.v = (uint8_t*)c.v;
  v.mass = c.mass;
  v.pos = c.pos;
  v.table = c.block_table;
  v.lengths = c.lengths;
  v.status = c.status;
  return v;
}

ft_status check_workspace(const ft_kv_cache& c, const void* workspace, int64_t bytes) {
  int64_t need = 0;
  KV_TRY(ft_kv_workspace_bytes(&c, &need));
  if (!workspace || bytes < need)
    return refuse(FT_ERR_INVALID, "workspace of %lld bytes, %lld needed", (long long)(workspace ? bytes : 0), (long long)need);
  if (!ft::aligned16(workspace)) return refuse(FT_ERR_INVALID, "workspace must start on a 16-byte boundary");
  return FT_OK;
}

}  // namespace

extern "C" ft_status ft_kv_workspace_bytes(const ft_kv_cache* kv, int64_t* bytes) {
  KV_TRY(check_shape(kv));
  if (!bytes) return refuse(FT_ERR_INVALID, "bytes is NULL");
  const int64_t a = ft::kv_attn_workspace(*kv), e = kv->mass && kv->pos ? ft::kv_evict_workspace(*kv) : 0;
  *bytes = a > e ? a : e;
  return FT_OK;
}

extern "C" ft_status ft_kv_geometry(const ft_kv_cache* kv, int64_t tiles, int32_t sms, int64_t out[4]) {
  KV_TRY(check_shape(kv));
  if (!out) return refuse(FT_ERR_INVALID, "out is NULL");
  if (kv->n_seqs < 1) return refuse(FT_ERR_INVALID, "n_seqs 0 has no split");
  if (tiles < 0 || tiles >= (int64_t)1 << 30) return refuse(FT_ERR_INVALID, "tiles %lld not in [0, 2^30)", (long long)tiles);
  if (sms < 16 || sms > 1024) return refuse(FT_ERR_INVALID, "sms %d not in [16, 1024]", sms);
  ft::kv_geometry(*kv, (int)tiles, sms, out);
  return FT_OK;
}

extern "C" ft_status ft_kv_append(const ft_kv_cache* kv, int64_t T, const void* q, int64_t q_stride, const void* k,
                                  int64_t k_stride, const void* v, int64_t v_stride, const int32_t* cu_new,
                                  const int32_t* positions, int32_t n_axes, const double* inv_freq,
                                  const int32_t* axis, int32_t rot_dim, void* q_out, uint32_t flags, void* stream) {
  KV_TRY(check_cache(kv));
  if (T < 0 || T >= ((int64_t)1 << 31)) return refuse(FT_ERR_INVALID, "T %lld not in [0, 2^31)", (long long)T);
  if (!cu_new && T != kv->n_seqs)
    return refuse(FT_ERR_INVALID, "T %lld without cu_new: one row a sequence, %d", (long long)T, kv->n_seqs);
  if (flags & ~FT_ROPE_ADJACENT) return refuse(FT_ERR_INVALID, "unknown flags 0x%x", flags);
  if (rot_dim < 0 || rot_dim > kv->head_dim || rot_dim % 16)
    return refuse(FT_ERR_INVALID, "rot_dim %d is not a multiple of 16 from 0 to head_dim", rot_dim);
  if (n_axes < 0 || n_axes > 4 || ((rot_dim || kv->pos || positions) && n_axes < 1))
    return refuse(FT_ERR_INVALID, "n_axes %d not in [1, 4]", n_axes);
  if (T == 0 || kv->n_seqs == 0) return FT_OK;
  if (!k || !v || (q == nullptr) != (q_out == nullptr)) return refuse(FT_ERR_INVALID, "NULL k or v, or one of q and q_out");
  if ((rot_dim || kv->pos) && !positions) return refuse(FT_ERR_INVALID, "NULL positions");
  if (rot_dim && (!inv_freq || !axis)) return refuse(FT_ERR_INVALID, "NULL inv_freq or axis");
  const int64_t wq = (int64_t)kv->n_heads * kv->head_dim, wk = (int64_t)kv->n_kv_heads * kv->head_dim;
  if (q) KV_TRY(check_rows("q", q, T, q_stride, wq));
  KV_TRY(check_rows("k", k, T, k_stride, wk));
  KV_TRY(check_rows("v", v, T, v_stride, wk));
  if (!ft::aligned16(q_out)) return refuse(FT_ERR_INVALID, "q_out must start on a 16-byte boundary");
  if (!aligned(cu_new, 4) || !aligned(positions, 4) || !aligned(axis, 4) || !aligned(inv_freq, 8))
    return refuse(FT_ERR_INVALID, "cu_new, positions, axis or inv_freq is not aligned to its elements");
  const int64_t out_bytes = T * wq * 2;
  if (overlap(q_out, out_bytes, q, rows_bytes(T, q_stride, wq)) || overlap(q_out, out_bytes, k, rows_bytes(T, k_stride, wk)) ||
      overlap(q_out, out_bytes, v, rows_bytes(T, v_stride, wk)))
    return refuse(FT_ERR_INVALID, "q_out must not overlap q, k or v");
  ft::KvView vw = view(*kv);
  Pointers at;
  KV_TRY(at.cache(*kv));
  KV_TRY(at.on("q", q));
  KV_TRY(at.on("k", k));
  KV_TRY(at.on("v", v));
  KV_TRY(at.on("cu_new", cu_new));
  KV_TRY(at.on("positions", positions));
  KV_TRY(at.on("inv_freq", inv_freq));
  KV_TRY(at.on("axis", axis));
  KV_TRY(at.on("q_out", q_out));
  int sms = 0;
  KV_TRY(sm_count(at.device, sms));
  const ft::KvAppendArgs a{vw,       T,         (const uint16_t*)q, (const uint16_t*)k, (const uint16_t*)v,
                           q_stride, k_stride,  v_stride,           cu_new,             positions,
                           n_axes,   inv_freq,  axis,               rot_dim,            (uint16_t*)q_out};
  return cu("ft_kv_append", ft::launch_kv_append(a, kv->format == FT_KV_E4M3, flags & FT_ROPE_ADJACENT, sms, (cudaStream_t)stream));
}

extern "C" ft_status ft_kv_attention(const ft_kv_cache* kv, const void* q, int64_t q_stride, float scale, void* out,
                                     float* lse, void* workspace, int64_t workspace_bytes, uint32_t flags, void* stream) {
  KV_TRY(check_cache(kv));
  if (flags & ~FT_KV_MASS) return refuse(FT_ERR_INVALID, "unknown flags 0x%x", flags);
  if ((flags & FT_KV_MASS) && !kv->mass) return refuse(FT_ERR_INVALID, "FT_KV_MASS without a mass pool");
  if (!std::isfinite(scale)) return refuse(FT_ERR_INVALID, "scale is not finite");
  if (!std::isfinite(scale * 1.4426950408889634f * kv->k_scale))
    return refuse(FT_ERR_INVALID, "scale %g times log2(e) and k_scale %g is not finite", scale, kv->k_scale);
  if (kv->n_seqs == 0) return FT_OK;
  if (!q || !out) return refuse(FT_ERR_INVALID, "NULL q or out");
  const int64_t width = (int64_t)kv->n_heads * kv->head_dim;
  KV_TRY(check_rows("q", q, kv->n_seqs, q_stride, width));
  if (!ft::aligned16(out)) return refuse(FT_ERR_INVALID, "out must start on a 16-byte boundary");
  if (!aligned(lse, 4)) return refuse(FT_ERR_INVALID, "lse must start on a 4-byte boundary");
  if (overlap(out, kv->n_seqs * width * 2, q, rows_bytes(kv->n_seqs, q_stride, width)))
    return refuse(FT_ERR_INVALID, "out must not overlap q");
  KV_TRY(check_workspace(*kv, workspace, workspace_bytes));
  Pointers at;
  KV_TRY(at.cache(*kv));
  KV_TRY(at.on("q", q));
  KV_TRY(at.on("out", out));
  KV_TRY(at.on("lse", lse));
  KV_TRY(at.on("workspace", workspace));
  int sms = 0;
  KV_TRY(sm_count(at.device, sms));
  const ft::KvAttnArgs a{view(*kv), (const uint16_t*)q, q_stride, scale, (uint16_t*)out, lse, (uint8_t*)workspace,
                         (flags & FT_KV_MASS) != 0};
  return cu("ft_kv_attention", ft::launch_kv_attention(a, kv->format == FT_KV_E4M3, at.device, sms, (cudaStream_t)stream));
}

extern "C" ft_status ft_kv_evict(const ft_kv_cache* kv, const int32_t* budgets, int32_t recent, void* workspace,
                                 int64_t workspace_bytes, void* stream) {
  KV_TRY(check_cache(kv));
  if (recent < 0) return refuse(FT_ERR_INVALID, "recent %d is negative", recent);
  if (kv->n_seqs == 0) return FT_OK;
  if (!kv->mass || !kv->pos) return refuse(FT_ERR_INVALID, "eviction needs the mass and pos pools");
  if (!budgets || !aligned(budgets, 4)) return refuse(FT_ERR_INVALID, "budgets is NULL or not on a 4-byte boundary");
  KV_TRY(check_workspace(*kv, workspace, workspace_bytes));
  Pointers at;
  KV_TRY(at.cache(*kv));
  KV_TRY(at.on("budgets", budgets));
  KV_TRY(at.on("workspace", workspace));
  int sms = 0;
  KV_TRY(sm_count(at.device, sms));
  const ft::KvEvictArgs a{view(*kv), budgets, recent, (uint8_t*)workspace};
  return cu("ft_kv_evict", ft::launch_kv_evict(a, kv->head_dim * element_size(*kv), at.device, sms, (cudaStream_t)stream));
}

extern "C" ft_status ft_kv_sync_status(const ft_kv_cache* kv, void* stream) {
  if (!kv) return refuse(FT_ERR_INVALID, "cache is NULL");
  cudaStream_t s = (cudaStream_t)stream;
  int bits = 0;
  if (kv->status) {
    KV_TRY(cu("status", cudaMemcpyAsync(&bits, kv->status, sizeof bits, cudaMemcpyDeviceToHost, s)));
    KV_TRY(cu("status", cudaMemsetAsync(kv->status, 0, sizeof bits, s)));
  }
  KV_TRY(cu("synchronise", cudaStreamSynchronize(s)));
  if (bits & ft::kStTimeout) return refuse(FT_ERR_TIMEOUT, "a wait for a copy inside the GPU gave up");
  if (bits & ft::kStBadId)
    return refuse(FT_ERR_INVALID, "the cache's contents: a page, length, position, axis or budget out of range");
  return FT_OK;
}

extern "C" ft_status ft_debug_kv_wait(int32_t blocks, int64_t limit_us, int64_t arrive_us, int32_t* lanes, void* stream) {
  if (blocks < 1 || blocks > 1024) return refuse(FT_ERR_INVALID, "blocks %d not in [1, 1024]", blocks);
  if (limit_us < 1 || limit_us > 1000000 || arrive_us > 1000000)
    return refuse(FT_ERR_INVALID, "limit_us %lld not in [1, 1e6], or arrive_us %lld above 1e6", (long long)limit_us,
                  (long long)arrive_us);
  if (!lanes || !aligned(lanes, 4)) return refuse(FT_ERR_INVALID, "lanes is NULL or not on a 4-byte boundary");
  Pointers at;
  KV_TRY(at.begin());
  KV_TRY(at.on("lanes", lanes));
  return cu("ft_debug_kv_wait", ft::launch_kv_wait(blocks, (uint64_t)limit_us * 1000, arrive_us < 0 ? -1 : arrive_us * 1000,
                                                   lanes, (cudaStream_t)stream));
}
