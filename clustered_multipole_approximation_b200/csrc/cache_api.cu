// C entry points of the paged K/V cache: argument checks, then one launch
// sequence on the caller's stream.
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "../../include/muse.h"
#include "cache.cuh"
#include "kernels.h"

namespace muse {
void set_last_error(const char* msg);
}

using namespace muse;

namespace {

muse_status fail(muse_status s, const char* msg) {
  set_last_error(msg);
  return s;
}
muse_status check_launch() {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return MUSE_OK;
  return fail(MUSE_ERR_CUDA, (std::string("CUDA launch failed: ") + cudaGetErrorString(e)).c_str());
}
bool misaligned(const void* p, size_t a) { return p && (reinterpret_cast<uintptr_t>(p) % a) != 0; }

// `queries`: the call has q-heads; else Hq may be 0, and its rows are not counted.
muse_status check_shape(const muse_shape* sh, bool queries) {
  if (!sh) return fail(MUSE_ERR_INVALID_ARG, "shape must not be NULL");
  if (sh->B < 1 || sh->Hq < (queries ? 1 : 0) || sh->Hkv < 1 || sh->N < 1)
    return fail(MUSE_ERR_INVALID_ARG, "B, Hq, Hkv and N must be >= 1");
  if (sh->Hq % sh->Hkv) return fail(MUSE_ERR_INVALID_ARG, "Hq must be a multiple of Hkv");
  if (sh->D != 64 && sh->D != 128) return fail(MUSE_ERR_UNSUPPORTED, "D must be 64 or 128");
  if (sh->dtype != MUSE_BF16 && sh->dtype != MUSE_F32)
    return fail(MUSE_ERR_INVALID_ARG, "dtype must be MUSE_BF16 or MUSE_F32");
  if (sh->out_f32) return fail(MUSE_ERR_UNSUPPORTED, "the cache calls answer in the input dtype (out_f32 = 0)");
  if (sh->N > 1 << 28) return fail(MUSE_ERR_UNSUPPORTED, "N must be <= 2^28");
  const __int128 rows = (__int128)sh->B * (queries ? sh->Hq : sh->Hkv) * sh->N;
  if (rows > (1LL << 31) - 1) return fail(MUSE_ERR_UNSUPPORTED, "B*H*N must be < 2^31");
  return MUSE_OK;
}

muse_status check_cache(const muse_cache* ca, const muse_cache_index* ix, int Hkv) {
  if (!ca || !ix) return fail(MUSE_ERR_INVALID_ARG, "cache and index must not be NULL");
  if (ca->dtype < MUSE_CACHE_BF16 || ca->dtype > MUSE_CACHE_I8)
    return fail(MUSE_ERR_INVALID_ARG, "unknown cache dtype");
  if (ca->pages < 1 || ca->page_size < 1 || ix->wide < 1)
    return fail(MUSE_ERR_INVALID_ARG, "pages, page_size and wide must be >= 1");
  if ((long long)ix->wide * ca->page_size > 1LL << 30)
    return fail(MUSE_ERR_UNSUPPORTED, "wide * page_size must be <= 2^30");
  if ((__int128)ca->pages * ca->page_size * Hkv > (1LL << 31) - 1)  // 128 bytes a row of K and V at least
    return fail(MUSE_ERR_UNSUPPORTED, "pages * Hkv * page_size must be < 2^31");
  if (!ca->k || !ca->v || !ix->table || !ix->kv_len)
    return fail(MUSE_ERR_INVALID_ARG, "k, v, table and kv_len must not be NULL");
  const bool scaled = ca->dtype == MUSE_CACHE_E4M3 || ca->dtype == MUSE_CACHE_I8;
  if (scaled && (!ca->k_scale || !ca->v_scale))
    return fail(MUSE_ERR_INVALID_ARG, "an 8-bit cache needs k_scale and v_scale");
  if (!scaled && (ca->k_scale || ca->v_scale))
    return fail(MUSE_ERR_INVALID_ARG, "only an 8-bit cache has k_scale and v_scale");
  if (misaligned(ca->k, 16) || misaligned(ca->v, 16))
    return fail(MUSE_ERR_INVALID_ARG, "the cache must be 16-byte aligned");
  if (misaligned(ca->k_scale, 4) || misaligned(ca->v_scale, 4) || misaligned(ix->table, 4) ||
      misaligned(ix->kv_len, 4) || misaligned(ix->new_len, 4))
    return fail(MUSE_ERR_INVALID_ARG, "scales and index arrays must be 4-byte aligned");
  return MUSE_OK;
}

muse_status check_strides(const muse_strides* s, const muse_shape* sh) {
  if (!s) return fail(MUSE_ERR_INVALID_ARG, "strides must not be NULL");
  const int unit = sh->dtype == MUSE_BF16 ? 8 : 4;
  if (s->b < 0 || s->h < 0 || s->t < 0 || s->b % unit || s->h % unit || s->t % unit)
    return fail(MUSE_ERR_INVALID_ARG, "strides must be non-negative multiples of 16 bytes");
  return MUSE_OK;
}

// Whether rows of a written tensor may share an element: taken by growing
// stride, each must reach past everything the smaller ones span.
bool overlaps(const muse_strides* s, const muse_shape* sh, int H) {
  std::pair<int64_t, int64_t> d[3] = {{s->b, sh->B}, {s->h, H}, {s->t, sh->N}};
  std::sort(d, d + 3);
  __int128 span = sh->D;
  for (const auto& e : d) {
    if (e.second == 1) continue;
    if (e.first < span) return true;
    span += (__int128)e.first * (e.second - 1);
  }
  return false;
}

// Whether two written buffers of this size share memory, other than one buffer
// that gets the same twice.
bool clash(const void* a, const void* b, __int128 bytes, bool same) {
  if (a == b && same) return false;
  const __int128 x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bytes && y < x + bytes;
}

Cache device_cache(const muse_shape* sh, const muse_cache* ca, const muse_cache_index* ix, int* err) {
  Cache c{};
  c.k = ca->k;
  c.v = ca->v;
  c.ks = ca->k_scale;
  c.vs = ca->v_scale;
  c.pages = ca->pages;
  c.Hkv = sh->Hkv;
  c.D = sh->D;
  c.page = fast_div((uint32_t)ca->page_size);
  c.table = ix->table;
  c.wide = ix->wide;
  c.kv_len = ix->kv_len;
  c.new_len = ix->new_len;
  c.n = sh->N;
  c.err = err;
  return c;
}

Strides as_strides(const muse_strides* s) { return Strides{s->b, s->h, s->t}; }

CacheAttn attn_args(const muse_shape* sh, const muse_cache* ca, const muse_cache_index* ix, int* err) {
  CacheAttn a{};
  a.c = device_cache(sh, ca, ix, err);
  a.B = sh->B;
  a.Hq = sh->Hq;
  a.G = sh->Hq / sh->Hkv;
  a.f32 = sh->dtype == MUSE_F32;
  a.type = (int)ca->dtype;
  return a;
}

void clear_error(int32_t* err, cudaStream_t st) {
  if (err) cudaMemsetAsync(err, 0, 4, st);
}

}  // namespace

extern "C" {

muse_status muse_cache_write(const void* K, const muse_strides* ks, const void* V,
                             const muse_strides* vs, const muse_shape* sh, const muse_cache* ca,
                             const muse_cache_index* ix, int32_t* device_error, cudaStream_t st) {
  muse_status s = check_shape(sh, false);
  if (s == MUSE_OK) s = check_cache(ca, ix, sh->Hkv);
  if (s == MUSE_OK) s = check_strides(ks, sh);
  if (s == MUSE_OK) s = check_strides(vs, sh);
  if (s != MUSE_OK) return s;
  if (!K || !V) return fail(MUSE_ERR_INVALID_ARG, "K and V must not be NULL");
  if (misaligned(K, 16) || misaligned(V, 16))
    return fail(MUSE_ERR_INVALID_ARG, "K and V must be 16-byte aligned");
  if (misaligned(device_error, 4))
    return fail(MUSE_ERR_INVALID_ARG, "device_error must be 4-byte aligned");
  const int size = ca->dtype == MUSE_CACHE_BF16 ? 2 : ca->dtype == MUSE_CACHE_F32 ? 4 : 1;
  const bool same = K == V && ks->b == vs->b && ks->h == vs->h && ks->t == vs->t;
  const __int128 rows = (__int128)ca->pages * sh->Hkv * ca->page_size;
  if (clash(ca->k, ca->v, rows * sh->D * size, same) ||
      (size == 1 && clash(ca->k_scale, ca->v_scale, rows * 4, same)))
    return fail(MUSE_ERR_INVALID_ARG, "the caches of K and V must not share memory");
  clear_error(device_error, st);
  run_cache_write(device_cache(sh, ca, ix, device_error), (int)ca->dtype, K, V, as_strides(ks),
                  as_strides(vs), sh->dtype == MUSE_F32, sh->B, st);
  return check_launch();
}

muse_status muse_cache_read(void* K, void* V, const muse_shape* sh, const muse_cache* ca,
                            const muse_cache_index* ix, const int32_t* start,
                            int32_t* device_error, cudaStream_t st) {
  muse_status s = check_shape(sh, false);
  if (s == MUSE_OK) s = check_cache(ca, ix, sh->Hkv);
  if (s != MUSE_OK) return s;
  if (!K || !V) return fail(MUSE_ERR_INVALID_ARG, "K and V must not be NULL");
  if (misaligned(K, 16) || misaligned(V, 16))
    return fail(MUSE_ERR_INVALID_ARG, "K and V must be 16-byte aligned");
  if (misaligned(device_error, 4) || misaligned(start, 4))
    return fail(MUSE_ERR_INVALID_ARG, "start and device_error must be 4-byte aligned");
  if (clash(K, V, (__int128)sh->B * sh->Hkv * sh->N * sh->D * (sh->dtype == MUSE_F32 ? 4 : 2),
            ca->k == ca->v && ca->k_scale == ca->v_scale))
    return fail(MUSE_ERR_INVALID_ARG, "K and V must not share memory");
  clear_error(device_error, st);
  Cache c = device_cache(sh, ca, ix, device_error);
  c.new_len = nullptr;
  run_cache_read(c, (int)ca->dtype, K, V, sh->dtype == MUSE_F32, sh->B, sh->N, start, st);
  return check_launch();
}

size_t muse_attn_cache_workspace_size(const muse_shape* sh, const muse_cache* ca,
                                      const muse_cache_index* ix) {
  if (check_shape(sh, true) != MUSE_OK || check_cache(ca, ix, sh->Hkv) != MUSE_OK) return 0;
  return cache_attn_workspace(attn_args(sh, ca, ix, nullptr));
}

void muse_debug_inject_cache_fault(int load) { set_cache_fault(load < 0 ? -1 : load); }

muse_status muse_debug_cache_division(const muse_shape* sh, const muse_cache* ca,
                                      const muse_cache_index* ix, int window, int len,
                                      muse_cache_division* out) {
  muse_status s = check_shape(sh, true);
  if (s == MUSE_OK) s = check_cache(ca, ix, sh->Hkv);
  if (s != MUSE_OK) return s;
  if (!out || window < 0 || len < 0 || len > ix->wide * ca->page_size)
    return fail(MUSE_ERR_INVALID_ARG, "out must not be NULL, window >= 0 and len within the table");
  CacheAttn a = attn_args(sh, ca, ix, nullptr);
  a.window = window >= 1 << 30 ? 0 : window;
  cache_attn_division(a, len, &out->parts, &out->keys);
  out->tiles = (long long)sh->B * sh->Hkv * a.RT;
  out->rows = a.PR;
  out->splits = a.S;
  out->cluster = a.cluster;
  out->quantum = a.quantum;
  return MUSE_OK;
}

muse_status muse_attn_cache(const void* Q, const muse_strides* qs, void* O, const muse_strides* os,
                            float* lse, const muse_shape* sh, const muse_cache* ca,
                            const muse_cache_index* ix, float scale, int causal, int window,
                            int32_t* device_error, void* ws, size_t ws_bytes, cudaStream_t st) {
  muse_status s = check_shape(sh, true);
  if (s == MUSE_OK) s = check_cache(ca, ix, sh->Hkv);
  if (s == MUSE_OK) s = check_strides(qs, sh);
  if (s == MUSE_OK) s = check_strides(os, sh);
  if (s != MUSE_OK) return s;
  if (!Q || !O) return fail(MUSE_ERR_INVALID_ARG, "Q and O must not be NULL");
  if (misaligned(Q, 16) || misaligned(O, 16))
    return fail(MUSE_ERR_INVALID_ARG, "Q and O must be 16-byte aligned");
  if (misaligned(lse, 4) || misaligned(device_error, 4))
    return fail(MUSE_ERR_INVALID_ARG, "lse and device_error must be 4-byte aligned");
  if (overlaps(os, sh, sh->Hq)) return fail(MUSE_ERR_INVALID_ARG, "the rows of O must not overlap");
  if (!isfinite(scale)) return fail(MUSE_ERR_INVALID_ARG, "scale must be finite");
  if (causal != 0 && causal != 1) return fail(MUSE_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (window < 0) return fail(MUSE_ERR_INVALID_ARG, "window must be >= 0");
  if (window && !causal) return fail(MUSE_ERR_INVALID_ARG, "a window needs causal = 1");
  CacheAttn a = attn_args(sh, ca, ix, device_error);
  if (misaligned(ws, 256)) return fail(MUSE_ERR_INVALID_ARG, "the workspace must be 256-byte aligned");
  if (!ws || ws_bytes < cache_attn_workspace(a))
    return fail(MUSE_ERR_WORKSPACE, "workspace too small");
  if (Q == O) return fail(MUSE_ERR_INVALID_ARG, "O must not share memory with Q");
  a.Q = Q;
  a.O = O;
  a.lse = lse;
  a.qs = as_strides(qs);
  a.os = as_strides(os);
  a.causal = causal;
  a.window = window >= 1 << 30 ? 0 : window;  // wider than any table: no limit
  a.scale = scale;
  a.ws = ws;
  clear_error(device_error, st);
  run_cache_attn(a, st);
  return check_launch();
}

}  // extern "C"
