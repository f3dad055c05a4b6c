// The paged K/V cache: geometry, the map from a sequence's positions to page
// rows, and the conversions between stored and computed values.
//
// A cache is K and V [pages, Hkv, page_size, D]; position p of sequence b is
// row p % page_size of page table[b][p / page_size].  kv_len[b] tokens are
// cached, new tokens included; new token i of the call's new_len[b] sits at
// position kv_len[b] - new_len[b] + i.  Nothing here trusts the device-side
// indices: lengths are clamped to the table, a table entry that names no page
// is "no row" (never dereferenced), and both are reported in the error word.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

namespace muse {

constexpr int kErrCacheIndex = 8;  // a length or a table entry outside its range

enum CacheType { kCacheBf16 = 0, kCacheF32 = 1, kCacheE4m3 = 2, kCacheI8 = 3 };

// n / d for 0 <= n < 2^31 by a multiplication: with s = ceil(log2 d) - 1 and
// mul = ceil(2^(32 + s) / d) < 2^32 the excess mul d - 2^(32 + s) < d <= 2^(s + 1)
// times n stays below 2^(32 + s).
struct FastDiv {
  uint32_t d, mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f{d, 0, 0};
  if (d > 1) {
    while ((2ull << f.shift) < d) ++f.shift;
    f.mul = (uint32_t)(((1ull << (32 + f.shift)) + d - 1) / d);
  }
  return f;
}
__host__ __device__ inline int div_by(const FastDiv& f, int n) {
#ifdef __CUDA_ARCH__
  return f.d == 1 ? n : (int)(__umulhi((uint32_t)n, f.mul) >> f.shift);
#else
  return f.d == 1 ? n : (int)((uint32_t)((uint64_t)(uint32_t)n * f.mul >> 32) >> f.shift);
#endif
}

struct Strides {  // elements
  long long b, h, t;
};

struct Cache {
  void *k, *v;          // [pages][Hkv][page][D]
  float *ks, *vs;       // [pages][Hkv][page], 8-bit caches only
  int pages, Hkv, D;
  FastDiv page;         // rows of a page
  const int* table;     // [B][wide]
  int wide;
  const int* kv_len;    // [B]
  const int* new_len;   // [B]; NULL: n everywhere
  int n;                // tokens a sequence can have in this call
  int* err;             // device error word or NULL
};

__device__ inline void flag_index(const Cache& c) {
  if (c.err) atomicOr(c.err, kErrCacheIndex);
}
// Cached and new tokens of sequence b, clamped to what the table and the call
// can hold (wide * page <= 2^30, so positions fit an int).
struct SeqLen {
  int kv;   // cached positions, [0, wide * page]
  int nn;   // new tokens, [0, n]
  int pos0; // position of new token 0 (negative when nn > kv)
};
__device__ inline SeqLen seq_len(const Cache& c, int b) {
  SeqLen s;
  const int cap = c.wide * (int)c.page.d;
  const int kv = c.kv_len[b], nn = c.new_len ? c.new_len[b] : c.n;
  s.kv = min(max(kv, 0), cap);
  s.nn = min(max(nn, 0), c.n);
  s.pos0 = s.kv - s.nn;
  if (s.kv != kv || s.nn != nn) flag_index(c);
  return s;
}
// First element row of (position's page row, head h): row index into
// [pages * Hkv * page] rows of D, or -1 when the table names no page.
__device__ inline long long row_of(const Cache& c, int b, int h, int pos) {
  const int p = div_by(c.page, pos);
  const int pg = __ldg(c.table + (long long)b * c.wide + p);
  if ((unsigned)pg >= (unsigned)c.pages) {
    flag_index(c);
    return -1;
  }
  return ((long long)pg * c.Hkv + h) * c.page.d + (pos - p * (int)c.page.d);
}

// Two e4m3 values held in the low 16 bits of x.
__device__ inline float2 e4m3x2(uint32_t x) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x & 0xFFFF), __NV_E4M3);
  return __half22float2(__half2(h));
}
// Eight consecutive values of row `row`, columns [8 c, 8 c + 8), in fp32 (with
// the row's scale where the cache has one).  row < 0: zeros.
template <int CT>
__device__ inline void load8(const void* base, const float* scales, long long row, int D, int c,
                             float (&x)[8]) {
  if (row < 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
    return;
  }
  const long long at = row * D + 8 * c;
  if (CT == kCacheF32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = p[0], b = p[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else if (CT == kCacheBf16) {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(v[e] << 16);
      x[2 * e + 1] = __uint_as_float(v[e] & 0xFFFF0000u);
    }
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const unsigned char*>(base) + at);
    const float s = scales[row];
    if (CT == kCacheE4m3) {
      const uint32_t v[4] = {w.x, w.x >> 16, w.y, w.y >> 16};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = e4m3x2(v[e]);
        x[2 * e] = f.x * s;
        x[2 * e + 1] = f.y * s;
      }
    } else {
      // q + 128 in the last bits of 2^23 (a conversion instruction takes four times
      // as long)
      const uint32_t v[2] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = (__uint_as_float(__byte_perm(v[e >> 2], 0x4B000000u, 0x7440 | (e & 3))) - 8388736.f) * s;
    }
  }
}

// The same from a strided tensor of a call (bf16 or fp32).
template <typename T>
__device__ inline void load8_in(const T* p, float (&x)[8]) {
  if (sizeof(T) == 4)
    load8<kCacheF32>(p, nullptr, 0, 0, 0, x);
  else
    load8<kCacheBf16>(p, nullptr, 0, 0, 0, x);
}

__device__ inline uint32_t bf16_bits2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ inline void store8(T* p, const float (&x)[8]) {
  if (sizeof(T) == 4) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(bf16_bits2(x[0], x[1]), bf16_bits2(x[2], x[3]),
                                              bf16_bits2(x[4], x[5]), bf16_bits2(x[6], x[7]));
  }
}

// A call of the attention over the cache (cache_attn*.cu).
struct CacheAttn {
  Cache c;
  const void* Q;  // strided, bf16 or fp32
  void* O;        // strided, Q's type
  float* lse;     // [B][Hq][n] or NULL
  Strides qs, os;
  int B, Hq, G;   // G = Hq / Hkv
  int f32;        // Q and O are fp32 (else bf16)
  int type;       // CacheType
  int causal;
  int window;     // 0: none
  float scale;
  // division of the keys (plan_cache_attn)
  int RT;         // row tiles of a kv-head
  int rows;       // packed rows of a tile
  int S;          // splits a row tile can have
  int minc;       // keys of a split, at least
  int quantum;    // a split's keys are a multiple of this
  int PR;         // rows of a split's partial
  int cluster;    // the splits of a tile are a cluster and join by themselves
  FastDiv by_G, by_Hkv, by_RT, by_S;
  int lost;       // failure tests: this load of every chunk CTA is never reported (-1: none)
  void* ws;       // partial o, then ml
  float2* ml;
};
// Keys that the query at position pos sees: [lo, hi), empty when hi <= lo.
__device__ inline int2 seen(const CacheAttn& a, const SeqLen& s, int pos) {
  if (!a.causal) return make_int2(0, s.kv);
  return make_int2(a.window ? max(0, pos - a.window + 1) : 0, min(pos + 1, s.kv));
}

void run_cache_write(const Cache& c, int type, const void* K, const void* V, const Strides& ks,
                     const Strides& vs, int f32, int B, cudaStream_t st);
void run_cache_read(const Cache& c, int type, void* K, void* V, int f32, int B, int N,
                    const int* start, cudaStream_t st);
size_t cache_attn_workspace(const CacheAttn& a);
// The division of the call's keys (a's fields), and what a row tile that sees
// `len` of them makes of it.
void cache_attn_division(CacheAttn& a, int len, int* parts, int* keys);
void run_cache_attn(const CacheAttn& a, cudaStream_t st);
void set_cache_fault(int load);

}  // namespace muse
