// Writing rows of K and V into the paged cache and reading them back.
//
// Both are one pass over the bytes: D / 16 lanes hold a row, two pieces of eight
// values each (D / 2 columns apart, so that neighbouring lanes touch
// neighbouring bytes), so that a row's largest magnitude is a shuffle reduction
// in registers and every load and store is 8 to 32 bytes a lane.  K and V of a
// row go through the same lanes (independent chains of loads).
//
// Bound by HBM where nothing is converted (32768 rows of 8 heads of 128, bf16:
// 45 us each way, 5.9 TB/s, 90 % of a copy's rate), by instructions beside it
// where rows are quantised (the same rows in int8: write 53 us, 3.9 TB/s; read
// 41 us, 4.9 TB/s; e4m3 of 64: write 21 us, 5.0 TB/s), by the launch where it is
// one token a sequence (4 us).  A piece a lane instead of two took 62 and 44 us.
#include "cache.cuh"
#include "kernels.h"

namespace muse {

namespace {

constexpr int kThreads = 256;

// Quantises sixteen values of a row whose D / 16 lanes form one shuffle group.
//   e4m3  scale 2^e, the smallest power of two with max|x| <= 448 2^e (e >=
//         -126): x / 2^e is exact, so the stored value is the one rounding of
//         the conversion; a finer scale would not buy a floating type more.
//   int8  scale max|x| / 127, q = the exact 127 x / max|x| rounded half to
//         even.  A product with 127 / max|x|, taken 2^-22 too large, decides:
//         its error lies below 127 (2^-22 + 2^-23) < 5e-5, and the half of the
//         maximum -- a tie at 63.5, and in bf16 rows by far the most frequent
//         one -- comes out above 63.5, so as 64, which is even.  Any other
//         value next to a half step h is decided exactly: with p = fl(h
//         max|x|), both 127 |x| - p (a multiple of |x|'s last bit, below
//         |x| / 16) and h max|x| - p are one FMA without error.  Rows far
//         outside the middle of the range are brought there by a power of two.
//   a row of zeros has scale 1; a row that holds an infinity or a NaN is
//   stored as zeros with scale NaN, so that it reads back as NaN as a whole.
template <int CT, int LPR>
__device__ inline void quantise(const float (&x0)[2][8], uint2 (&out)[2], float& scale) {
  uint32_t bits = 0;  // magnitudes as integers: a NaN is above infinity
#pragma unroll
  for (int e = 0; e < 16; ++e) bits = max(bits, __float_as_uint(x0[e >> 3][e & 7]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, o, LPR));
  out[0] = out[1] = make_uint2(0, 0);
  if (bits == 0 || bits >= 0x7F800000u) {
    scale = bits ? __int_as_float(0x7FC00000) : 1.f;
    return;
  }
  if (CT == kCacheE4m3) {  // 448 = 1.75 2^8
    int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    e = max(e, -126);
    scale = __uint_as_float((uint32_t)(e + 127) << 23);
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(x0[u][2 * i] * inv, x0[u][2 * i + 1] * inv), __NV_SATFINITE,
                                        __NV_E4M3);
      out[u] = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
    }
    return;
  }
  float top = __uint_as_float(bits), x[16];
  scale = __fdiv_rn(top, 127.f);
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] = x0[e >> 3][e & 7];
  if (bits < (27u << 23) || bits > (227u << 23)) {  // outside 2^-100 .. 2^100
    const float f = bits > (127u << 23) ? 0x1p-64f : 0x1p64f;
    top *= f;
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] *= f;
  }
  float inv = __fdiv_rn(127.f, top);
  inv = fmaf(inv, 0x1p-22f, inv);
  const float half = 0.5f * top;
  constexpr float kMagic = 12582912.f;  // 1.5 2^23: its sum with y ends in y's nearest integer
  uint32_t q[16];
  float far = 0.f;  // largest distance from the integers
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float t = fmaf(x[e], inv, kMagic);
    q[e] = __float_as_uint(t);
    const float rest = fabsf(fmaf(x[e], inv, -(t - kMagic)));
    far = fmaxf(far, fabsf(x[e]) == half ? 0.f : rest);
  }
  if (far > 0.5f - 5e-5f) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float ax = fabsf(x[e]), y = ax * inv, h = floorf(y) + 0.5f;
      if (fabsf(y - h) < 1e-4f) {
        const float p = h * top, d = fmaf(ax, 127.f, -p), r = fmaf(h, top, -p);
        const int lo = (int)(h - 0.5f);
        const int m = d > r ? lo + 1 : d < r ? lo : lo + (lo & 1);
        q[e] = (uint32_t)(x[e] < 0.f ? -m : m);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t* z = q + 8 * u + 4 * i;
      w[i] = __byte_perm(__byte_perm(z[0], z[1], 0x0040), __byte_perm(z[2], z[3], 0x0040), 0x5410);
    }
    out[u] = make_uint2(w[0], w[1]);
  }
}

// A lane's two pieces of a row to the cache; every lane of the row takes part.
template <int CT, int LPR>
__device__ inline void put(void* base, float* scales, long long row, int D, int c, bool live,
                           const float (&x)[2][8]) {
  if (CT == kCacheF32 || CT == kCacheBf16) {
    if (!live) return;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const long long at = row * D + 8 * (c + LPR * u);
      if (CT == kCacheF32)
        store8(static_cast<float*>(base) + at, x[u]);
      else
        store8(static_cast<__nv_bfloat16*>(base) + at, x[u]);
    }
  } else {
    float s;
    uint2 w[2];
    quantise<CT, LPR>(x, w, s);
    if (!live) return;
#pragma unroll
    for (int u = 0; u < 2; ++u)
      *reinterpret_cast<uint2*>(static_cast<unsigned char*>(base) + row * D + 8 * (c + LPR * u)) = w[u];
    if (c == 0) scales[row] = s;
  }
}

// Work item: (sequence, token, head), heads fastest (the order of a
// projection's output, whose rows of one token lie side by side).
template <typename T, int CT, int D>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(Cache c, const T* K, const T* V,
                                                               Strides ks, Strides vs, int rows,
                                                               FastDiv heads, FastDiv tokens) {
  constexpr int LPR = D / 16;
  const long long r = (long long)blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;
  const int col = threadIdx.x % LPR;
  long long row = -1;
  const T *kp = K, *vp = V;
  if (r < rows) {
    const int bt = div_by(heads, (int)r), h = (int)r - bt * c.Hkv;
    const int b = div_by(tokens, bt), i = bt - b * c.n;
    const SeqLen s = seq_len(c, b);
    const int pos = s.pos0 + i;
    if (i < s.nn && pos >= 0) row = row_of(c, b, h, pos);
    kp += b * ks.b + h * ks.h + i * ks.t + 8 * col;
    vp += b * vs.b + h * vs.h + i * vs.t + 8 * col;
  }
  float x[2][8] = {}, y[2][8] = {};
  if (row >= 0) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      load8_in(kp + 8 * LPR * u, x[u]);
      load8_in(vp + 8 * LPR * u, y[u]);
    }
  }
  put<CT, LPR>(c.k, c.ks, row, D, col, row >= 0, x);
  put<CT, LPR>(c.v, c.vs, row, D, col, row >= 0, y);
}

// Work item: (sequence, head, row of the output), the output's own order.  (Two
// rows a lane put more bytes behind the chain length, page, row, but took the
// registers of half the warps: 59 us against 42.)
template <typename T, int CT, int D>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(Cache c, T* K, T* V, const int* start,
                                                              int N, int rows, FastDiv heads,
                                                              FastDiv tokens) {
  constexpr int LPR = D / 16;
  const long long r = (long long)blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;
  const int col = threadIdx.x % LPR;
  if (r >= rows) return;
  const int bh = div_by(tokens, (int)r), i = (int)r - bh * N;
  const int b = div_by(heads, bh), h = bh - b * c.Hkv;
  const int kv = seq_len(c, b).kv;
  const int s0 = start ? start[b] : 0;
  if (s0 < 0) flag_index(c);
  const long long pos = (long long)max(s0, 0) + i;
  const long long row = pos < kv ? row_of(c, b, h, (int)pos) : -1;
  float x[2][8], y[2][8];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    load8<CT>(c.k, c.ks, row, D, col + LPR * u, x[u]);
    load8<CT>(c.v, c.vs, row, D, col + LPR * u, y[u]);
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    store8(K + r * D + 8 * (col + LPR * u), x[u]);
    store8(V + r * D + 8 * (col + LPR * u), y[u]);
  }
}

template <typename T, int CT>
void write_as(const Cache& c, const void* K, const void* V, const Strides& ks, const Strides& vs,
              int B, cudaStream_t st) {
  const int rows = B * c.n * c.Hkv;  // < 2^31, checked
  const unsigned blocks = (unsigned)(((long long)rows * (c.D / 16) + kThreads - 1) / kThreads);
  const FastDiv heads = fast_div((uint32_t)c.Hkv), tokens = fast_div((uint32_t)c.n);
  const T *k = static_cast<const T*>(K), *v = static_cast<const T*>(V);
  if (c.D == 64)
    cache_write_kernel<T, CT, 64><<<blocks, kThreads, 0, st>>>(c, k, v, ks, vs, rows, heads, tokens);
  else
    cache_write_kernel<T, CT, 128><<<blocks, kThreads, 0, st>>>(c, k, v, ks, vs, rows, heads, tokens);
}
template <typename T, int CT>
void read_as(const Cache& c, void* K, void* V, int B, int N, const int* start, cudaStream_t st) {
  const int rows = B * c.Hkv * N;  // < 2^31, checked
  const unsigned blocks = (unsigned)(((long long)rows * (c.D / 16) + kThreads - 1) / kThreads);
  const FastDiv heads = fast_div((uint32_t)c.Hkv), tokens = fast_div((uint32_t)N);
  T *k = static_cast<T*>(K), *v = static_cast<T*>(V);
  if (c.D == 64)
    cache_read_kernel<T, CT, 64><<<blocks, kThreads, 0, st>>>(c, k, v, start, N, rows, heads, tokens);
  else
    cache_read_kernel<T, CT, 128><<<blocks, kThreads, 0, st>>>(c, k, v, start, N, rows, heads, tokens);
}

}  // namespace

void run_cache_write(const Cache& c, int type, const void* K, const void* V, const Strides& ks,
                     const Strides& vs, int f32, int B, cudaStream_t st) {
  ProfScope ps(st, "cache_write");
  switch (type * 2 + f32) {
    case 0: return write_as<__nv_bfloat16, kCacheBf16>(c, K, V, ks, vs, B, st);
    case 1: return write_as<float, kCacheBf16>(c, K, V, ks, vs, B, st);
    case 2: return write_as<__nv_bfloat16, kCacheF32>(c, K, V, ks, vs, B, st);
    case 3: return write_as<float, kCacheF32>(c, K, V, ks, vs, B, st);
    case 4: return write_as<__nv_bfloat16, kCacheE4m3>(c, K, V, ks, vs, B, st);
    case 5: return write_as<float, kCacheE4m3>(c, K, V, ks, vs, B, st);
    case 6: return write_as<__nv_bfloat16, kCacheI8>(c, K, V, ks, vs, B, st);
    default: return write_as<float, kCacheI8>(c, K, V, ks, vs, B, st);
  }
}

void run_cache_read(const Cache& c, int type, void* K, void* V, int f32, int B, int N,
                    const int* start, cudaStream_t st) {
  ProfScope ps(st, "cache_read");
  switch (type * 2 + f32) {
    case 0: return read_as<__nv_bfloat16, kCacheBf16>(c, K, V, B, N, start, st);
    case 1: return read_as<float, kCacheBf16>(c, K, V, B, N, start, st);
    case 2: return read_as<__nv_bfloat16, kCacheF32>(c, K, V, B, N, start, st);
    case 3: return read_as<float, kCacheF32>(c, K, V, B, N, start, st);
    case 4: return read_as<__nv_bfloat16, kCacheE4m3>(c, K, V, B, N, start, st);
    case 5: return read_as<float, kCacheE4m3>(c, K, V, B, N, start, st);
    case 6: return read_as<__nv_bfloat16, kCacheI8>(c, K, V, B, N, start, st);
    default: return read_as<float, kCacheI8>(c, K, V, B, N, start, st);
  }
}

}  // namespace muse
