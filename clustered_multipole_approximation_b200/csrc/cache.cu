// Writing rows of K and V into the paged cache and reading them back.
//
// Both are one pass over the bytes: D / 8 lanes hold a row, eight values each,
// so that a row's largest magnitude is a shuffle reduction in registers and
// every load and store is 8 to 32 bytes a lane.  K and V of a row go through
// the same thread (two independent chains of loads).  Bound by HBM where the
// call is large, by the launch where it is one token a sequence.
#include "cache.cuh"
#include "kernels.h"

namespace muse {

namespace {

constexpr int kThreads = 256;

// Quantises eight values of a row whose D / 8 lanes form one shuffle group.
//   e4m3  scale 2^e, the smallest power of two with max|x| <= 448 2^e (e >=
//         -126): x / 2^e is exact, so the stored value is the one rounding of
//         the conversion; a finer scale would not buy a floating type more.
//   int8  scale max|x| / 127, q = the exact 127 x / max|x| rounded half to
//         even: a product with the rounded 127 / max|x| decides, except within
//         1e-4 of a half step (its error is below 127 2^-22), where the
//         quotient is formed in 64 bits.
//   a row of zeros has scale 1; a row that holds an infinity or a NaN is
//   stored as zeros with scale NaN, so that it reads back as NaN as a whole.
template <int CT, int LPR>
__device__ inline uint2 quantise8(const float (&x)[8], float& scale) {
  float top = 0.f;
  bool finite = true;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    top = fmaxf(top, fabsf(x[e]));  // fmaxf drops a NaN: kept in `finite`
    finite = finite && fabsf(x[e]) <= 3.4028234e38f;
  }
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) {
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o, LPR));
    finite = __shfl_xor_sync(0xffffffffu, (int)finite, o, LPR) && finite;
  }
  if (!finite || top == 0.f) {
    scale = finite ? 1.f : __int_as_float(0x7FC00000);
    return make_uint2(0, 0);
  }
  uint32_t w[2] = {0, 0};
  if (CT == kCacheE4m3) {
    const uint32_t u = __float_as_uint(top);  // 448 = 1.75 2^8
    int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    e = max(e, -126);
    scale = __uint_as_float((uint32_t)(e + 127) << 23);
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * inv, x[2 * i + 1] * inv),
                                                      __NV_SATFINITE, __NV_E4M3)
                   << (16 * (i & 1));
  } else {
    scale = __fdiv_rn(top, 127.f);
    const float inv = __fdiv_rn(127.f, top);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = x[i] * inv;
      float q = rintf(y);
      const float f = fabsf(y) - floorf(fabsf(y));
      if (!(fabsf(f - 0.5f) > 1e-4f))  // also a product that overflowed
        q = (float)rint((double)x[i] * 127.0 / (double)top);
      w[i >> 2] |= (uint32_t)((int)q & 0xFF) << (8 * (i & 3));
    }
  }
  return make_uint2(w[0], w[1]);
}

template <int CT, int LPR>
__device__ inline void put8(void* base, float* scales, long long row, int D, int c, bool live,
                            const float (&x)[8]) {
  if (CT == kCacheF32 || CT == kCacheBf16) {
    if (!live) return;
    const long long at = row * D + 8 * c;
    if (CT == kCacheF32)
      store8(static_cast<float*>(base) + at, x);
    else
      store8(static_cast<__nv_bfloat16*>(base) + at, x);
  } else {
    float s;
    const uint2 w = quantise8<CT, LPR>(x, s);  // every lane of the group takes part
    if (!live) return;
    *reinterpret_cast<uint2*>(static_cast<unsigned char*>(base) + row * D + 8 * c) = w;
    if (c == 0) scales[row] = s;
  }
}

// Work item: (sequence, token, head), heads fastest (the order of a
// projection's output, whose rows of one token lie side by side).
template <typename T, int CT, int D>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(Cache c, const T* K, const T* V,
                                                               Strides ks, Strides vs, long long rows) {
  constexpr int LPR = D / 8;
  const long long r = ((long long)blockIdx.x * kThreads + threadIdx.x) / LPR;
  const int col = threadIdx.x % LPR;
  long long row = -1;
  const T *kp = K, *vp = V;
  if (r < rows) {
    const long long bt = r / c.Hkv;
    const int h = (int)(r - bt * c.Hkv);
    const int b = (int)(bt / c.n), i = (int)(bt - (long long)b * c.n);
    const SeqLen s = seq_len(c, b);
    const int pos = s.pos0 + i;
    if (i < s.nn && pos >= 0) row = row_of(c, b, h, pos);
    kp += b * ks.b + h * ks.h + i * ks.t + 8 * col;
    vp += b * vs.b + h * vs.h + i * vs.t + 8 * col;
  }
  float x[8] = {}, y[8] = {};
  if (row >= 0) {
    load8_in(kp, x);
    load8_in(vp, y);
  }
  put8<CT, LPR>(c.k, c.ks, row, D, col, row >= 0, x);
  put8<CT, LPR>(c.v, c.vs, row, D, col, row >= 0, y);
}

// Work item: (sequence, head, row of the output), the output's own order.
template <typename T, int CT, int D>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(Cache c, T* K, T* V, const int* start,
                                                              int N, long long rows) {
  constexpr int LPR = D / 8;
  const long long r = ((long long)blockIdx.x * kThreads + threadIdx.x) / LPR;
  const int col = threadIdx.x % LPR;
  if (r >= rows) return;
  const long long bh = r / N;
  const int i = (int)(r - bh * N);
  const int b = (int)(bh / c.Hkv), h = (int)(bh - (long long)b * c.Hkv);
  const int kv = seq_len(c, b).kv;
  const int s0 = start ? start[b] : 0;
  if (s0 < 0) flag_index(c);
  const long long pos = (long long)max(s0, 0) + i;
  const long long row = pos < kv ? row_of(c, b, h, (int)pos) : -1;
  float x[8], y[8];
  load8<CT>(c.k, c.ks, row, D, col, x);
  load8<CT>(c.v, c.vs, row, D, col, y);
  store8(K + r * D + 8 * col, x);
  store8(V + r * D + 8 * col, y);
}

template <typename T, int CT>
void write_as(const Cache& c, const void* K, const void* V, const Strides& ks, const Strides& vs,
              int B, cudaStream_t st) {
  const long long rows = (long long)B * c.n * c.Hkv;
  const unsigned blocks = (unsigned)((rows * (c.D / 8) + kThreads - 1) / kThreads);
  const T *k = static_cast<const T*>(K), *v = static_cast<const T*>(V);
  if (c.D == 64)
    cache_write_kernel<T, CT, 64><<<blocks, kThreads, 0, st>>>(c, k, v, ks, vs, rows);
  else
    cache_write_kernel<T, CT, 128><<<blocks, kThreads, 0, st>>>(c, k, v, ks, vs, rows);
}
template <typename T, int CT>
void read_as(const Cache& c, void* K, void* V, int B, int N, const int* start, cudaStream_t st) {
  const long long rows = (long long)B * c.Hkv * N;
  const unsigned blocks = (unsigned)((rows * (c.D / 8) + kThreads - 1) / kThreads);
  T *k = static_cast<T*>(K), *v = static_cast<T*>(V);
  if (c.D == 64)
    cache_read_kernel<T, CT, 64><<<blocks, kThreads, 0, st>>>(c, k, v, start, N, rows);
  else
    cache_read_kernel<T, CT, 128><<<blocks, kThreads, 0, st>>>(c, k, v, start, N, rows);
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
