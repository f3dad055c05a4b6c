// Attention of a chunk of new tokens over the paged cache on the
// fifth-generation tensor cores (tcgen05, TMEM), bf16 queries.
//
// One CTA takes up to 256 packed rows of one (sequence, kv-head) -- all heads
// that share the keys -- and one split of its keys, in tiles of 128.  Two
// streams of 128 threads, a thread a row (its TMEM lane), take turns on the
// tensor cores: while one forms its softmax the other's products run.
//   S = Q K^T     tcgen05.mma, M = 128 rows, N = 128 keys, both operands in
//                 shared memory, the accumulator in TMEM;
//   P             2^(scale log2e S - m) rounded to bf16, stored over S;
//   O += P V      tcgen05.mma with P from TMEM, V MN-major in shared memory.
// With more than 128 rows the streams are two halves of the rows over the
// same key tiles; otherwise they are the even and the odd tiles of the same
// rows, joined at the end.  m moves only when a logit exceeds it by more than
// kSlack, so O is rescaled rarely.
//
// Pages are gathered by four load warps: a lane looks up the page row of one
// key, the warp copies whole rows into the 128-byte-swizzled operand form
// (cp.async), so that any page size is the same to them.  8-bit rows come
// through a raw ring and are converted on the way, exactly: V to bf16, K to fp16
// (half the instructions), which Q's rows, brought into fp16's range by powers
// of two, then are as well.  Scales of 8-bit rows multiply S's and P's columns.
//
// Warps 0-7: softmax of stream 0 (0-3) and 1 (4-7); 8-11: loads; 12: products.
// One warp issues all products, the streams in turn: that keeps them half a
// step apart (two issuing warps drift into step, softmax against softmax).
// Every wait is bounded.  After one that gives up each role leaves its loop: no
// further copies, products or reports; copies and products on their way are
// waited for before the CTA ends, the rows are NaN and kErrMmaWait is set.
//
// What bounds it: a stream's chain S -> maximum -> exponentials -> P V -> S,
// about 3300 cycles a tile pair at D = 128 where the products alone take 2100.
// 2048 tokens of 32 heads (8 kv-heads of 128) at 32768: 940 us in a short run,
// 1.13 PFLOP/s.  Tried and slower: tiles of 64 keys with two S buffers (the
// smaller products run at half rate: 1221 us against 1122), four softmax
// warpgroups (1223 against 1124), a polynomial for part of the exponentials
// (1145 against 977: instructions, not the special-function unit, are short).
#include "cache_attn.cuh"
#include "kernels.h"
#include "mma_sync.cuh"

#include <type_traits>

namespace muse {

namespace {

constexpr int kKeys = 128;    // keys of a tile
// Scales of a tile come with its K and are read until its softmax ends.  K[t + 8]
// is loaded after load 2 t + 9 or a later one was freed (at most 6 stages), which
// P V of tile t precedes.
constexpr int kScales = 8;
constexpr int kThreads = 512;
constexpr int kLoad = 128;    // load threads
// Registers a thread: 256 softmax x 192 + 128 load x 80 + 128 product x 48
// = the 512 x 128 of the launch.

__device__ inline int swz(int r, int q) { return r * 128 + ((q ^ (r & 7)) << 4); }
// K-major operand, 128-byte swizzle, 8-row groups 1 KB apart
__device__ inline uint64_t desc_k(uint32_t a) {
  return (uint64_t)((a >> 4) & 0x3FFF) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// MN-major operand, 128-byte swizzle: lbo = bytes between 64-element column chunks
__device__ inline uint64_t desc_mn(uint32_t a, uint32_t lbo) {
  return (uint64_t)((a >> 4) & 0x3FFF) | ((uint64_t)((lbo >> 4) & 0x3FFF) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ inline void umma(uint32_t tmem, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(tmem),
      "l"(ad), "l"(bd), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ inline void umma_ts(uint32_t tmem, uint32_t at, uint64_t bd, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(tmem),
      "r"(at), "l"(bd), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ inline void umma_commit(uint32_t mbar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(mbar)
               : "memory");
}
__device__ inline bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(e));
  return e != 0;
}
__device__ inline void mbar_init(uint32_t mbar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(mbar), "r"(count));
}
__device__ inline void mbar_arrive(uint32_t mbar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(mbar) : "memory");
}
__device__ inline bool mbar_test(uint32_t mbar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(done)
      : "r"(mbar), "r"(parity)
      : "memory");
  return done != 0;
}
// Bounded wait for the phase of this parity: false when it gave up, after half
// a second or because another wait of the CTA did.
__device__ inline bool mbar_wait(uint32_t mbar, uint32_t parity, volatile int* fail) {
  uint64_t start = 0;
  for (int it = 0; it < (1 << 24); ++it) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(done)
        : "r"(mbar), "r"(parity)
        : "memory");
    if (done) return true;
    if ((it & 63) == 63) {
      uint64_t now;
      asm volatile("mov.u64 %0, %%globaltimer;\n" : "=l"(now));
      if (start == 0) start = now;
      if (*fail || now - start > 500000000ull) break;
    }
  }
  *fail = 1;
  return false;
}
__device__ inline void tld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ inline void tst32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ inline void tst16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Two fp32 at a time: r[0..1] *= (a, b); r[0..1] = r aa + bb; s += r.
__device__ inline void mul2(uint32_t* r, float a, float b) {
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}\n"
      : "+r"(r[0]), "+r"(r[1])
      : "f"(a), "f"(b));
}
__device__ inline void fma2(uint32_t* r, uint64_t aa, uint64_t bb) {
  asm("{\n\t.reg .b64 x;\n\tmov.b64 x, {%0, %1};\n\tfma.rn.f32x2 x, x, %2, %3;\n\tmov.b64 {%0, %1}, x;\n\t}\n"
      : "+r"(r[0]), "+r"(r[1])
      : "l"(aa), "l"(bb));
}
__device__ inline uint64_t twice(float a) {
  uint64_t x;
  asm("mov.b64 %0, {%1, %1};\n" : "=l"(x) : "f"(a));
  return x;
}
__device__ inline void add2(uint64_t& s, const uint32_t* r) {
  asm("{\n\t.reg .b64 x;\n\tmov.b64 x, {%1, %2};\n\tadd.rn.f32x2 %0, %0, x;\n\t}\n"
      : "+l"(s)
      : "r"(r[0]), "r"(r[1]));
}
// The wait for this thread's TMEM loads, tied to their registers so that no
// use of them moves above it.
__device__ inline void tld_wait(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                 "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]),
                 "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]),
                 "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ inline void tst_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
__device__ inline void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ inline void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ inline void fence_async() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }
__device__ inline void streams_sync() { asm volatile("bar.sync 1, 256;\n" ::: "memory"); }
// The same barrier; whether any of its threads says so.
__device__ inline bool streams_any(bool x) {
  uint32_t y;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\tbar.red.or.pred p, 1, 256, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(y)
      : "r"((uint32_t)x)
      : "memory");
  return y != 0;
}

template <int CT, int D>
struct ChunkL {
  static constexpr int KB = D / 64;           // 64-column chunks
  static constexpr int QC = 128 * 128;        // bytes of one chunk of 128 rows
  static constexpr int Q = 0;                 // [stream][chunk][128 rows][128 B]
  static constexpr int STAGES = Q + 2 * KB * QC;
  static constexpr int SS = KB * QC;          // one tile of K or V
  static constexpr int NS = CT == kCacheBf16 ? (D == 128 ? 5 : 8) : (D == 128 ? 3 : 6);
  static constexpr int LAG = NS - 2;  // copies on their way while stages are free
  static constexpr int SC = STAGES + NS * SS;  // 8-bit: (k, v) scales [tile % kScales][2][128]
  static constexpr int RS = D == 128 ? 3 : 6;  // 8-bit: raw loads on their way, and the bytes of
  static constexpr int RAWW = 32 * D + 32 * 8;  // a load warp's share of one (rows, scales)
  static constexpr int RAW = SC + (CT == kCacheBf16 ? 0 : kScales * 2 * kKeys * 4);
  static constexpr int JOIN = D * 128 * 4 + 128 * 8;  // the second stream's o, (m, l)
  static constexpr int TOTAL = RAW + (CT == kCacheBf16 ? 0 : 4 * RS * RAWW) + 1024;
};

template <int CT, int D>
__global__ void __launch_bounds__(kThreads, 1) cache_chunk_kernel(const __grid_constant__ CacheAttn a) {
  using L = ChunkL<CT, D>;
  constexpr bool k8 = CT != kCacheBf16;
  constexpr int KB = L::KB, NS = L::NS;
  extern __shared__ __align__(1024) unsigned char chunk_raw[];
  unsigned char* sm = chunk_raw + ((1024 - (smem_u32(chunk_raw) & 1023)) & 1023);
  const uint32_t sb = smem_u32(sm);
  __shared__ __align__(8) uint64_t mFull[NS], mEmpty[NS], mS[2], mP[2][2], mO[2], mDone;
  __shared__ uint32_t tslot;
  __shared__ int sbad, sfail;
  __shared__ float qback[k8 ? 256 : 1];  // 8-bit: the power of two that undoes a row's factor

  const Place at0 = place_of(a);
  const int tile = at0.tile, split = at0.split, b = at0.b, h = at0.h;
  const SeqLen s = seq_len(a.c, b);
  const int r0 = at0.rt * 256;
  if (r0 >= s.nn * a.G) return;
  const RowTile rt = row_tile(a, s, r0, 256);
  const int len = rt.hi - rt.lo, parts = split_count(a, len);
  if (split >= parts) return;
  const int keys = split_keys(a, len);
  const int t0 = rt.lo + split * keys, t1 = min(rt.hi, t0 + keys);
  const int nt = (max(0, t1 - t0) + kKeys - 1) / kKeys;  // key tiles
  const bool two = rt.r1 - r0 > 128;  // the streams are row halves (else tile parities)
  auto steps = [&](int w) { return two ? nt : (nt - w + 1) >> 1; };
  auto tile_at = [&](int w, int k) { return two ? k : 2 * k + w; };
  // loads in the order of their use: K0, K1, V0, K2, V1, ... K[nt - 1], V[nt - 2],
  // V[nt - 1]; the number of a load is its place in that order.  The stage of
  // load i is freed by products that wait for no load past i + 1.
  auto k_item = [](int t) { return t == 0 ? 0 : 2 * t - 1; };
  auto v_item = [&](int t) { return min(2 * t + 2, 2 * nt - 1); };

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(&tslot)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
    if (lane == 0) {
      for (int i = 0; i < NS; ++i) {
        mbar_init(smem_u32(&mFull[i]), kLoad / 32);
        mbar_init(smem_u32(&mEmpty[i]), 1);
      }
      for (int w = 0; w < 2; ++w) {
        mbar_init(smem_u32(&mS[w]), 1);
        mbar_init(smem_u32(&mP[w][0]), 4);
        mbar_init(smem_u32(&mP[w][1]), 4);
        mbar_init(smem_u32(&mO[w]), 1);
      }
      mbar_init(smem_u32(&mDone), 1);
      sbad = sfail = 0;
      asm volatile("fence.mbarrier_init.release.cluster;\n");
    }
  }
  const int lw = warp - 8;  // of a load warp: its keys of a tile are 32 lw + lane
  auto lookup = [&](int T) -> int {
    const int t = t0 + T * kKeys + 32 * lw + lane;
    return T < nt && t < t1 ? (int)row_of(a.c, b, h, t) : -1;
  };
  const int first = warp >= 8 && warp < 12 ? lookup(0) : -1;  // on its way beside the queries
  {  // the query rows; rows past the tile are zero
    const __nv_bfloat16* Q = static_cast<const __nv_bfloat16*>(a.Q);
    constexpr int P = D / 8;  // 16-byte pieces of a row
    for (int e = tid; e < (two ? 256 : 128) * P; e += kThreads) {
      const int r = e / P, q = e % P;
      const bool live = r0 + r < rt.r1;
      const long long src = live ? row_at(a, b, h, r0 + r).q + 8 * q : 0;
      unsigned char* dst = sm + L::Q + (r >> 7) * KB * L::QC + (q >> 3) * L::QC + swz(r & 127, q & 7);
      if (!k8) {
        cp16(dst, Q + src, live ? 16 : 0);
      } else {
        // fp16 for the fp16 form of an 8-bit K, the row brought to a maximum in
        // [2^14, 2^15) by a power of two: exact for values down to 2^-31 of it
        const uint4 v = live ? *reinterpret_cast<const uint4*>(Q + src) : make_uint4(0, 0, 0, 0);
        float x[8];
        load8_in(reinterpret_cast<const __nv_bfloat16*>(&v), x);
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
        for (int o = P / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float2 f = half_factor(top);
        *reinterpret_cast<uint4*>(dst) =
            make_uint4(pack_h2(x[0] * f.x, x[1] * f.x), pack_h2(x[2] * f.x, x[3] * f.x),
                       pack_h2(x[4] * f.x, x[5] * f.x), pack_h2(x[6] * f.x, x[7] * f.x));
        if (q == 0) qback[r] = f.y;
      }
    }
    cp_commit();
    cp_wait<0>();
    fence_async();
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tbase = tslot;
  bool ok = true;  // this lane's waits; a warp goes on while all its lanes may
  auto all_ok = [&]() { return __all_sync(0xffffffffu, ok) != 0; };
  auto wait = [&](uint64_t& bar, int use) { ok = ok && mbar_wait(smem_u32(&bar), (uint32_t)(use & 1), &sfail); };

  if (warp >= 8 && warp < 12) {
    // ---- loads -----------------------------------------------------------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;\n");
    auto report = [&](int item) {
      fence_async();
      __syncwarp();
      if (lane == 0 && item != a.lost) mbar_arrive(smem_u32(&mFull[item % NS]));
    };
    auto begin = [&](int item) {  // its stage is free
      if (item >= NS) wait(mEmpty[item % NS], item / NS - 1);
    };
    // bf16: while stages are free, copies run LAG loads ahead of the report of
    // their arrival; before a wait for a stage every arrival is reported
    int signalled = 0, issued = 0;
    auto report_to = [&](int end) {
      for (; signalled < end; ++signalled) report(signalled);
    };
    auto copy = [&](int item, const void* base, int row) {
      if (item >= NS && !__all_sync(0xffffffffu, mbar_test(smem_u32(&mEmpty[item % NS]), (item / NS - 1) & 1))) {
        cp_wait<0>();
        report_to(issued);
        begin(item);
        if (!all_ok()) {
          ok = false;
          return;
        }
      }
      unsigned char* st = sm + L::STAGES + (item % NS) * L::SS;
      constexpr int LPR = D / 8, RPI = 32 / LPR;
      const int q = lane % LPR;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(base) + 8 * q;
      if (__all_sync(0xffffffffu, row >= 0)) {
#pragma unroll
        for (int j = 0; j < 32 / RPI; ++j) {
          const int r = j * RPI + lane / LPR;
          cp16(st + (q >> 3) * L::QC + swz(32 * lw + r, q & 7), src + (long long)__shfl_sync(0xffffffffu, row, r) * D);
        }
      } else {
#pragma unroll 1
        for (int j = 0; j < 32 / RPI; ++j) {
          const int r = j * RPI + lane / LPR;
          const int pr = __shfl_sync(0xffffffffu, row, r);
          cp16(st + (q >> 3) * L::QC + swz(32 * lw + r, q & 7), src + (long long)max(pr, 0) * D, pr < 0 ? 0 : 16);
        }
      }
      cp_commit();
    };
    // 8-bit: the raw rows of the next RS loads are on their way to a ring of this
    // thread's own (it converts the bytes that it copied)
    constexpr int LPR8 = D / 16, RPI8 = 32 / LPR8, N8 = 32 / RPI8;
    unsigned char* raw = sm + L::RAW + lw * (L::RS * L::RAWW);
    int fetched = 0, row_next = first, row_cur = -1, row_prev = -1;
    auto is_k = [&](int item) { return item == 0 || ((item & 1) && item < 2 * nt - 1); };
    auto fetch = [&]() {
      if (fetched < 2 * nt) {
        const bool k = is_k(fetched);
        if (k) {
          row_prev = row_cur;
          row_cur = row_next;
          row_next = lookup((fetched + 1) / 2 + 1);
        }
        // V[t] follows K[t + 1], the last V its own K
        const int row = k || fetched == 2 * nt - 1 ? row_cur : row_prev;
        unsigned char* dst = raw + (fetched % L::RS) * L::RAWW;
        const unsigned char* src = static_cast<const unsigned char*>(k ? a.c.k : a.c.v) + 16 * (lane % LPR8);
        if (__all_sync(0xffffffffu, row >= 0)) {
#pragma unroll
          for (int j = 0; j < N8; ++j)
            cp16(dst + (j * 32 + lane) * 16,
                 src + (long long)__shfl_sync(0xffffffffu, row, j * RPI8 + lane / LPR8) * D);
        } else {
#pragma unroll 1
          for (int j = 0; j < N8; ++j) {
            const int pr = __shfl_sync(0xffffffffu, row, j * RPI8 + lane / LPR8);
            cp16(dst + (j * 32 + lane) * 16, src + (long long)max(pr, 0) * D, pr < 0 ? 0 : 16);
          }
        }
        if (k) {
          cp4(dst + 32 * D + 8 * lane, a.c.ks + max(row, 0), row < 0 ? 0 : 4);
          cp4(dst + 32 * D + 8 * lane + 4, a.c.vs + max(row, 0), row < 0 ? 0 : 4);
        }
      }
      ++fetched;
      cp_commit();
    };
    auto convert = [&](int item, auto is_key) {
      constexpr bool K = decltype(is_key)::value;
      const unsigned char* from = raw + (item % L::RS) * L::RAWW;
      unsigned char* st = sm + L::STAGES + (item % NS) * L::SS;
      const int q = 2 * (lane % LPR8);
#pragma unroll
      for (int j = 0; j < N8; ++j) {
        const int r = 32 * lw + j * RPI8 + lane / LPR8;
        const uint4 u = *reinterpret_cast<const uint4*>(from + (j * 32 + lane) * 16);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        uint32_t y[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint2 z = K ? half_of_word<CT>(w[e]) : bf16_of_word<CT>(w[e]);
          y[2 * e] = z.x;
          y[2 * e + 1] = z.y;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<uint4*>(st + (q >> 3) * L::QC + swz(r, (q & 7) + e)) =
              make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
      }
      if (K) {  // its scales, and those of V[t]
        float* sc = reinterpret_cast<float*>(sm + L::SC) + (((item + 1) / 2) % kScales) * 2 * kKeys + 32 * lw + lane;
        const float2 f = *reinterpret_cast<const float2*>(from + 32 * D + 8 * lane);
        sc[0] = f.x;
        sc[kKeys] = f.y;
      }
    };
    if (nt > 0) {
      if (k8) {
        for (int i = 0; i < L::RS - 1; ++i) fetch();
        for (int item = 0; item < 2 * nt; ++item) {
          fetch();
          cp_wait<L::RS - 1>();
          begin(item);
          if (item >= NS && !all_ok()) break;
          if (is_k(item))
            convert(item, std::true_type());
          else
            convert(item, std::false_type());
          report(item);
        }
        cp_wait<0>();
      } else {
        int rk = first, rv = rk;  // page rows of the next K and the next V
        auto pump = [&]() {
          ++issued;
          cp_wait<L::LAG>();
          report_to(issued - L::LAG);
        };
        copy(k_item(0), a.c.k, rk);
        pump();
        for (int T = 0; T < nt; ++T) {
          rv = rk;
          rk = lookup(T + 1);
          if (T + 1 < nt) {
            copy(k_item(T + 1), a.c.k, rk);
            if (!ok) break;
            pump();
          }
          copy(v_item(T), a.c.v, rv);
          if (!ok) break;
          pump();
        }
        cp_wait<0>();
        if (ok) report_to(2 * nt);
      }
    }
  } else if (warp >= 12) {
    // ---- products --------------------------------------------------------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;\n");
    if (warp == 12) {
      // The whole warp walks the loop and one elected lane issues: operands stay in
      // uniform registers (a lane's own branch costs about 40 cycles a product).
      const uint32_t id_s = (1u << 4) | (k8 ? 0u : (1u << 7) | (1u << 10)) | ((uint32_t)(kKeys >> 3) << 17) | (8u << 24);
      const uint32_t id_pv = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | (8u << 24);
      const uint64_t qd = desc_k(sb + L::Q), kd = desc_k(sb + L::STAGES), vd = desc_mn(sb + L::STAGES, L::QC);
      const int unt = __shfl_sync(0xffffffffu, nt, 0);
      const uint32_t tb = __shfl_sync(0xffffffffu, tbase, 0);
      const bool both = __shfl_sync(0xffffffffu, (int)two, 0) != 0;
      const int n0 = both ? unt : (unt + 1) >> 1, n1 = both ? unt : unt >> 1;
      auto issue_s = [&](int w, int item) {
        const int st = item % NS;
        const uint64_t ad = qd + (both ? w : 0) * (KB * L::QC >> 4), bd = kd + st * (L::SS >> 4);
        if (elect_one()) {
#pragma unroll
          for (int q = 0; q < 4 * KB; ++q) {
            const uint32_t at = (q >> 2) * (L::QC >> 4) + 2 * (q & 3);
            umma(tb + 128 * w, ad + at, bd + at, id_s, q ? 1u : 0u);
          }
          umma_commit(smem_u32(&mS[w]));
          if (!both || w == 1) umma_commit(smem_u32(&mEmpty[st]));
        }
        __syncwarp();
      };
      for (int w = 0; w < 2; ++w)
        if ((w ? n1 : n0) > 0) {
          const int it = k_item(both ? 0 : w);
          wait(mFull[it % NS], it / NS);
          fence_after();
          if (all_ok()) issue_s(w, it);
        }
#pragma unroll 1
      for (int k = 0; k < n0 && all_ok(); ++k) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {  // step k of stream 0, then of stream 1
          const int n = w ? n1 : n0;
          if (k >= n) break;
          // the operands first, so that nothing stands between P V and the next S
          const int T = both ? k : 2 * k + w, more = k + 1 < n;
          const int vi = min(2 * T + 2, 2 * unt - 1), ki = more ? 2 * (both ? T + 1 : T + 2) - 1 : vi;
          const int vst = vi % NS;
          if (!both || w == 0) {
            wait(mFull[vst], vi / NS);
            wait(mFull[ki % NS], ki / NS);
          }
          bool go = true;
#pragma unroll
          for (int u = 0; u < 2; ++u) {  // P V of the tile's halves, as P comes
            wait(mP[w][u], k);
            fence_after();
            go = all_ok();  // the warp's vote: with a lane's own state the products are slower
            if (!go) break;
            if (elect_one()) {
              const uint64_t bd = vd + vst * (L::SS >> 4);
#pragma unroll
              for (int q = 4 * u; q < 4 * u + 4; ++q)
                umma_ts(tb + 256 + D * w, tb + 128 * w + 8 * q, bd + 128 * q, id_pv, (k | q) ? 1u : 0u);
              if (u && (!both || w == 1)) umma_commit(smem_u32(&mEmpty[vst]));
              if (u && !more) umma_commit(smem_u32(&mO[w]));
            }
            __syncwarp();
          }
          if (more && go) issue_s(w, ki);
        }
      }
      // what was issued still reads shared memory and writes TMEM and barriers, and after
      // a wait that gave up no softmax warp waits for its end
      int late = 0;
      if (elect_one()) umma_commit(smem_u32(&mDone));
      __syncwarp();
      mbar_wait(smem_u32(&mDone), 0, &late);
      if (late) sfail = 1;
    }
  } else {
    // ---- softmax: thread = row -------------------------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;\n");
    const int w = warp >> 2, row = tid & 127;
    const int pr = r0 + (two ? 128 * w : 0) + row;  // packed row
    const bool live = pr < rt.r1;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tbase + 128 * w + lanes, tO = tbase + 256 + D * w + lanes;
    // what this row, and every row of the stream, sees
    const int2 see = live ? seen(a, s, s.pos0 + div_by(a.by_G, pr)) : make_int2(0, 0);
    int alo = rt.alo, ahi = rt.ahi;
    if (two) {
      const int f = r0 + 128 * w, e = min(rt.r1, f + 128) - 1;
      alo = seen(a, s, s.pos0 + div_by(a.by_G, e)).x;
      ahi = seen(a, s, s.pos0 + div_by(a.by_G, f)).y;
    }
    const float sl2 = a.scale * kLog2e * (k8 ? qback[two ? 128 * w + row : row] : 1.f);
    // 8-bit: not the scale's sign, as a product of small factors may be zero, and 0 x -inf is
    // no mask (bf16: one branch for all rows)
    const bool pos = k8 ? sl2 > 0.f : a.scale > 0.f;
    const float mul = pos ? sl2 : 1.f;
    const uint64_t mul2x = twice(mul);
    float m = kFloor, l = 0.f;
    const int n = steps(w);
    // values that are not numbers would reach the rows that do not see them; every
    // warp of the stream looks through its keys, one without rows too.  (8-bit: before
    // S is loaded, 131 us against 134 for windowed chunks of e4m3; bf16: behind it,
    // 1088 us against 1105 for 2048 tokens at 32768.)
    auto look = [&](int T) {
      const int tb = t0 + T * kKeys, vi = v_item(T);
      if (CT == kCacheI8 || (tb >= alo && tb + kKeys <= ahi)) return;
      wait(mFull[vi % NS], vi / NS);
      constexpr int P = D / 8, RP = 128 / P;  // pieces of a key, keys of a pass
      const int c = row % P;
      const unsigned char* sv = sm + L::STAGES + (vi % NS) * L::SS + (c >> 3) * L::QC;
      uint32_t f = 0;  // a half's upper bit: its exponent is all ones
#pragma unroll 8
      for (int r = row / P; r < kKeys; r += RP) {
        const uint4 u = *reinterpret_cast<const uint4*>(sv + swz(r, c & 7));
        const uint32_t z = ((u.x & 0x7F807F80u) + 0x00800080u) | ((u.y & 0x7F807F80u) + 0x00800080u) |
                           ((u.z & 0x7F807F80u) + 0x00800080u) | ((u.w & 0x7F807F80u) + 0x00800080u);
        f |= tb + r >= alo && tb + r < ahi ? 0 : z;  // (a key that every row sees may be anything)
      }
      if (f & 0x80008000u) sbad = 1;
    };
    const bool idle = !__any_sync(0xffffffffu, live);
    for (int k = 0; idle && k < n; ++k) {  // no row of this warp is used, whatever its P is
      wait(mS[w], k);
      if (!all_ok()) break;
      look(tile_at(w, k));
      __syncwarp();
      if (lane < 2 && ok) mbar_arrive(smem_u32(&mP[w][lane]));
    }
    for (int k = 0; !idle && k < n && all_ok(); ++k) {
      const int T = tile_at(w, k), tb = t0 + T * kKeys;
      wait(mS[w], k);
      fence_after();
      if (k8) look(T);
      const float* sc = reinterpret_cast<const float*>(sm + L::SC) + (T % kScales) * 2 * kKeys;
      const bool edge = tb < alo || tb + kKeys > ahi || tb + kKeys > t1;
      const int clo = see.x - tb, chi = min(see.y, t1) - tb;
      uint32_t x[kKeys];
      // S of columns [c0, c0 + 64): scales, sign, mask
      auto logits = [&](int c0) {
        uint32_t* y = x + c0;
        if (k8) {
#pragma unroll
          for (int c = 0; c < 64; c += 4) {
            const float4 f = *reinterpret_cast<const float4*>(sc + c0 + c);
            mul2(y + c, f.x, f.y);
            mul2(y + c + 2, f.z, f.w);
          }
        }
        if (!pos) {  // logits first: the largest product need not be the largest logit
#pragma unroll
          for (int c = 0; c < 64; c += 2) mul2(y + c, sl2, sl2);
        }
        if (edge) {
#pragma unroll
          for (int q = 0; q < 64; q += 32) {
            // bit c: this row sees column c0 + q + c; most quarters are seen by every
            // row of the warp, or by none
            const int lo = min(max(clo - c0 - q, 0), 32), hi = min(max(chi - c0 - q, 0), 32);
            const uint32_t seen_cols = lo < hi ? (0xFFFFFFFFu >> (32 - hi)) & (0xFFFFFFFFu << lo) : 0u;
            if (__all_sync(0xffffffffu, seen_cols == 0xFFFFFFFFu)) continue;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!(seen_cols & (1u << c))) y[q + c] = 0xFF800000u;
          }
        }
      };
      uint64_t sum[2];
      uint32_t p[32];
      // weights of columns [c0, c0 + 64) from their logits
      auto weights = [&](int c0) {
        const uint64_t mm = twice(-m);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int c = c0 + 2 * e;
          fma2(x + c, mul2x, mm);
          x[c] = __float_as_uint(fast_exp2(__uint_as_float(x[c])));
          x[c + 1] = __float_as_uint(fast_exp2(__uint_as_float(x[c + 1])));
          add2(sum[e & 1], x + c);
          if (!k8) p[e] = bf16_bits2(__uint_as_float(x[c]), __uint_as_float(x[c + 1]));
        }
        if (k8) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const int c = c0 + 2 * e;
            const float4 f = *reinterpret_cast<const float4*>(sc + kKeys + c);
            mul2(x + c, f.x, f.y);
            mul2(x + c + 2, f.z, f.w);
          }
          if (edge) {  // a masked key's scale need not be a number
#pragma unroll
            for (int c = c0; c < c0 + 64; ++c)
              if (c < clo || c >= chi) x[c] = 0;
          }
#pragma unroll
          for (int e = 0; e < 32; ++e)
            p[e] = bf16_bits2(__uint_as_float(x[c0 + 2 * e]), __uint_as_float(x[c0 + 2 * e + 1]));
        }
      };
      auto store = [&](int u) {
        tst32(tS + 32 * u, p);
        tst_wait();
        fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(smem_u32(&mP[w][u]));
      };
#pragma unroll
      for (int q = 0; q < 4; ++q) tld32(tS + 32 * q, x + 32 * q);
#pragma unroll
      for (int q = 0; q < 4; ++q) tld_wait(x + 32 * q);
      if (!k8) look(T);
      logits(0);
      logits(64);
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < kKeys; c += 2)
        mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
      const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * mul;
      const bool move = top > m + kSlack;
      if (__any_sync(0xffffffffu, move)) {
        const float f = move ? fast_exp2(m - top) : 1.f;
        m = move ? top : m;
        l *= f;
        if (k > 0) {  // the stream's last P V is done: S came after it
#pragma unroll 1
          for (int d = 0; d < D; d += 32) {
            uint32_t r[32];
            tld32(tO + d, r);
            tld_wait(r);
#pragma unroll
            for (int e = 0; e < 32; e += 2) mul2(r + e, f, f);
            tst32(tO + d, r);
          }
        }
      }
      sum[0] = sum[1] = 0;
      weights(0);
      store(0);
      weights(64);
      store(1);
      const uint32_t odd[2] = {(uint32_t)sum[1], (uint32_t)(sum[1] >> 32)};
      add2(sum[0], odd);
      l += __uint_as_float((uint32_t)sum[0]) + __uint_as_float((uint32_t)(sum[0] >> 32));
    }
    if (n > 0) {
      wait(mO[w], 0);
      fence_after();
    }

    // ---- the rows: joined streams, normalised (or a split's partial) --------------
    float* jo = reinterpret_cast<float*>(sm + L::STAGES);  // [column][row]; every load was used
    float2* jml = reinterpret_cast<float2*>(jo + D * 128);
    // then the tile's rows, to be stored line by line
    unsigned char* rows_sm = sm + L::STAGES + (two ? 0 : L::JOIN);
    const int pitch = (parts > 1 ? 4 : 2) * D + 16;
    // Both streams' products are done, and with them all that was loaded -- or a wait
    // gave up: no numbers, whoever reads the flag.
    const bool failed = streams_any(!ok);
    if (failed) {
      for (int r = warp; r < rt.r1 - r0; r += 8) {
        const float nan = __int_as_float(0x7FC00000), y[8] = {nan, nan, nan, nan, nan, nan, nan, nan};
        const RowAt at = row_at(a, b, h, r0 + r);
        if (lane < D / 8) {
          if (parts > 1)
            store8(part_o<D>(a, tile, split, r) + 8 * lane, y);
          else
            store8(static_cast<__nv_bfloat16*>(a.O) + at.o + 8 * lane, y);
        }
        if (lane == 0 && parts > 1) *part_ml(a, tile, split, r) = make_float2(nan, nan);
        if (lane == 0 && parts == 1 && a.lse) a.lse[at.lse] = nan;
      }
    } else {
      if (!two) {
        if (w == 1 && n > 0) {
#pragma unroll
          for (int d = 0; d < D; d += 32) {
            uint32_t r[32];
            tld32(tO + d, r);
            tld_wait(r);
#pragma unroll
            for (int e = 0; e < 32; ++e) jo[(d + e) * 128 + row] = __uint_as_float(r[e]);
          }
          jml[row] = make_float2(m, l);
        }
        streams_sync();
      }
      const bool join = !two && steps(1) > 0;
      if (two || w == 0) {
        float f0 = 1.f, f1 = 0.f;
        if (join) {
          const float2 ml = jml[row];
          const float mn = fmaxf(m, ml.x);
          f0 = fast_exp2(m - mn);
          f1 = fast_exp2(ml.x - mn);
          m = mn;
          l = l * f0 + ml.y * f1;
        }
        const float inv = parts > 1 ? 1.f : l == 0.f ? 0.f : 1.f / l;
        unsigned char* to = rows_sm + (two ? 128 * w + row : row) * pitch;
#pragma unroll 1
        for (int d = 0; d < D; d += 32) {
          uint32_t r[32];
          if (n > 0) {
            tld32(tO + d, r);
            tld_wait(r);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = 0;
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              y[e] = __uint_as_float(r[8 * c + e]);
              if (join) y[e] = y[e] * f0 + jo[(d + 8 * c + e) * 128 + row] * f1;
              y[e] *= inv;
            }
            if (parts > 1)
              store8(reinterpret_cast<float*>(to) + d + 8 * c, y);
            else
              store8(reinterpret_cast<__nv_bfloat16*>(to) + d + 8 * c, y);
          }
        }
        if (live) {
          if (parts > 1)
            *part_ml(a, tile, split, pr - r0) = make_float2(m, l);
          else if (a.lse)
            a.lse[row_at(a, b, h, pr).lse] = lse_of(m, l);
        }
      }
      streams_sync();
      // whole rows from there: a lane's own row to global memory would touch 32 lines
      // a store (up to 8000 cycles a tile, 16 % of it)
      if (parts > 1) {
        constexpr int P = D / 4;
        const int c = tid % P;
        for (int r = tid / P; r < rt.r1 - r0; r += 256 / P)
          *reinterpret_cast<uint4*>(part_o<D>(a, tile, split, r) + 4 * c) =
              *reinterpret_cast<const uint4*>(rows_sm + r * pitch + 16 * c);
      } else {
        constexpr int P = D / 8;
        const int c = tid % P;
        for (int r = tid / P; r < rt.r1 - r0; r += 256 / P)
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.O) + row_at(a, b, h, r0 + r).o + 8 * c) =
              *reinterpret_cast<const uint4*>(rows_sm + r * pitch + 16 * c);
      }
      streams_sync();
      if (sbad)
        for (int r = r0 + warp; r < rt.r1; r += 8)
          redo_row<__nv_bfloat16, CT, D>(a, s, b, h, r, t0, t1, tile, split, parts, r0);
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (tid == 0 && sfail && a.c.err) atomicOr(a.c.err, kErrMmaWait);
  if (warp == 12)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tbase));
}

template <int CT, int D>
void launch(const CacheAttn& a, cudaStream_t st) {
  const int smem = ChunkL<CT, D>::TOTAL;
  static LargeShared allowed;
  allowed.ensure((const void*)cache_chunk_kernel<CT, D>, smem);
  const long long blocks = (long long)a.B * a.c.Hkv * a.RT * a.S;
  cache_chunk_kernel<CT, D><<<(unsigned)blocks, kThreads, smem, st>>>(a);
}

}  // namespace

void run_cache_chunk(const CacheAttn& a, cudaStream_t st) {
  ProfScope ps(st, "cache_chunk");
  switch (a.type * 2 + (a.c.D == 128)) {
    case 2 * kCacheBf16: return launch<kCacheBf16, 64>(a, st);
    case 2 * kCacheBf16 + 1: return launch<kCacheBf16, 128>(a, st);
    case 2 * kCacheE4m3: return launch<kCacheE4m3, 64>(a, st);
    case 2 * kCacheE4m3 + 1: return launch<kCacheE4m3, 128>(a, st);
    case 2 * kCacheI8: return launch<kCacheI8, 64>(a, st);
    default: return launch<kCacheI8, 128>(a, st);
  }
}

}  // namespace muse
