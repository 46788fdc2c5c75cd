// Differential attention on sm_100a:
//
//   O = A_1 V - lambda_h A_2 V,  A_m = softmax(Q_m K_m^T * scale) over the
//   allowed keys, Q = [Q_1 | Q_2] and K = [K_1 | K_2] with d / 2 channels
//   each, V with d;  lambda_h = exp(a_1 . b_1) - exp(a_2 . b_2) + lambda_init
//   from four learned vectors per head;  then, with norm weights, per head
//   O <- O / sqrt(mean(O^2) + eps) * w * (1 - lambda_init).
//
// The dense forward's roles (attn_fwd.cu), with the two maps of ONE 128-row
// query tile in the place of its two query tiles: both read the same V tile,
// and each takes its half of the channels of the same Q and K tiles, so the
// shared-memory and L2 traffic of a key tile serves both maps.  Per key tile
// the CTA does 2 x 128 x 128 exponentials (the dense kernel's count) for 3/4
// of its products.  Neither unit is full (exponential unit 55% active, tensor
// pipe 46% at 12 heads x 4736): what bounds a long walk is the softmax warps'
// turns on the exponential unit, about 650 clocks per half and 150 for the
// hand-over, of which the unit works 430.
//   warps 0..3  softmax of map 0, warps 4..7 of map 1: one thread per query
//               row, online softmax with lazy rescale, P into the S columns;
//               then O_1 / l_1 - lambda O_2 / l_2 for half of the channels
//               each: both maps' accumulators lie in the same TMEM lanes, so
//               only the row sums and the norm's partial sums of squares go
//               through shared memory.
//   warp 8      issues map 0's products, warp 11 map 1's, after it has found
//               the CTA's share of the work (one warp for both maps: 8 single
//               queries over 16384 keys took 111 us, so 104; prompts 1% more);
//               warp 9 TMA producer, warp 10 zeroes the V rows of masked keys
//               in shared memory (their P is 0, and 0 * NaN would not be).
// Keys are walked in halves of 64: each map has two S buffers of 64 TMEM
// columns, and Q.K^T of half i + 2 is issued behind P.V of half i, so S of
// half i + 1 is there when the softmax of half i ends and the softmax warps
// do not wait for the tensor pipe.  TMEM: S [0, 256), O_1 [256, +d), O_2 [384,
// +d).
// Query rows of the heads that share a K/V head are packed into one row
// range where the strides allow it, so a cache is read once for the group.
// Work: an item is one 128-row tile of one range.  Whole waves of items go
// one item at a time to the SMs (neighbouring CTAs then walk the same keys);
// the items of the last, partial wave -- all items of a single-token call --
// are cut into equal runs of key tiles, one per CTA.  A CTA that has a part of
// an item writes its normalised output and log-sum-exp; a second kernel
// merges the parts.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "jattn.h"
#include "jattn_internal.h"
#include "ptx_sm100.cuh"

namespace jattn {

namespace {

constexpr int BM = 128;                // query rows per tile
constexpr int BN = 128;                // keys per tile
constexpr int kMmaWarp = 8, kProducerWarp = 9, kMaskWarp = 10, kShareWarp = 11;
constexpr int kThreads = 384;
// Register split after setmaxnreg, together the 384 x 168 the block launches
// with: the fewest spills (-Xptxas -v: 8 or 16 bytes of stores, 32 or 40 in three
// of the four few-row forms).
template <int D> __host__ __device__ constexpr uint32_t regs_softmax() { return D == 128 ? 208u : 216u; }
template <int D> __host__ __device__ constexpr uint32_t regs_other() { return (kThreads * 168u - 256u * regs_softmax<D>()) / 128u; }
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleThreshold = 15.0f;   // log2 units; P <= 2^15 in 16 bits
// Every kGatherKeys / 64 halves a row's accumulator is added to fp32 sums in the
// workspace and starts again from zero: the tensor cores' own sums lose a part of
// a unit at every addition, always towards zero, 6e-9 of the result per key (whole
// walks over 2^18 and 2^20 keys were 1.6e-3 and 6.6e-3 too small).
constexpr int kGather = kGatherKeys / 64;
// Every kPolyEvery-th pair of exponentials is done on the FMA pipe: at 48 heads
// x 4608 and 6 x 16896 tokens every 8th pair took 886 and 1308 us, every 6th
// 880 and 1298, every 5th 887 and 1318, every 4th 896 and 1304; all on the
// exponential unit 3% more than every 8th.
constexpr int kPolyEvery = 6;

__host__ __device__ constexpr uint32_t col_s(int t, int buf) { return static_cast<uint32_t>(t * 128 + buf * 64); }
__host__ __device__ constexpr uint32_t col_o(int t) { return 256u + static_cast<uint32_t>(t) * 128u; }

template <int D>
struct Cfg {
  static constexpr int RB = D * 2;                    // row bytes
  static constexpr int NBOX = RB / 128;               // 128-byte swizzled boxes per tile
  static constexpr int BOXB = BM * 128;
  static constexpr int TB = BM * RB;
  static constexpr int KS = D == 128 ? 3 : 4;
  static constexpr int VS = D == 128 ? 3 : 4;
  static constexpr int EX = 4 * BM * 4;               // row sums and squares of both maps
  static constexpr int SLACK = 640;                   // to align the tiles to 1024 bytes
  static constexpr int SMEM = (1 + KS + VS) * TB + EX + 384 + SLACK;
};

// This CTA's run of the shared items' key tiles: from tile `off` of item
// `item` on, `count` tiles.
struct Share {
  long long item, count;
  int off;
};

struct __align__(8) Bars {
  uint64_t q_full, q_empty;
  uint64_t k_full[4], k_empty[4];
  uint64_t v_full[4], v_empty[4], v_ready[4];
  uint64_t s_full[2][2], p_full[2][2];                // [map][buffer]
  uint64_t exchange[3];
  uint64_t turn[2][4];                                // [map][warp]
  Share share;
  uint32_t tmem_base;
  uint32_t abort;
};
// Every lane waits; the warp goes on together, or not at all.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtl& ctl) {
  const bool ok = mbar_wait(bar, parity, ctl);
  return __all_sync(0xffffffffu, ok);
}
// An arrival by the lane with `lead` set, without a branch.
__device__ __forceinline__ void arrive_if(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];\n\t}\n"
      ::"r"(smem_u32(bar)), "r"(lead)
      : "memory");
}
// 32 TMEM columns per lane; tmem_wait_st waits for it.
__device__ __forceinline__ void tmem_st32_issue(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
               ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
               : "memory");
}
__device__ __forceinline__ void tmem_st16_issue(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
               ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
               : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
               "tcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr));
}
// The MMA and commit instructions by the lane with `lead` set.
__device__ __forceinline__ void mma_ss_if(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts_if(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n"
      ::"r"(smem_u32(bar)), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, const WaitCtl& ctl) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > ctl.limit_ns) {
      atomicOr(ctl.status, JATTN_DEV_TIMEOUT);
      return;
    }
  }
}
__device__ __forceinline__ void tma_load_4d(const CUtensorMap* map, uint64_t* bar, void* dst, int32_t c0, int32_t c1,
                                            int32_t c2, int32_t c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2),
        "r"(c3)
      : "memory");
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack_x2(float a, float b) {
  if constexpr (BF16) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  } else {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Two exponentials on the FMA pipe: 2^x = 2^n 2^f, n the nearest integer (by
// adding and subtracting 1.5 * 2^23, whose low bits then hold n), f in [-1/2,
// 1/2], 2^f by the degree-4 polynomial with value 1 at 0 that minimises the
// largest relative error there (2.8e-6; coefficients by iteratively
// reweighted least squares), n added to the exponent bits.  x is clamped at
// -127, where the result is exactly 0.  NaN does not survive the bit
// arithmetic: the caller sees to it.
__device__ __forceinline__ float2 ex2_poly(float2 x) {
  x = make_float2(fmaxf(x.x, -127.f), fmaxf(x.y, -127.f));
  const float2 magic = make_float2(12582912.f, 12582912.f);
  const float2 t = __fadd2_rn(x, magic);
  const float2 n = __fadd2_rn(t, make_float2(-12582912.f, -12582912.f));
  const float2 f = __ffma2_rn(n, make_float2(-1.f, -1.f), x);
  float2 q = __ffma2_rn(f, make_float2(0x1.3a02ccp-7f, 0x1.3a02ccp-7f), make_float2(0x1.c9fc46p-5f, 0x1.c9fc46p-5f));
  q = __ffma2_rn(q, f, make_float2(0x1.ec0378p-3f, 0x1.ec0378p-3f));
  q = __ffma2_rn(q, f, make_float2(0x1.62e12cp-1f, 0x1.62e12cp-1f));
  q = __ffma2_rn(q, f, make_float2(1.f, 1.f));
  return make_float2(__uint_as_float(__float_as_uint(q.x) + (__float_as_uint(t.x) << 23)),
                     __uint_as_float(__float_as_uint(q.y) + (__float_as_uint(t.y) << 23)));
}
// NaN if any value is one (max.f32 alone would drop it).
__device__ __forceinline__ float row_max(const float (&v)[64]) {
  float a[21];
#pragma unroll
  for (int i = 0; i < 21; ++i) a[i] = max3(v[3 * i], v[3 * i + 1], v[3 * i + 2]);
  float c[7];
#pragma unroll
  for (int i = 0; i < 7; ++i) c[i] = max3(a[3 * i], a[3 * i + 1], a[3 * i + 2]);
  return max3(max3(c[0], c[1], c[2]), max3(c[3], c[4], c[5]), max3(c[6], v[63], v[63]));
}

// Keys of batch entry b (the length clamped into the cache).
__device__ __forceinline__ int key_count(const DiffParams& p, int b) {
  return p.kv_len != nullptr ? min(max(__ldg(p.kv_len + b), 0), p.S_kv) : p.S_kv;
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// Exponent e of the power of two that V is divided by before it is rounded to
// fp16, from the bits of its largest finite magnitude: brings that into
// [2^14, 2^15), so that values down to 2^-29 of it keep all their bits.
// Clamped so that 2^e and 2^-e are normal fp32 numbers.
__device__ __forceinline__ int v_exponent(uint32_t amax_bits) {
  return amax_bits == 0u ? 0 : min(max(static_cast<int>(amax_bits >> 23) - 127 - 14, -126), 126);
}

template <int E>
struct alignas(4 * E) Vec4or2 {
  float e[E];
};

// Of 16 or 32.
template <int N>
__device__ __forceinline__ float row_max(const float (&v)[N]) {
  float a[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
  for (int i = 4; i < N; i += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k) a[k] = max3(a[k], v[i + k], v[i + 4 < N ? i + 4 + k : i + k]);
  return max3(max3(a[0], a[1], a[2]), a[3], a[3]);
}

// V's largest finite magnitude per (batch entry, K/V head) over its allowed
// keys, then its fp16 copy, zeros at masked keys: 8 channels of a row per
// thread and step, blockIdx.y = the head, kConvRows rows per block.
constexpr int kConvRows = 128;
template <int D, bool CONVERT>
__global__ void __launch_bounds__(256) widen_v_kernel(const DiffParams p) {
  constexpr int TPR = D / 8;
  const int bh = blockIdx.y, b = bh / p.H_kv, h = bh % p.H_kv;
  const int len = key_count(p, b);
  const int c = threadIdx.x % TPR * 8;
  const __nv_bfloat16* v = p.v + b * p.v_stride[0] + h * p.v_stride[1] + c;
  const float f = CONVERT ? pow2(-v_exponent(p.v_amax[bh])) : 1.f;
  uint32_t most = 0u;
#pragma unroll 4
  for (int i = threadIdx.x / TPR; i < kConvRows; i += 256 / TPR) {
    const int s = blockIdx.x * kConvRows + i;
    if (s >= p.S_kv) break;
    const bool in = s < len && (p.key_mask == nullptr || __ldg(p.key_mask + static_cast<size_t>(b) * p.S_kv + s) != 0);
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (in) x = __ldg(reinterpret_cast<const uint4*>(v + static_cast<int64_t>(s) * p.v_stride[2]));
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if constexpr (CONVERT) {
      uint32_t y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        y[j] = pack_x2<false>(__uint_as_float(w[j] << 16) * f, __uint_as_float(w[j] & 0xFFFF0000u) * f);
      *reinterpret_cast<uint4*>(p.v16 + (static_cast<size_t>(bh) * p.S_kv + s) * D + c) = make_uint4(y[0], y[1], y[2], y[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = (w[j] << 16) & 0x7FFF0000u, hi = w[j] & 0x7FFF0000u;
        if (lo < 0x7F800000u) most = max(most, lo);
        if (hi < 0x7F800000u) most = max(most, hi);
      }
    }
  }
  if constexpr (!CONVERT) {
    most = __reduce_max_sync(0xffffffffu, most);
    if ((threadIdx.x & 31) == 0 && most != 0u) atomicMax(p.v_amax + bh, most);
  }
}

// lambda of one head, fp32 sums of the two dot products.
__device__ __forceinline__ float lambda_of(const DiffParams& p, int head, int dm) {
  const size_t plane = static_cast<size_t>(p.H) * dm;
  const float* a = p.lam + static_cast<size_t>(head) * dm;
  float s1 = 0.f, s2 = 0.f;
  for (int i = 0; i < dm; i += 4) {
    const float4 x = *reinterpret_cast<const float4*>(a + i);
    const float4 y = *reinterpret_cast<const float4*>(a + plane + i);
    const float4 z = *reinterpret_cast<const float4*>(a + 2 * plane + i);
    const float4 w = *reinterpret_cast<const float4*>(a + 3 * plane + i);
    s1 += x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
    s2 += z.x * w.x + z.y * w.y + z.z * w.z + z.w * w.w;
  }
  return expf(s1) - expf(s2) + p.lambda_init;
}

// The same by a whole warp.
__device__ __forceinline__ float lambda_by_warp(const DiffParams& p, int head, int dm) {
  const int lane = threadIdx.x & 31;
  const size_t plane = static_cast<size_t>(p.H) * dm;
  float a1 = 0.f, a2 = 0.f;
  for (int i = lane; i < dm; i += 32) {
    const float* l = p.lam + static_cast<size_t>(head) * dm + i;
    a1 = fmaf(l[0], l[plane], a1);
    a2 = fmaf(l[2 * plane], l[3 * plane], a2);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a1 += __shfl_xor_sync(0xffffffffu, a1, o);
    a2 += __shfl_xor_sync(0xffffffffu, a2, o);
  }
  return expf(a1) - expf(a2) + p.lambda_init;
}

// a / b of non-negative numbers, almost always small ones (64-bit divisions
// cost a microsecond each few).
__device__ __forceinline__ long long divide(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}
// Key tiles of an item of batch entry b; an empty one counts as one tile, so
// that some CTA writes its zeros.
__device__ __forceinline__ int tiles_of(const DiffParams& p, int b) { return max((key_count(p, b) + BN - 1) / BN, 1); }
// Tiles of the shared items (numbers >= p.items_whole) of batch entry b.
__device__ __forceinline__ long long shared_tiles(const DiffParams& p, int b) {
  const long long per = static_cast<long long>(p.n_groups) * p.n_rt, lo = b * per;
  const long long from = max(lo, p.items_whole);
  return lo + per <= from ? 0 : (lo + per - from) * tiles_of(p, b);
}
// A whole warp: the sum of shared_tiles over the first nb batch entries.
__device__ __forceinline__ long long shared_prefix(const DiffParams& p, int nb) {
  long long t = 0;
  for (int b = threadIdx.x & 31; b < nb; b += 32) t += shared_tiles(p, b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return t;
}
// A whole warp: the item that holds tile g of the shared items, and g's place
// in it.
__device__ __forceinline__ void locate(const DiffParams& p, long long g, long long& item, int& off) {
  const int lane = threadIdx.x & 31;
  int b = 0;
  for (int b0 = 0;; b0 += 32) {
    const long long mine = b0 + lane < p.B ? shared_tiles(p, b0 + lane) : 0;
    long long sum = mine;                               // inclusive, over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += t;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, g < sum);
    const long long before = sum - mine;
    if (past != 0) {
      const int l = __ffs(past) - 1;
      b = b0 + l;
      g -= __shfl_sync(0xffffffffu, before, l);
      break;
    }
    g -= __shfl_sync(0xffffffffu, sum, 31);
    if (b0 + 32 >= p.B) {                               // g past the end: not called so
      b = p.B - 1;
      g = 0;
      break;
    }
  }
  const long long per = static_cast<long long>(p.n_groups) * p.n_rt;
  const int nt = tiles_of(p, b);
  const long long n = divide(g, nt);
  item = max(b * per, p.items_whole) + n;
  off = static_cast<int>(g - n * nt);
}
// The `total` shared tiles in equal runs, one more for the first CTAs.
struct Runs {
  long long q;
  int rem;
  __device__ __forceinline__ Runs(long long total, int ctas) : q(divide(total, ctas)), rem(static_cast<int>(total - q * ctas)) {}
  __device__ __forceinline__ long long start(int c) const { return c * q + min(c, rem); }
  // The CTA that has tile g.
  __device__ __forceinline__ int owner(long long g) const {
    const long long head = rem * (q + 1);
    return static_cast<int>(g < head ? divide(g, q + 1) : rem + divide(g - head, q));
  }
};

// A thread's row of the accumulator at `to` and its sums in the workspace, in
// units of 2^(its maximum then) with `any`, else none yet.  OUT: the accumulator
// is added to the sums and set to zero; otherwise the sums to the accumulator.
template <int D, bool OUT>
__device__ __forceinline__ void gather_row(const DiffParams& p, uint32_t to, float m_run, bool any) {
  const size_t at = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
  float* sums = p.sums + at * D;
  const float m = any ? p.sums_m[at] : -INFINITY;
  const float f = m == -INFINITY ? 0.f : ex2_approx(m - m_run);
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    uint32_t o[32];
    __syncwarp();
    tmem_ld32(to + c, o);
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      float4* dst = reinterpret_cast<float4*>(sums + c + e);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (any) x = *dst;
      x.x = fmaf(x.x, f, __uint_as_float(o[e]));
      x.y = fmaf(x.y, f, __uint_as_float(o[e + 1]));
      x.z = fmaf(x.z, f, __uint_as_float(o[e + 2]));
      x.w = fmaf(x.w, f, __uint_as_float(o[e + 3]));
      if constexpr (OUT) *dst = x;
      o[e] = OUT ? 0u : __float_as_uint(x.x);
      o[e + 1] = OUT ? 0u : __float_as_uint(x.y);
      o[e + 2] = OUT ? 0u : __float_as_uint(x.z);
      o[e + 3] = OUT ? 0u : __float_as_uint(x.w);
    }
    tmem_st32(to + c, o);
  }
  if constexpr (OUT) p.sums_m[at] = m_run;
}

// One piece of work: key tiles [t0, t0 + n_kv) of an item.
struct Segment {
  int b, gi, rt, len, t0, n_kv, n_half;
  bool whole, from_start;        // all of the item's tiles; starts with its first
};
__device__ __forceinline__ Segment segment_of(const DiffParams& p, long long item, int t0, int n, int nt) {
  Segment s;
  const int g = static_cast<int>(divide(item, p.n_rt));
  s.rt = static_cast<int>(item - static_cast<long long>(g) * p.n_rt);
  s.gi = g % p.n_groups;
  s.b = g / p.n_groups;
  s.len = key_count(p, s.b);
  s.t0 = t0;
  s.n_kv = s.len > 0 ? n : 0;
  // a last tile of at most 64 keys is one half
  s.n_half = 2 * s.n_kv - (s.n_kv > 0 && s.len - (t0 + n - 1) * BN <= 64 ? 1 : 0);
  s.whole = n == nt;
  s.from_start = t0 == 0;
  return s;
}
// This CTA's work in order: whole items first, then its share of the others.
struct Walk {
  long long item, left;
  int off;
  bool whole;
  __device__ __forceinline__ Walk(const DiffParams& p, const Share& s) {
    whole = blockIdx.x < p.items_whole;
    item = whole ? blockIdx.x : s.item;
    left = s.count;
    off = whole ? 0 : s.off;
  }
  __device__ __forceinline__ bool next(const DiffParams& p, const Share& share, Segment& s) {
    if (!whole && left <= 0) return false;
    const int nt = tiles_of(p, static_cast<int>(divide(item, p.n_groups * p.n_rt)));
    const int n = whole ? nt : static_cast<int>(min(static_cast<long long>(nt - off), left));
    s = segment_of(p, item, off, n, nt);
    if (whole) {
      item += gridDim.x;
      if (item >= p.items_whole) {
        whole = false;
        item = share.item;
        off = share.off;
      }
    } else {
      left -= n;
      off = 0;
      ++item;
    }
    return true;
  }
};

// KIND: the operands' types and how P keeps its precision.  P in bf16 alone
// costs the output 1.9e-3 (relative, N(0, 1) inputs), more than the bf16
// output's own rounding, because the difference of the maps cancels.
enum : int {
  kF16 = 0,        // fp16 operands, P in fp16
  kBf16WideV = 1,  // bf16 Q and K; V converted to fp16 (scaled by a power of two per head), P in fp16
  kBf16Split = 2,  // bf16 operands, P as the sum of two bf16: twice the P.V products, no second copy of V
};

// QUAD: a range of at most 32 rows (a few queries, one each in the single-token
// form).  They stand four times in the Q tile, once in each quarter of 32 TMEM
// lanes, so that the softmax of a half's 64 keys is spread over the four warps
// of its map: each takes its columns of S, puts its P there and zeros in the
// other columns of its rows, and has running maxima, sums and accumulator rows
// of its own, which meet at the segment's end.  With kBf16Split two warps take
// 32 columns each, and two more the same columns for P's low parts (one P.V
// product instead of two); with kF16 each takes 16.  One warp per map and part
// took 1340 of the 1550 clocks of a half, and bounded the walk at 5.4 TB/s.
//
// LONG: S_kv > kGatherKeys, the walk that empties its accumulators on the way: a
// kernel of its own, because the branch alone cost the shorter walks 4 to 8% and
// these take 4% longer (148 row tiles over 2^18 keys: 3.62 -> 3.78 ms).
template <int D, int KIND, bool QUAD, bool LONG>
__global__ void __launch_bounds__(kThreads, 1)
diff_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const DiffParams p) {
  using C = Cfg<D>;
  constexpr int DM = D / 2;
  constexpr bool QK_BF16 = KIND != kF16, PV_BF16 = KIND == kBf16Split;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t skew = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  if (skew > static_cast<uint32_t>(C::SLACK)) {       // uniform; the layout gives no such base
    if (threadIdx.x == 0) atomicOr(p.status, JATTN_DEV_CHECK);
    return;
  }
  uint8_t* sQ = smem_raw + skew;
  uint8_t* sK = sQ + C::TB;
  uint8_t* sV = sK + C::KS * C::TB;
  float* sL = reinterpret_cast<float*>(sV + C::VS * C::TB);   // [2][BM] 1 / l
  float* sSq = sL + 2 * BM;                                   // [2][BM] sums of squares
  Bars* bar = reinterpret_cast<Bars*>(sSq + 2 * BM);
  static_assert(sizeof(Bars) <= 384, "room for the barriers");

  // from one lane, so that the compiler sees the roles' branches as uniform
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(&bar->q_full, 1);
    mbar_init(&bar->q_empty, 2);
    for (int s = 0; s < C::KS; ++s) {
      mbar_init(&bar->k_full[s], 1);
      mbar_init(&bar->k_empty[s], 2);
    }
    for (int s = 0; s < C::VS; ++s) {
      mbar_init(&bar->v_full[s], 1);
      mbar_init(&bar->v_empty[s], 2);
      mbar_init(&bar->v_ready[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bar->s_full[t][i], 1);
        mbar_init(&bar->p_full[t][i], BM / 32);
      }
      mbar_init(&bar->exchange[t], QUAD ? 8 : 2 * BM);
    }
    mbar_init(&bar->exchange[2], 8);
    for (int i = 0; i < 8; ++i) mbar_init(&bar->turn[0][i], 1);
    bar->abort = 0;
    fence_mbarrier_init();
  }
  if (warp == kMmaWarp) {
    __syncwarp();
    tmem_alloc(&bar->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  if (warp == kProducerWarp && lane < 3) tma_prefetch_desc(lane == 0 ? &tmQ : (lane == 1 ? &tmK : &tmV));
  if (warp == kShareWarp) {
    Share mine{0, 0, 0};
    if (p.items > p.items_whole) {
      const long long total = shared_prefix(p, p.B);
      const Runs runs(total, gridDim.x);
      const long long g0 = runs.start(blockIdx.x), g1 = runs.start(blockIdx.x + 1);
      mine.count = g1 - g0;
      if (g1 > g0) locate(p, g0, mine.item, mine.off);
    }
    if (lane == 0) bar->share = mine;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;
  const Share share = bar->share;
  // the merge may find its rows on idle SMs meanwhile
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const WaitCtl ctl{&bar->abort, p.status, p.timeout_ns};
  auto kv_head = [&](int gi) { return static_cast<int>(static_cast<long long>(gi) * p.H_kv / p.n_groups); };
  // V rows of masked keys have to be zeroed: a mask, or a length inside the
  // cache (rows past the cache arrive as zeros from TMA; the converted V has
  // its masked rows zeroed).  In such a call every V tile goes through the mask
  // warp and the products wait for v_ready, in segments without a masked key
  // too: v_full would let them release a stage that the mask warp has yet to
  // pass, and a parity wait that misses a phase takes the next one for it.
  const bool masks = KIND != kBf16WideV && (p.key_mask != nullptr || p.kv_len != nullptr);

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(regs_other<D>()));
    if (warp == kProducerWarp) {
      if (lane == 0) {
        int nq = 0, nk = 0;                             // Q tiles, key tiles (K and V) loaded so far
        bool v_behind = false;                          // the last key tile's V was not issued
        Segment s;
        bool ok = true;
        for (Walk walk(p, share); ok && walk.next(p, share, s);) {
          if (s.n_kv == 0) continue;
          // the Q buffer is free once the previous segment's Q.K^T are done
          if (nq > 0 && !mbar_wait(&bar->q_empty, (nq - 1) & 1, ctl)) break;
          // and, QUAD, once it has served that segment's epilogue
          if (QUAD && nq > 0 && !mbar_wait(&bar->exchange[2], (nq - 1) & 1, ctl)) break;
          mbar_arrive_expect_tx(&bar->q_full, C::TB);
          for (int x = 0; x < C::NBOX; ++x) {
            if constexpr (QUAD) {
              for (int k = 0; k < 4; ++k)
                tma_load_4d(&tmQ, &bar->q_full, sQ + x * C::BOXB + k * 32 * 128, x * 64, 0, s.gi, s.b);
            } else {
              tma_load_4d(&tmQ, &bar->q_full, sQ + x * C::BOXB, x * 64, s.rt * BM, s.gi, s.b);
            }
          }
          ++nq;
          const int kvh = kv_head(s.gi);
          for (int j = 0; j < s.n_kv; ++j, ++nk) {
            const int ks = nk % C::KS, vs = nk % C::VS;
            ok = mbar_wait(&bar->k_empty[ks], ((nk / C::KS) & 1) ^ 1, ctl);
            if (!ok) break;
            mbar_arrive_expect_tx(&bar->k_full[ks], C::TB);
            for (int x = 0; x < C::NBOX; ++x)
              tma_load_4d(&tmK, &bar->k_full[ks], sK + ks * C::TB + x * C::BOXB, x * 64, (s.t0 + j) * BN, kvh, s.b);
            ok = mbar_wait(&bar->v_empty[vs], ((nk / C::VS) & 1) ^ 1, ctl);
            if (!ok) {
              v_behind = true;
              ++nk;
              break;
            }
            mbar_arrive_expect_tx(&bar->v_full[vs], C::TB);
            for (int x = 0; x < C::NBOX; ++x)
              tma_load_4d(&tmV, &bar->v_full[vs], sV + vs * C::TB + x * C::BOXB, x * 64, (s.t0 + j) * BN, kvh, s.b);
          }
        }
        // every load issued must have landed before the CTA may exit
        if (nq > 0) drain_wait(&bar->q_full, (nq - 1) & 1, ctl);
        for (int i = max(nk - C::KS, 0); i < nk; ++i) drain_wait(&bar->k_full[i % C::KS], (i / C::KS) & 1, ctl);
        const int nv = nk - (v_behind ? 1 : 0);
        for (int i = max(nv - C::VS, 0); i < nv; ++i) drain_wait(&bar->v_full[i % C::VS], (i / C::VS) & 1, ctl);
      }
    } else if (warp == kMmaWarp || warp == kShareWarp) {
      const int t = warp == kMmaWarp ? 0 : 1;         // the map whose products this warp issues
      // The whole warp walks, one lane issues: the descriptors are then warp
      // uniform and live in uniform registers.  With one lane walking, each
      // MMA cost 72 clocks to issue (measured; its execution 48 or 64).
      const uint32_t lead = elect_one() ? 1u : 0u;
      const uint32_t idesc_qk = instr_desc(QK_BF16, QK_BF16, 0, BM, BN / 2);
      const uint32_t idesc_pv = instr_desc(PV_BF16, PV_BF16, 1, BM, D);
      const uint32_t sQa = smem_u32(sQ), sKa = smem_u32(sK), sVa = smem_u32(sV);
      // Descriptors differ in the address field alone (bits [0, 14), 16-byte
      // units; shared memory ends below 2^18), so one is another plus a
      // constant: the issuing thread's instructions are on the S -> P chain.
      const uint64_t qd0 = smem_desc(sQa, 16, 1024, 2u), kd0 = smem_desc(sKa, 16, 1024, 2u);
      const uint64_t vd0 = smem_desc(sVa, C::BOXB, 1024, 2u);
      // S of the map, keys [64 half, +64) of the K tile in stage ks
      auto issue_qk = [&](int ks, int half, int buf) {
        const uint64_t kd = kd0 + static_cast<uint32_t>(ks * (C::TB / 16) + half * (64 * 128 / 16));
#pragma unroll
        for (int kk = 0; kk < DM / 16; ++kk) {
          const uint32_t at = t * DM * 2 + kk * 32;          // byte of the row
          const uint32_t off = (at / 128 * C::BOXB + at % 128) / 16;
          mma_ss_if(lead, tmem + col_s(t, buf), qd0 + off, kd + off, idesc_qk, kk > 0);
        }
      };
      auto issue_pv = [&](int vs, int half, int buf, bool acc) {
        const uint64_t vd = vd0 + static_cast<uint32_t>(vs * (C::TB / 16) + half * (64 * 128 / 16));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ts_if(lead, tmem + col_o(t), tmem + col_s(t, buf) + kk * 8, vd + kk * 128, idesc_pv, acc || kk > 0);
        if constexpr (KIND == kBf16Split && !QUAD) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)                     // the low parts, in the columns behind
            mma_ts_if(lead, tmem + col_o(t), tmem + col_s(t, buf) + 32 + kk * 8, vd + kk * 128, idesc_pv, 1);
        }
      };
      int nq = 0, nk = 0, nv = 0;                     // segments, K tiles, V tiles so far
      uint32_t idx = 0, p_phase = 0;                  // S commits of the CTA; parity bits of p_full
      Segment s;
      bool ok = true;
      for (Walk walk(p, share); ok && walk.next(p, share, s);) {
        if (s.n_kv == 0) continue;
        const int n = s.n_half;
        ok = warp_wait(&bar->q_full, nq & 1, ctl) && warp_wait(&bar->k_full[nk % C::KS], (nk / C::KS) & 1, ctl);
        if (!ok) break;
        tc_fence_after();
        // Every S buffer hand-over is one commit: of halves 0 and 1 here,
        // of half i + 2 behind P.V of half i -- also where there is no such
        // half, so that S commit n + 1 proves the last P.V done.
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i < n) issue_qk(nk % C::KS, i, (idx + i) & 1);
          commit_if(lead, &bar->s_full[t][(idx + i) & 1]);
        }
        commit_if(lead, &bar->k_empty[nk % C::KS]);
        ++nk;
        if (n <= 2) commit_if(lead, &bar->q_empty);
        int vs = nv % C::VS, ks = nk % C::KS;
        uint32_t v_par = (nv / C::VS) & 1, k_par = (nk / C::KS) & 1;
#pragma unroll 1
        for (int i = 0; i < n && ok; ++i) {
          const int buf = (idx + i) & 1, half = i & 1;
          const bool more = i + 2 < n, v_last = half || i + 1 == n;
          if (!half) {
            ok = warp_wait(masks ? &bar->v_ready[vs] : &bar->v_full[vs], v_par, ctl) &&
                 (!more || warp_wait(&bar->k_full[ks], k_par, ctl));
            if (!ok) break;
          }
          ok = warp_wait(&bar->p_full[t][buf], (p_phase >> buf) & 1, ctl);
          if (!ok) break;
          tc_fence_after();
          issue_pv(vs, half, buf, i > 0);
          if (more) issue_qk(ks, half, buf);
          commit_if(lead, &bar->s_full[t][buf]);
          p_phase ^= 1u << buf;
          if (v_last) {
            commit_if(lead, &bar->v_empty[vs]);
            ++nv;
            if (++vs == C::VS) { vs = 0; v_par ^= 1; }
          }
          if (more && (half || i + 3 == n)) {         // the K tile's last half
            commit_if(lead, &bar->k_empty[ks]);
            ++nk;
            if (++ks == C::KS) { ks = 0; k_par ^= 1; }
          }
          if (i + 3 == n) commit_if(lead, &bar->q_empty);  // the segment's last Q.K^T
        }
        idx += n + 2;
        ++nq;
      }
      // the softmax warps wait for the last S commit of every segment; an
      // aborted walk gives the products in flight time to end
      if (*ctl.abort) {
        const uint64_t t = globaltimer_ns();
        while (globaltimer_ns() - t < 1000000ull) {
        }
      }
    } else if (warp == kMaskWarp) {
      if constexpr (KIND != kBf16WideV) {
        if (masks) {
          int nv = 0;
          Segment s;
          bool ok = true;
          for (Walk walk(p, share); ok && walk.next(p, share, s);) {
            const bool fix = p.key_mask != nullptr || s.len < p.S_kv;
            const uint8_t* mask = p.key_mask != nullptr ? p.key_mask + static_cast<size_t>(s.b) * p.S_kv : nullptr;
            for (int j = 0; j < s.n_kv; ++j, ++nv) {
              const int vs = nv % C::VS, key0 = (s.t0 + j) * BN;
              if (!fix) {
                // no masked key in this segment
                ok = warp_wait(&bar->v_full[vs], (nv / C::VS) & 1, ctl);
                if (!ok) break;
                if (lane == 0) mbar_arrive(&bar->v_ready[vs]);
                continue;
              }
              bool drop[4];                                 // keys key0 + 32 w + lane
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const int key = key0 + 32 * w + lane;
                drop[w] = key < p.S_kv && (key >= s.len || (mask != nullptr && __ldg(mask + key) == 0));
              }
              ok = warp_wait(&bar->v_full[vs], (nv / C::VS) & 1, ctl);
              if (!ok) break;
              uint8_t* tile = sV + vs * C::TB;
              bool wrote = false;
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                uint32_t todo = __ballot_sync(0xffffffffu, drop[w]);
                wrote = wrote || todo != 0;
                // a row is 128 bytes of each box, wherever the swizzle put its pieces
                while (todo != 0) {
                  const int r = 32 * w + __ffs(todo) - 1;
                  todo &= todo - 1;
#pragma unroll
                  for (int x = 0; x < C::NBOX; ++x)
                    *reinterpret_cast<uint32_t*>(tile + x * C::BOXB + r * 128 + lane * 4) = 0u;
                }
              }
              if (wrote) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              __syncwarp();
              if (lane == 0) mbar_arrive(&bar->v_ready[vs]);
            }
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(regs_softmax<D>()));
    const int t = warp >> 2;                            // map of this warpgroup
    // QUAD: the key columns of a half that are this warp's, and whether it has P's low parts
    constexpr int NC = !QUAD ? 64 : (KIND == kBf16Split ? 32 : 16);
    const int group = !QUAD ? 0 : (KIND == kBf16Split ? warp & 1 : warp & 3);
    const bool lo_role = KIND == kBf16Split && QUAD && ((warp >> 1) & 1) != t;
    const int row = QUAD ? lane : (warp & 3) * 32 + lane;   // of the tile; TMEM lane (warp & 3) * 32 + lane
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t to = lane_base + col_o(t);
    const float c_j = p.scale_log2;
    constexpr int E = D / 32;                           // QUAD's epilogue: channels per lane
    const size_t rows = static_cast<size_t>(p.B) * p.H * p.S_q;
    uint32_t idx = 0, ex_phase = 0, turns = 0;
    uint32_t segments = 0, pass_phase = 0;              // QUAD: with keys, so far; parity of exchange[1]
    float norm_mine[E];                                 // QUAD: of channels lane * E on
    if constexpr (QUAD) {
#pragma unroll
      for (int e = 0; e < E; ++e) norm_mine[e] = p.norm_w != nullptr ? __ldg(p.norm_w + lane * E + e) : 1.f;
    }
    Segment s;
    bool ok = true;
    for (Walk walk(p, share); ok && walk.next(p, share, s);) {
      const uint8_t* mask = p.key_mask != nullptr ? p.key_mask + static_cast<size_t>(s.b) * p.S_kv : nullptr;
      const int r = s.rt * BM + row;                    // row of the range
      const bool live = r < p.R;
      const bool warp_live = QUAD || s.rt * BM + (warp & 3) * 32 < p.R;
      const int head = s.gi * p.hpg + (live ? r / p.S_q : 0), s_q = live ? r % p.S_q : 0;
      const int n = s.n_half, key0 = s.t0 * BN;
      // needed at the end; read while the first tiles are on their way
      float lam = 0.f;
      if constexpr (QUAD) {
        if (s.whole && warp < p.R) lam = lambda_by_warp(p, s.gi * p.hpg + warp / p.S_q, DM);
      } else {
        if (s.whole && live) lam = lambda_of(p, head, DM);
      }
      float m_run = -INFINITY, l_run = 0.f;
      constexpr int MW = QUAD ? 1 : 2;
      uint8_t mb[MW];
      auto load_mask = [&](int i) {
#pragma unroll
        for (int w = 0; w < MW; ++w) {
          const int key = key0 + i * 64 + group * NC + 32 * w + lane;
          mb[w] = key < p.S_kv ? __ldg(mask + key) : 0;
        }
      };
      if (mask != nullptr && n > 0) load_mask(0);
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const uint32_t at = idx + i, buf = at & 1;
        uint32_t keep[MW];
#pragma unroll
        for (int w = 0; w < MW; ++w) keep[w] = ~0u;
        if (mask != nullptr) {
#pragma unroll
          for (int w = 0; w < MW; ++w) keep[w] = __ballot_sync(0xffffffffu, mb[w] != 0);
          if (i + 1 < n) load_mask(i + 1);
        }
        ok = warp_wait(&bar->s_full[t][buf], (at >> 1) & 1, ctl);
        if (!ok) break;
        if (!warp_live) {                               // rows past the last: nothing to compute
          arrive_if(lane == 0, &bar->p_full[t][buf]);
          continue;
        }
        tc_fence_after();
        const uint32_t ts = lane_base + col_s(t, buf);
        float v[NC];
        {
          uint32_t raw[NC];
          if constexpr (NC == 64) tmem_ld64(ts, raw);
          else if constexpr (NC == 32) tmem_ld32(ts + group * NC, raw);
          else tmem_ld16(ts + group * NC, raw);
#pragma unroll
          for (int e = 0; e < NC; ++e) v[e] = __uint_as_float(raw[e]);
        }
        const int valid = s.len - key0 - i * 64 - group * NC;
        if (valid < NC) {
#pragma unroll
          for (int e = 0; e < NC; ++e)
            if (e >= valid) v[e] = -INFINITY;
        }
        if ((keep[0] & keep[MW - 1]) != ~0u) {
#pragma unroll
          for (int e = 0; e < NC; ++e)
            if (!((keep[e >> 5] >> (e & 31)) & 1u)) v[e] = -INFINITY;
        }
        const float mx = row_max(v) * c_j;
        const float m_new = fmaxf(m_run, mx);
        float alpha = 1.f;
        const bool resc = (m_new - m_run) > kRescaleThreshold;
        if (resc) {
          alpha = ex2_approx(m_run - m_new);
          m_run = m_new;
          l_run *= alpha;
        }
        __syncwarp();
        if (i > 0 && __any_sync(0xffffffffu, resc)) {
          // S commit i + 1 proves P.V of half i - 1 done: O_t is stable until
          // this half's P is handed over
          ok = warp_wait(&bar->s_full[t][buf ^ 1], ((at + 1) >> 1) & 1, ctl);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(to + c * 32, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(to + c * 32, o);
          }
        }
        if (LONG && i > 0 && i % kGather == 0) {
          ok = warp_wait(&bar->s_full[t][buf ^ 1], ((at + 1) >> 1) & 1, ctl);
          if (!ok) break;
          tc_fence_after();
          gather_row<D, true>(p, to, m_run, i > kGather);
        }
        // The two warps of a scheduler (map 0's and map 1's of the same rows)
        // take the exponential unit in turns: left to themselves they fall into
        // step, want it at the same time and leave it idle at the same time.
        if constexpr (!QUAD) {
          ok = warp_wait(&bar->turn[t][warp & 3], (turns ^ (t ^ 1)) & 1, ctl);
          if (!ok) break;
          ++turns;
        }
        // no key so far: every probability is exp2(-inf) = 0
        const float neg_m = m_run == -INFINITY ? 0.f : -m_run;
        const float2 c2 = make_float2(c_j, c_j), nm2 = make_float2(neg_m, neg_m);
        float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
        uint32_t pk[NC / 2], lo[KIND == kBf16Split ? NC / 2 : 1];
#pragma unroll
        for (int c = 0; c < NC / 2; ++c) {
          const float2 x = __ffma2_rn(make_float2(v[2 * c], v[2 * c + 1]), c2, nm2);
          const float2 e = c % kPolyEvery == kPolyEvery - 1 ? ex2_poly(x) : make_float2(ex2_approx(x.x), ex2_approx(x.y));
          if (c & 1) acc1 = __fadd2_rn(acc1, e);
          else acc0 = __fadd2_rn(acc0, e);
          // P in V's type (the MMA wants one type); l sums the unrounded values
          pk[c] = pack_x2<PV_BF16>(e.x, e.y);
          if constexpr (KIND == kBf16Split)
            lo[c] = pack_x2<true>(e.x - __uint_as_float(pk[c] << 16), e.y - __uint_as_float(pk[c] & 0xFFFF0000u));
        }
        if constexpr (!QUAD) {
          tmem_st32_issue(ts, pk);
          if constexpr (KIND == kBf16Split) tmem_st32_issue(ts + 32, lo);
        } else if constexpr (KIND == kBf16Split) {
          uint32_t zero[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            pk[c] = lo_role ? lo[c] : pk[c];
            zero[c] = 0u;
          }
          tmem_st16_issue(ts + group * 16, pk);
          tmem_st16_issue(ts + (group ^ 1) * 16, zero);
        } else {
          uint32_t all[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) all[c] = c / 8 == group ? pk[c % 8] : 0u;
          tmem_st32_issue(ts, all);
        }
        // passed earlier, among the last exponentials, it cost 3%
        if constexpr (!QUAD) arrive_if(lane == 0, &bar->turn[t ^ 1][warp & 3]);
        tmem_wait_st();
        l_run += (acc0.x + acc0.y) + (acc1.x + acc1.y);
        // NaN in, NaN out, and so for a logit of +inf
        if (!(mx < INFINITY)) l_run = __int_as_float(0x7FFFFFFF);
        // one arrival per warp: 128 to one address take turns
        tc_fence_before();
        __syncwarp();
        arrive_if(lane == 0, &bar->p_full[t][buf]);
      }
      if (!ok) break;
      if (n > 0) {
        ok = warp_wait(&bar->s_full[t][(idx + n + 1) & 1], ((idx + n + 1) >> 1) & 1, ctl);
        if (!ok) break;
        idx += n + 2;
      }
      tc_fence_after();
      if (LONG && n > kGather && warp_live) gather_row<D, false>(p, to, m_run, true);
      if constexpr (QUAD) {
        if (n == 0) {                                   // no key: zeros
          for (int q = warp; q < p.R; q += 8) {
            const int h = s.gi * p.hpg + q / p.S_q;
            const size_t at = (static_cast<size_t>(s.b) * p.H + h) * p.S_q + q % p.S_q;
            uint32_t* dst = reinterpret_cast<uint32_t*>(
                p.o + ((static_cast<size_t>(s.b) * p.S_q + q % p.S_q) * p.H + h) * D) + lane * (E / 2);
#pragma unroll
            for (int e = 0; e < E / 2; ++e) dst[e] = 0u;
            if (p.lse != nullptr && lane < 2) p.lse[lane * rows + at] = -INFINITY;
          }
          continue;
        }
        // Every quarter of the TMEM lanes has its keys' part of every row.
        // They meet in the Q tile's memory, [map][quarter][row][channel], eight
        // rows at a time: warp w adds up row w of them.  The tile's last use
        // has to be over for both maps; the producer loads it again after
        // exchange[2].
        ok = warp_wait(&bar->q_empty, segments & 1, ctl);
        if (!ok) break;
        float* meet = reinterpret_cast<float*>(sQ);
        float2* sums = reinterpret_cast<float2*>(sL);   // [map][quarter][row]: maximum and sum
        for (int r0 = 0; r0 < p.R; r0 += 8) {
          const int mine = lane - r0;                   // this lane's row of the eight
          if (r0 > 0) {
            if (s.whole && r0 + warp < p.R) lam = lambda_by_warp(p, s.gi * p.hpg + (r0 + warp) / p.S_q, DM);
            __syncwarp();
            arrive_if(lane == 0, &bar->exchange[1]);
            ok = warp_wait(&bar->exchange[1], pass_phase, ctl);
            if (!ok) break;
            pass_phase ^= 1u;
          }
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t x[32];
            __syncwarp();
            tmem_ld32(to + c, x);
            // channel quads at [quad ^ row]: eight rows of one quad share no bank
            if (mine >= 0 && mine < 8) {
              uint4* at = reinterpret_cast<uint4*>(meet + (warp * 8 + mine) * D);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                at[(c / 4 + e) ^ mine] = make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
            }
          }
          if (mine >= 0 && mine < 8) sums[warp * 8 + mine] = make_float2(m_run, l_run);
          __syncwarp();
          arrive_if(lane == 0, &bar->exchange[0]);
          ok = warp_wait(&bar->exchange[0], ex_phase, ctl);
          if (!ok) break;
          ex_phase ^= 1u;
          const int q = r0 + warp;
          if (q >= p.R) continue;
          float out[2][E], lse2[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float2 ml[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) ml[k] = sums[(u * 4 + k) * 8 + warp];
            const float m = fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
            float l = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) out[u][e] = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float w = ml[k].x == -INFINITY ? 0.f : ex2_approx(ml[k].x - m);
              // with P in two parts, quarters 2 u and 2 u + 1 have the first ones and the sums
              if (KIND != kBf16Split || k / 2 == u) l = fmaf(w, ml[k].y, l);
              const float* at = meet + ((u * 4 + k) * 8 + warp) * D + (((lane * E) / 4) ^ warp) * 4 + lane * E % 4;
              if (w == 0.f && ml[k].y == 0.f) continue; // no key of this quarter
#pragma unroll
              for (int e = 0; e < E; ++e) out[u][e] = fmaf(w, at[e], out[u][e]);
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
            lse2[u] = l == 0.f ? -INFINITY : m + __log2f(l);
#pragma unroll
            for (int e = 0; e < E; ++e) out[u][e] *= inv;
          }
          if (!s.whole) {
            // this part's normalised output and log-sum-exp of each map
            const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (s.from_start ? 1 : 0);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              float* dst = p.part_o + ((slot * 2 + u) * BM + q) * D + lane * E;
#pragma unroll
              for (int e = 0; e < E; ++e) dst[e] = out[u][e];
              if (lane == 0) p.part_l[(slot * 2 + u) * BM + q] = lse2[u];
            }
            continue;
          }
          const int h = s.gi * p.hpg + q / p.S_q;
          float y[E], sq = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            y[e] = fmaf(-lam, out[1][e], out[0][e]);
            sq = fmaf(y[e], y[e], sq);
          }
          if (p.norm_w != nullptr) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
            const float f = rsqrtf(sq * (1.f / D) + p.eps) * (1.f - p.lambda_init);
#pragma unroll
            for (int e = 0; e < E; ++e) y[e] *= f * norm_mine[e];
          }
          uint32_t* dst = reinterpret_cast<uint32_t*>(
              p.o + ((static_cast<size_t>(s.b) * p.S_q + q % p.S_q) * p.H + h) * D) + lane * (E / 2);
#pragma unroll
          for (int e = 0; e < E / 2; ++e) dst[e] = pack_x2<true>(y[2 * e], y[2 * e + 1]);
          if (p.lse != nullptr && lane < 2)
            p.lse[lane * rows + (static_cast<size_t>(s.b) * p.H + h) * p.S_q + q % p.S_q] =
                (lane == 0 ? lse2[0] : lse2[1]) * 0.69314718055994531f;
        }
        if (!ok) break;
        ++segments;
        tc_fence_before();                              // before the next segment's P.V overwrites O_t
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        arrive_if(lane == 0, &bar->exchange[2]);
        continue;
      }
      float inv = l_run == 0.f ? 0.f : 1.f / l_run;
      if constexpr (KIND == kBf16WideV)                 // undo V's power of two
        inv *= pow2(v_exponent(__ldg(p.v_amax + static_cast<size_t>(s.b) * p.H_kv + kv_head(s.gi))));
      const float lse2 = l_run == 0.f ? -INFINITY : m_run + __log2f(l_run);
      if (!s.whole) {
        // this part's normalised output and log-sum-exp of its map
        const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (s.from_start ? 1 : 0);
        if (warp_live) {
          float* dst = p.part_o + ((slot * 2 + t) * BM + row) * D;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            __syncwarp();
            tmem_ld32(to + c, o);
            if (live) {
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
#pragma unroll
              for (int e = 0; e < 32; e += 8)           // whole 32-byte sectors of the thread's row
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                             ::"l"(dst + c + e), "r"(o[e]), "r"(o[e + 1]), "r"(o[e + 2]), "r"(o[e + 3]), "r"(o[e + 4]),
                               "r"(o[e + 5]), "r"(o[e + 6]), "r"(o[e + 7])
                             : "memory");
            }
          }
          if (live) p.part_l[(slot * 2 + t) * BM + row] = lse2;
        }
        tc_fence_before();                              // before the next segment's P.V overwrites O_t
        continue;
      }
      __nv_bfloat16* o_row = p.o + ((static_cast<size_t>(s.b) * p.S_q + s_q) * p.H + head) * D;
      float* lse_row = p.lse != nullptr && live
                           ? p.lse + static_cast<size_t>(t) * rows + (static_cast<size_t>(s.b) * p.H + head) * p.S_q + s_q
                           : nullptr;
      sL[t * BM + row] = inv;
      tc_fence_before();
      mbar_arrive(&bar->exchange[0]);
      ok = warp_wait(&bar->exchange[0], ex_phase, ctl);
      if (!ok) break;
      tc_fence_after();
      // channels [t * D / 2, +D / 2) of the row
      const float w1 = sL[row], w2 = -lam * sL[BM + row];
      float o[DM];
      float sq = 0.f;
      if (n > 0) {
        const uint32_t o1 = lane_base + col_o(0) + t * DM, o2 = lane_base + col_o(1) + t * DM;
#pragma unroll
        for (int c = 0; c < DM; c += 32) {
          uint32_t x[32], y[32];
          tmem_ld32(o1 + c, x);
          tmem_ld32(o2 + c, y);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            o[c + e] = fmaf(__uint_as_float(x[e]), w1, __uint_as_float(y[e]) * w2);
            sq = fmaf(o[c + e], o[c + e], sq);
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < DM; ++e) o[e] = 0.f;
      }
      // also the point after which neither O is read any more
      sSq[t * BM + row] = sq;
      tc_fence_before();
      mbar_arrive(&bar->exchange[1]);
      ok = warp_wait(&bar->exchange[1], ex_phase, ctl);
      if (!ok) break;
      ex_phase ^= 1u;
      if (p.norm_w != nullptr) {
        const float f = rsqrtf((sSq[row] + sSq[BM + row]) * (1.f / D) + p.eps) * (1.f - p.lambda_init);
#pragma unroll
        for (int e = 0; e < DM; e += 4) {
          const float4 w = __ldg(reinterpret_cast<const float4*>(p.norm_w + t * DM + e));
          o[e] *= f * w.x;
          o[e + 1] *= f * w.y;
          o[e + 2] *= f * w.z;
          o[e + 3] *= f * w.w;
        }
      }
      if (live) {
        __nv_bfloat16* dst = o_row + t * DM;
        uint32_t w[DM / 2];
#pragma unroll
        for (int e = 0; e < DM / 2; ++e) w[e] = pack_x2<true>(o[2 * e], o[2 * e + 1]);
        if ((reinterpret_cast<uintptr_t>(p.o) & 31u) == 0) {
#pragma unroll
          for (int e = 0; e < DM / 2; e += 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                         ::"l"(dst + 2 * e), "r"(w[e]), "r"(w[e + 1]), "r"(w[e + 2]), "r"(w[e + 3]), "r"(w[e + 4]),
                           "r"(w[e + 5]), "r"(w[e + 6]), "r"(w[e + 7])
                         : "memory");
        } else {
#pragma unroll
          for (int e = 0; e < DM / 2; e += 4)
            *reinterpret_cast<uint4*>(dst + 2 * e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
        }
        if (lse_row != nullptr) *lse_row = lse2 * 0.69314718055994531f;
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Merge of the items that several CTAs shared: each map's parts weighted by
// 2^(lse_part - lse), then the difference and the norm.  blockIdx.x + 1 = a CTA
// of the walk; the first whose share starts inside an item answers for that
// item.  WPR warps per query row take the parts in turns (a single-token call
// has few rows and up to a part per CTA, the tail of a long prompt many rows
// of two or three parts); sums in a fixed order.
constexpr int kMergeParts = 4;                          // loads in flight per warp and map
template <int D, int WPR>
__global__ void __launch_bounds__(128) diff_merge_kernel(const DiffParams p, int ctas) {
  constexpr int E = D / 32;                             // channels per lane
  using Chunk = Vec4or2<E>;
  __shared__ float sums[4][2][D + 1];                   // [warp][map]: weighted outputs, weights
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % WPR;
  const int row = (blockIdx.y * 4 + warp) / WPR;
  const int cta = blockIdx.x + 1;
  const long long total = shared_prefix(p, p.B);
  const Runs runs(total, ctas);
  const long long g = runs.start(cta);
  long long item = 0;
  int off = 0;
  if (g < total) locate(p, g, item, off);
  const bool first = off > 0 && runs.start(cta - 1) <= g - off;
  const int range = static_cast<int>(divide(item, p.n_rt)), b = range / p.n_groups, gi = range % p.n_groups;
  const int r = static_cast<int>(item - static_cast<long long>(range) * p.n_rt) * BM + row;
  const bool work = first && r < p.R;
  // the last CTA that has a part of the item, by its last tile
  const int parts = work ? runs.owner(g - off + tiles_of(p, b) - 1) - cta + 2 : 0;
  const int head = work ? gi * p.hpg + r / p.S_q : 0, s_q = work ? r % p.S_q : 0;
  const size_t rows = static_cast<size_t>(p.B) * p.H * p.S_q;
  const size_t rg = (static_cast<size_t>(b) * p.H + head) * p.S_q + s_q;
  const float lam = lambda_by_warp(p, head, D / 2);
  float norm[E];
#pragma unroll
  for (int e = 0; e < E; ++e) norm[e] = p.norm_w != nullptr ? __ldg(p.norm_w + lane * E + e) : 1.f;
  // Everything above is the inputs' alone; the parts from here on.  Every block
  // waits for the walk, also one without work: this grid's end has to mean the
  // walk's end for what the stream holds next.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!work) return;                                    // WPR 4: the whole block
  // part 0 is the end of CTA cta - 1's share, part i the start of cta + i - 1's
  auto part_at = [&](int i, int t) {
    const size_t slot = i == 0 ? 2 * static_cast<size_t>(cta - 1) + 1 : 2 * static_cast<size_t>(cta + i - 1);
    return (slot * 2 + t) * BM + row;
  };
  Chunk x[kMergeParts][2];
  float l[kMergeParts][2];
  auto load = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kMergeParts; ++k)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const size_t at = part_at(min(i0 + k * WPR, parts - 1), t);
        l[k][t] = p.part_l[at];
        x[k][t] = *reinterpret_cast<const Chunk*>(p.part_o + at * D + lane * E);
      }
  };
  load(sub);                                            // on its way under the maxima's
  float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    for (int i = lane; i < parts; i += 32) {
      const float m = p.part_l[part_at(i, t)];
      mx[t] = m > mx[t] || m != m ? m : mx[t];          // a NaN stays
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float m = __shfl_xor_sync(0xffffffffu, mx[t], o);
      mx[t] = m > mx[t] || m != m ? m : mx[t];
    }
  }
  float acc[2][E], tot[2] = {0.f, 0.f};
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int e = 0; e < E; ++e) acc[t][e] = 0.f;
  for (int i0 = sub;;) {
#pragma unroll
    for (int k = 0; k < kMergeParts; ++k)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        // a part without keys, or no part: weight 0, and its output may be unwritten
        if (i0 + k * WPR >= parts || l[k][t] == -INFINITY) continue;
        const float w = ex2_approx(l[k][t] - mx[t]);
        tot[t] += w;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[t][e] = fmaf(w, x[k][t].e[e], acc[t][e]);
      }
    i0 += WPR * kMergeParts;
    if (i0 >= parts) break;
    load(i0);
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int e = 0; e < E; ++e) sums[warp][t][lane * E + e] = acc[t][e];
      if (lane == 0) sums[warp][t][D] = tot[t];
    }
    __syncthreads();
    if (sub != 0) return;
#pragma unroll
    for (int t = 0; t < 2; ++t)
      for (int k = 1; k < WPR; ++k) {
#pragma unroll
        for (int e = 0; e < E; ++e) acc[t][e] += sums[warp + k][t][lane * E + e];
        tot[t] += sums[warp + k][t][D];
      }
  }
  float out[E];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const float inv = mx[t] == -INFINITY ? 0.f : 1.f / tot[t];
    const float f = t == 0 ? inv : -lam * inv;
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] = t == 0 ? f * acc[0][e] : fmaf(f, acc[1][e], out[e]);
    if (p.lse != nullptr && lane == 0)
      p.lse[static_cast<size_t>(t) * rows + rg] =
          mx[t] == -INFINITY ? -INFINITY : (mx[t] + __log2f(tot[t])) * 0.69314718055994531f;
  }
  if (p.norm_w != nullptr) {
    float sq = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) sq = fmaf(out[e], out[e], sq);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    const float f = rsqrtf(sq * (1.f / D) + p.eps) * (1.f - p.lambda_init);
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] *= f * norm[e];
  }
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + ((static_cast<size_t>(b) * p.S_q + s_q) * p.H + head) * D) + lane * (E / 2);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) dst[e] = pack_x2<true>(out[2 * e], out[2 * e + 1]);
}

template <int D, int KIND, bool QUAD, bool LONG>
cudaError_t launch_t(const DiffParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                     cudaStream_t st) {
  using C = Cfg<D>;
  static_assert(C::SMEM <= 232448, "shared memory budget");
  auto kern = diff_attn_kernel<D, KIND, QUAD, LONG>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  if (KIND == kBf16WideV && p.S_kv > 0) {
    const dim3 grid(static_cast<unsigned>((p.S_kv + kConvRows - 1) / kConvRows), static_cast<unsigned>(p.B * p.H_kv));
    if ((e = cudaMemsetAsync(p.v_amax, 0, static_cast<size_t>(p.B) * p.H_kv * 4, st)) != cudaSuccess) return e;
    widen_v_kernel<D, false><<<grid, 256, 0, st>>>(p);
    widen_v_kernel<D, true><<<grid, 256, 0, st>>>(p);
  }
  kern<<<p.ctas, kThreads, C::SMEM, st>>>(tq, tk, tv, p);
  if ((e = cudaGetLastError()) != cudaSuccess || !p.merge) return e;
  constexpr int WPR = QUAD ? 4 : 1;
  const dim3 grid(static_cast<unsigned>(p.ctas - 1), static_cast<unsigned>(((p.R < BM ? p.R : BM) * WPR + 3) / 4));
  // launched while the walk runs (it waits for its end before it reads)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, diff_merge_kernel<D, WPR>, p, p.ctas);
}

template <int D, bool LONG>
cudaError_t launch_d(const DiffParams& p, bool in_bf16, const CUtensorMap& tq, const CUtensorMap& tk,
                     const CUtensorMap& tv, cudaStream_t st) {
  if (p.R <= kQuadRows)
    return in_bf16 ? launch_t<D, kBf16Split, true, LONG>(p, tq, tk, tv, st) : launch_t<D, kF16, true, LONG>(p, tq, tk, tv, st);
  if (!in_bf16) return launch_t<D, kF16, false, LONG>(p, tq, tk, tv, st);
  return p.v16 != nullptr ? launch_t<D, kBf16WideV, false, LONG>(p, tq, tk, tv, st)
                          : launch_t<D, kBf16Split, false, LONG>(p, tq, tk, tv, st);
}

}  // namespace

// How the items are walked: pure host arithmetic.
DiffWalk diff_walk(long long items, int n_rt, int S_kv, int sms) {
  const long long tiles = (S_kv + BN - 1) / BN;
  DiffWalk w{};
  if (items < sms) {
    // fewer items than SMs: cut them where a CTA still gets a few key tiles
    // (every such call; what the parts' way through memory costs is not weighed
    // against the tiles saved as it is for the last wave below)
    w.ctas = static_cast<int>(items);
    if (tiles >= 8) {
      const long long c = items * tiles / 4;
      w.ctas = static_cast<int>(c < sms ? c : sms);
      w.items_whole = 0;
      w.merge = w.ctas > 1;
      if (w.ctas < items) w.ctas = static_cast<int>(items);
      return w;
    }
    w.items_whole = items;
    return w;
  }
  w.ctas = sms;
  w.items_whole = items;
  if (tiles >= 8) {
    // One row tile per range: every key tile is read once, in any order.
    // Otherwise the last wave, where the key tiles it saves each CTA (about
    // 1.5 us each) exceed the parts' way through memory (about 12 us).
    const long long rest = items % sms;
    if (n_rt == 1) w.items_whole = 0;
    else if (rest > 0 && (sms - rest) * tiles > 8ll * sms) w.items_whole = items - rest;
  }
  w.merge = w.items_whole < items;
  return w;
}

// Whether bf16 operands get an fp16 copy of V: about 8 us and three passes over
// V, against a fifth of the walk for P in two parts.  Several row tiles have to
// share each V tile, and the walk to be long: 2 x 24 heads, 1000 tokens (20 key
// tiles per SM): 73 us with the copy, 72 without; 2 x 24 x 4608: 833 and 1040;
// 8 heads, 2000 tokens (14): 76 and 71; 24 heads, 300 x 8000 (3 row tiles):
// 122 and 100.
bool diff_widens_v(long long items, int n_rt, int S_kv, int sms) {
  return n_rt >= 4 && items * ((S_kv + BN - 1) / BN) >= 18ll * sms;
}

cudaError_t launch_diff_attn(const DiffParams& p, int d, bool in_bf16, const CUtensorMap& tq, const CUtensorMap& tk,
                             const CUtensorMap& tv, cudaStream_t st) {
  static_assert(kQuadRows == 32, "one quarter of the TMEM lanes");
  if (p.S_kv > kGatherKeys)
    return d == 128 ? launch_d<128, true>(p, in_bf16, tq, tk, tv, st) : launch_d<64, true>(p, in_bf16, tq, tk, tv, st);
  return d == 128 ? launch_d<128, false>(p, in_bf16, tq, tk, tv, st) : launch_d<64, false>(p, in_bf16, tq, tk, tv, st);
}

}  // namespace jattn
