// Linear layer on sm_100a: y = act(x W^T + bias) + residual, 16-bit operands,
// fp32 accumulation in tensor memory, the epilogue fused.
//
// Two kernels share the epilogue:
//   pair   256 x 256 output tiles by a cluster of two CTAs (cta_group::2):
//          each CTA holds 128 rows of x and 128 rows of W per 64-deep K step,
//          so an operand byte in shared memory feeds twice the MACs of a
//          single-CTA tile; persistent, two accumulators in TMEM, so one
//          tile's epilogue overlaps the next tile's products.
//   tile   128 x BN output tiles by one CTA, for problems with too few 256 x
//          256 tiles to fill the GPU; K may be split over a cluster of up to
//          8 CTAs that add their accumulators through distributed shared
//          memory (in rank order: same bits every run, no workspace).  Few
//          rows of x: the roles are swapped (W's rows are the MMA's 128 rows,
//          x the BN), so the tile wastes no work on absent rows and W streams
//          once.
// Operands that TMA cannot address are copied to rows that it can first.
//
// The tensor cores' own fp32 sums lose a little at every addition (about half
// a unit per 16 products, and always towards zero: 2e-6 of the result at K =
// 3000, 6e-3 at K = 2^20 where all products have one sign).  For fp32 outputs,
// and for 16-bit ones of sums so long that it would show beside their rounding
// (gathers), the accumulator is emptied every kFlushSteps K steps into fp32
// registers that add with rounding (FLUSH; two accumulators, so the products go
// on meanwhile).
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "jattn.h"
#include "jattn_internal.h"
#include "ptx_sm100.cuh"

namespace jattn {

namespace {

constexpr int BK = 64;                 // K per stage: one 128-byte swizzle row
constexpr int kEpiThreads = 128;       // warps 0..3
constexpr int kThreads = 192;          // + warp 4 (loads), warp 5 (MMA)

constexpr int kFlushSteps = 8;         // 512 products

struct __align__(8) TileBars {
  uint64_t full[8], empty[8];
  uint64_t acc_full[2], acc_empty[2];
  uint32_t tmem_base;
  uint32_t abort;
};

__device__ __forceinline__ uint32_t pack2(float a, float b, bool bf16) {
  if (bf16) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ float widen16(uint16_t u, bool bf16) {
  return bf16 ? __uint_as_float(static_cast<uint32_t>(u) << 16) : __half2float(__ushort_as_half(u));
}
// One element of type dt at index i.
__device__ __forceinline__ float load_as_f32(const void* p, int64_t i, int dt) {
  if (dt == JATTN_FP32) return static_cast<const float*>(p)[i];
  return widen16(static_cast<const uint16_t*>(p)[i], dt == JATTN_BF16);
}
__device__ __forceinline__ void store_from_f32(void* p, int64_t i, int dt, float v) {
  if (dt == JATTN_FP32) static_cast<float*>(p)[i] = v;
  else if (dt == JATTN_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// The activations, in fp32.  For 16-bit outputs exp and the reciprocal are the
// hardware's approximate ones (2^-21 relative or better, far under the
// output's rounding).
__device__ __forceinline__ float sigmoid_f32(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }
// For fp32 outputs: exp to 2 ulp, the reciprocal with one Newton step (without
// the branches of a division, which kept the elements of a row from
// interleaving: 8 us on a 128 x 128 tile).  Below -87 the reciprocal is no
// normal number: 0.
__device__ __forceinline__ float sigmoid_precise(float x) {
  const float d = 1.f + expf(fminf(-x, 87.f));
  const float r = __fdividef(1.f, d);
  return x < -87.f ? 0.f : fmaf(r, fmaf(-d, r, 1.f), r);
}
// x Phi(x) with the small values of negative x kept: 1 + erf(x / sqrt 2) cancels
// there (off by 3e-4 at -4, 4% at -5), and erfcf took 659 us in the product of
// 16896 x 8192 x 2048 where this takes 413 (1 + erff: 427).  Phi(-z) = e^(-z^2 / 2) R(z), R(z) =
// erfcx(z / sqrt 2) / 2 as t (c0 + ... + c7 t^7), t = 1 / (1 + 0.3 z): the
// polynomial with the smallest largest relative error on z in [0, 14.5] (1.6e-7;
// coefficients by iteratively reweighted least squares).  Past 16 Phi(-z) is 0.
__device__ __forceinline__ float gelu_f32(float x) {
  const float z = fminf(fabsf(x), 16.f);
  const float t = __fdividef(1.f, fmaf(0.3f, z, 1.f));
  float r = fmaf(0x1.22317ep-5f, t, -0x1.3fd080p-3f);
  r = fmaf(r, t, 0x1.a2ef72p-3f);
  r = fmaf(r, t, -0x1.aa45d0p-5f);
  r = fmaf(r, t, 0x1.058392p-3f);
  r = fmaf(r, t, 0x1.9a51eep-4f);
  r = fmaf(r, t, 0x1.ee6fe0p-4f);
  r = fmaf(r, t, 0x1.ea0340p-4f);
  const float phi = r * t * ex2_approx(z * z * -0.72134752044448170f);
  return x > 0.f ? fmaf(-z, phi, x) : x * phi;           // NaN stays, and -inf gives it as -inf * 0 does
}
template <int ACT, bool PRECISE>
__device__ __forceinline__ float activate_as(float x) {
  auto sigmoid = [](float t) { return PRECISE ? sigmoid_precise(t) : sigmoid_f32(t); };
  if constexpr (ACT == JATTN_ACT_GELU) return gelu_f32(x);
  // 0.5 (1 + tanh u) = sigmoid(2 u)
  if constexpr (ACT == JATTN_ACT_GELU_TANH) return x * sigmoid(1.5957691216057308f * (x + 0.044715f * x * x * x));
  if constexpr (ACT == JATTN_ACT_SILU) return x * sigmoid(x);
  if constexpr (ACT == JATTN_ACT_RELU) return x < 0.f ? 0.f : x;     // keeps NaN
  return x;
}
template <int ACT, int W>
__device__ __forceinline__ void activate_all(float (&v)[W], bool precise) {
  if (precise) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = activate_as<ACT, true>(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = activate_as<ACT, false>(v[i]);
  }
}
// One branch per array, not per element: the elements' chains interleave.
template <int W>
__device__ __forceinline__ void activate(float (&v)[W], const LinearParams& p) {
  const bool precise = p.out_dtype == JATTN_FP32;
  switch (p.act) {
    case JATTN_ACT_GELU: activate_all<JATTN_ACT_GELU>(v, precise); break;
    case JATTN_ACT_GELU_TANH: activate_all<JATTN_ACT_GELU_TANH>(v, precise); break;
    case JATTN_ACT_SILU: activate_all<JATTN_ACT_SILU>(v, precise); break;
    case JATTN_ACT_RELU: activate_all<JATTN_ACT_RELU>(v, precise); break;
    default: break;
  }
}

// Whether 32-element chunks of a row-major matrix (type dt, row stride ld)
// may be moved with 16- or 32-byte accesses: bytes of the widest, else 0.
__host__ __device__ inline int vector_bytes(const void* p, int64_t ld, int dt) {
  const int64_t es = dt == JATTN_FP32 ? 4 : 2;
  const uint64_t m = reinterpret_cast<uint64_t>(p) | static_cast<uint64_t>(ld * es);
  return (m & 31) == 0 ? 32 : ((m & 15) == 0 ? 16 : 0);
}

template <int WORDS>
__device__ __forceinline__ void load_row(const uint32_t* src, uint32_t (&w)[WORDS], int vec) {
  if (WORDS % 8 == 0 && vec == 32) {
#pragma unroll
    for (int i = 0; i + 7 < WORDS; i += 8)
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]), "=r"(w[i + 4]), "=r"(w[i + 5]),
                     "=r"(w[i + 6]), "=r"(w[i + 7])
                   : "l"(src + i)
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < WORDS; i += 4) {
      const uint4 t = *reinterpret_cast<const uint4*>(src + i);
      w[i] = t.x; w[i + 1] = t.y; w[i + 2] = t.z; w[i + 3] = t.w;
    }
  }
}
template <int WORDS>
__device__ __forceinline__ void store_row(uint32_t* dst, const uint32_t (&w)[WORDS], int vec) {
  if (WORDS % 8 == 0 && vec == 32) {
#pragma unroll
    for (int i = 0; i + 7 < WORDS; i += 8)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                   ::"l"(dst + i), "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]),
                     "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < WORDS; i += 4) *reinterpret_cast<uint4*>(dst + i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  }
}

// Floats of one warp's staging block: 32 rows of up to 32 columns, one word
// apart so that neither its rows nor its columns share a bank.
constexpr int kStageFloats = 32 * 33;

// A whole warp: columns [n, n + W) of rows m0 + lane from the accumulator, bias
// already fp32 in shared memory (zeros past N or without a bias).  Rows that
// can be moved in 16 bytes are finished by their thread; others (odd row
// strides, the last columns) go through `stage`, so that the lanes of an access
// are neighbours in a row instead of 32 rows apart (4234 x 270 x 123: 21 -> 15 us).
template <int W>
__device__ __forceinline__ void finish_rows(const LinearParams& p, float (&v)[W], const float* bias, int64_t m0, int n,
                                            float* stage) {
  const int lane = threadIdx.x & 31;
  const int64_t m = m0 + lane;
#pragma unroll
  for (int i = 0; i < W; i += 4) {
    const float4 b = *reinterpret_cast<const float4*>(bias + i);
    v[i] += b.x;
    v[i + 1] += b.y;
    v[i + 2] += b.z;
    v[i + 3] += b.w;
  }
  activate(v, p);
  const bool f32 = p.out_dtype == JATTN_FP32, bf16 = p.out_dtype == JATTN_BF16;
  if (n + W > p.N || p.vec_y == 0 || (p.residual != nullptr && p.vec_r == 0)) {
    __syncwarp();                                        // the block's last use is over
#pragma unroll
    for (int i = 0; i < W; ++i) stage[lane * (W + 1) + i] = v[i];
    __syncwarp();
    // column n + c of the rows r0, r0 + 32 / W, ...: every residual element on
    // its way before the first is used (clamped addresses: no branch between)
    constexpr int ROUNDS = W;
    const int c = lane % W, r0 = lane / W;
    const bool in = n + c < p.N;
    const int64_t n_at = min(n + c, p.N - 1);
    float x[ROUNDS];
    if (p.residual != nullptr) {
      const int64_t last = p.M - 1;
      if (f32) {
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k)
          x[k] = static_cast<const float*>(p.residual)[min(m0 + r0 + k * (32 / W), last) * p.ldr + n_at];
      } else {
        uint16_t h[ROUNDS];
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k)
          h[k] = static_cast<const uint16_t*>(p.residual)[min(m0 + r0 + k * (32 / W), last) * p.ldr + n_at];
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k) x[k] = widen16(h[k], bf16);
      }
    } else {
#pragma unroll
      for (int k = 0; k < ROUNDS; ++k) x[k] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < ROUNDS; ++k) {
      const int r = r0 + k * (32 / W);
      if (in && m0 + r < p.M) store_from_f32(p.y, (m0 + r) * p.ldy + n_at, p.out_dtype, x[k] + stage[r * (W + 1) + c]);
    }
    return;
  }
  if (m >= p.M) return;
  if (p.residual != nullptr) {
    const int64_t at = m * p.ldr + n;
    if (f32) {
      uint32_t w[W];
      load_row(static_cast<const uint32_t*>(p.residual) + at, w, p.vec_r);
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] += __uint_as_float(w[i]);
    } else {
      uint32_t w[W / 2];
      load_row(reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.residual) + at), w, p.vec_r);
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        v[2 * i] += widen16(static_cast<uint16_t>(w[i]), bf16);
        v[2 * i + 1] += widen16(static_cast<uint16_t>(w[i] >> 16), bf16);
      }
    }
  }
  const int64_t at = m * p.ldy + n;
  if (f32) {
    uint32_t w[W];
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = __float_as_uint(v[i]);
    store_row(static_cast<uint32_t*>(p.y) + at, w, p.vec_y);
  } else {
    uint32_t w[W / 2];
#pragma unroll
    for (int i = 0; i < W / 2; ++i) w[i] = pack2(v[2 * i], v[2 * i + 1], bf16);
    store_row(reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.y) + at), w, p.vec_y);
  }
}

__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Address of the same shared-memory location in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// The MMA (one CTA's, or the pair's) and commit instructions by the lane with
// `lead` set, the rest of the warp along: descriptors that the compiler knows
// to be warp uniform live in uniform registers, where the instruction wants
// them; in a branch of one lane each MMA took about 70 clocks to issue.
template <int CTAS>
__device__ __forceinline__ void mma_f16_if(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t acc) {
  if constexpr (CTAS == 1)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
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
// Arrives at the same barrier of both CTAs.
__device__ __forceinline__ void commit_pair_if(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2;\n\t}\n"
      ::"r"(smem_u32(bar)), "r"(lead), "h"(static_cast<uint16_t>(3))
      : "memory");
}

// Bounded wait of a whole warp (the tcgen05.ld that follows is collective).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtl& ctl) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    const bool ok = mbar_try_wait(bar, parity);
    if (__all_sync(0xffffffffu, ok)) return true;
    if ((i & 63u) == 0u) {
      int stop = 0;
      if (lane_id() == 0) {
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        if (*ctl.abort) {
          stop = 1;
        } else if (now - t0 > ctl.limit_ns) {
          atomicOr(ctl.status, JATTN_DEV_TIMEOUT);
          *ctl.abort = 1u;
          stop = 1;
        }
      }
      if (__shfl_sync(0xffffffffu, stop, 0)) return false;
    }
  }
}
// After an abort: leave copies in flight time to land before the CTA's
// shared memory goes away (they need microseconds).
__device__ __forceinline__ void settle() {
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < 1000000ull) {
  }
}

// 16 columns per lane, into the first half of r.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void tma_load_2d(const CUtensorMap* map, uint64_t* bar, void* dst, int32_t c0, int32_t c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}
// Into this CTA's shared memory, counted on the pair's leader's barrier (the
// peer bit of the barrier address cleared).
__device__ __forceinline__ void tma_load_2d_pair(const CUtensorMap* map, uint64_t* bar, void* dst, int32_t c0,
                                                 int32_t c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4}], [%2];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar) & 0xFEFFFFFFu), "r"(c0), "r"(c1)
      : "memory");
}

// An epilogue warp's sums of the `parts` accumulators (two buffers of BN
// columns from tl on; `before` of them were used before, both CTAs' epilogues
// of a pair tell its leader), rounded to nearest in fp32 registers, written to
// the columns at `out` for the epilogue.  The last buffer is not handed back.
template <int BN, bool PAIR = false>
__device__ __forceinline__ bool gather_parts(TileBars* bar, uint32_t tl, int parts, int before, uint32_t out,
                                             const WaitCtl& ctl) {
  constexpr int CH = BN < 32 ? BN : 32;
  float sum[BN];
#pragma unroll
  for (int i = 0; i < BN; ++i) sum[i] = 0.f;
#pragma unroll 1
  for (int q = 0; q < parts; ++q) {
    const int at = before + q, buf = at & 1;
    if (!warp_wait(&bar->acc_full[buf], (at >> 1) & 1, ctl)) return false;
    __syncwarp();
    tc_fence_after();
#pragma unroll
    for (int c = 0; c < BN; c += CH) {
      uint32_t r[32];
      if constexpr (CH == 16) tmem_ld16(tl + buf * BN + c, r);
      else tmem_ld32(tl + buf * BN + c, r);
#pragma unroll
      for (int i = 0; i < CH; ++i) sum[c + i] += __uint_as_float(r[i]);
    }
    if (q + 1 < parts) {
      tc_fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) {
        if constexpr (PAIR)
          asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];"
                       ::"r"(map_rank(smem_u32(&bar->acc_empty[buf]), 0)) : "memory");
        else
          mbar_arrive(&bar->acc_empty[buf]);
      }
    }
  }
  __syncwarp();
#pragma unroll
  for (int c = 0; c < BN; c += CH) {
    uint32_t r[32];
#pragma unroll
    for (int i = 0; i < CH; ++i) r[i] = __float_as_uint(sum[c + i]);
    if constexpr (CH == 16) {
      uint32_t h[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) h[i] = r[i];
      tmem_st16(out + c, h);
    } else {
      tmem_st32(out + c, r);
    }
  }
  return true;
}

// ---------------------------------------------------------------- one-CTA tiles

// SWAP: the MMA's 128 rows are W's and its BN columns x's.  DEEP: all of an
// SM's shared memory for one CTA's stages, where there are no more CTAs than
// SMs; otherwise half, so that two share an SM.
template <int BN, bool SWAP, bool DEEP, bool FLUSH>
struct TileCfg {
  static constexpr int STAGE = (128 + BN) * BK * 2;
  static constexpr int ST = DEEP ? (BN >= 128 ? 6 : 8) : (BN >= 128 ? 3 : (BN >= 64 ? 4 : 5));
  static constexpr int PIPE = ST * STAGE;
  static constexpr int RED = 128 * BN * 4;              // split K: this CTA's accumulator tile
  static constexpr int DATA = PIPE;                     // behind RED, the epilogue's staging blocks
  static_assert(SWAP ? PIPE >= RED : PIPE >= RED + 4 * 32 * 33 * 4, "room for the epilogue");
  static constexpr int SMEM = DATA + BN * 4 + 512 + 1024;
  static constexpr uint32_t TCOLS = FLUSH ? 2u * BN : (BN < 32 ? 32u : static_cast<uint32_t>(BN));
};

// Copies of operands whose rows TMA cannot address (row strides or addresses
// that are not multiples of 16 bytes), rows of a multiple of 8 elements with
// zeros behind K.  blockIdx.y = the operand.  A thread writes 8 elements; they
// lie in at most two aligned 16-byte pieces, loaded whole and shifted into
// place.  The copy costs one pass over the operand and the product then runs
// at TMA's speed; staging such rows by plain loads inside the product took
// 375 us for 9000 x 7000 x 501 and 58 us for 1531 x 777 x 1003, this 155 and 22.
struct RepackParams {
  const uint16_t* src[2];
  uint16_t* dst[2];
  int64_t ld[2], rows[2];
  int K, Kp;
};
// The aligned 8 elements at `at`, or what of them lies in [lo, hi).
__device__ __forceinline__ uint4 load_piece(const uint16_t* at, const uint16_t* lo, const uint16_t* hi) {
  if (at >= lo && at + 8 <= hi) return __ldg(reinterpret_cast<const uint4*>(at));
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (at + i >= lo && at + i < hi) w[i >> 1] |= static_cast<uint32_t>(__ldg(at + i)) << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__global__ void __launch_bounds__(256) repack_kernel(const RepackParams p) {
  const bool second = blockIdx.y != 0;
  const int chunks = p.Kp / 8;
  const uint16_t* g = second ? p.src[1] : p.src[0];
  if (g == nullptr) return;
  uint16_t* dst = second ? p.dst[1] : p.dst[0];
  const int64_t ld = second ? p.ld[1] : p.ld[0], rows = second ? p.rows[1] : p.rows[0];
  const int64_t total = rows * chunks;
  const uint16_t* hi = g + (rows - 1) * ld + p.K;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t row = i / chunks;
    const int k = static_cast<int>(i % chunks) * 8;
    const uint16_t* at = g + row * ld + k;
    const uint32_t o = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at) >> 1) & 7u;
    const uint4 x = load_piece(at - o, g, hi);
    const uint4 y = o != 0 ? load_piece(at - o + 8, g, hi) : make_uint4(0u, 0u, 0u, 0u);
    uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int j = 0; j < 6; ++j) w[j] = o & 4u ? w[j + 2] : w[j];
#pragma unroll
    for (int j = 0; j < 5; ++j) w[j] = o & 2u ? w[j + 1] : w[j];
    const uint32_t sh = o & 1u ? 16u : 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __funnelshift_r(w[j], w[j + 1], sh);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (p.K - k <= 2 * j) w[j] = 0u;
      else if (p.K - k == 2 * j + 1) w[j] &= 0xFFFFu;
    }
    *reinterpret_cast<uint4*>(dst + row * p.Kp + k) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <int BN, bool SWAP, bool DEEP, bool FLUSH>
__global__ void __launch_bounds__(kThreads, DEEP ? 1 : 2)
linear_tile_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const LinearParams p) {
  using C = TileCfg<BN, SWAP, DEEP, FLUSH>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float* sBias = reinterpret_cast<float*>(smem + C::DATA);
  TileBars* bar = reinterpret_cast<TileBars*>(smem + C::DATA + BN * 4);
  // from one lane, so that the compiler sees the roles' branches as uniform
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  // tile (a, b) = rows a * 128 of A, rows b * BN of B; the cluster's CTAs
  // share a tile and take the K steps [kb, ke)
  const int split = p.splits, rank = split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int tile = blockIdx.x / split;
  const int ta = tile % p.tiles_a, tb = tile / p.tiles_a;
  const int ksteps = (p.K + BK - 1) / BK;
  const int kb = static_cast<int>(static_cast<long long>(ksteps) * rank / split);
  const int ke = static_cast<int>(static_cast<long long>(ksteps) * (rank + 1) / split);

  auto load = [&](int k) {                               // K step k of the whole, into its stage
    const int s = (k - kb) % C::ST;
    mbar_arrive_expect_tx(&bar->full[s], C::STAGE);
    tma_load_2d(&tmA, &bar->full[s], smem + s * C::STAGE, k * BK, ta * 128);
    tma_load_2d(&tmB, &bar->full[s], smem + s * C::STAGE + 128 * BK * 2, k * BK, tb * BN);
  };
  if (threadIdx.x == 128) {
    for (int s = 0; s < C::ST; ++s) {
      mbar_init(&bar->full[s], 1);
      mbar_init(&bar->empty[s], 1);
    }
    for (int i = 0; i < (FLUSH ? 2 : 1); ++i) {
      mbar_init(&bar->acc_full[i], 1);
      mbar_init(&bar->acc_empty[i], 4);                  // the epilogue warps
    }
    bar->abort = 0;
    fence_mbarrier_init();
    // the first stages are free: their loads leave before the block meets
    for (int k = kb; k < min(ke, kb + C::ST); ++k) load(k);
  }
  if (warp == 5) {
    __syncwarp();
    tmem_alloc(&bar->tmem_base, C::TCOLS);
    tmem_relinquish();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;
  const WaitCtl ctl{&bar->abort, p.status, p.timeout_ns};

  if (warp == 4) {
    if (lane == 0) {
      bool ok = true;
      for (int k = kb + C::ST; k < ke && ok; ++k) {
        const int i = k - kb;
        ok = mbar_wait(&bar->empty[i % C::ST], ((i / C::ST) & 1) ^ 1, ctl);
        if (ok) load(k);
      }
      // the last stages' commits have arrived before the CTA may exit
      for (int i = ke - kb > C::ST ? ke - kb - C::ST : 0; i < ke - kb && ok; ++i)
        ok = mbar_wait(&bar->empty[i % C::ST], (i / C::ST) & 1, ctl);
      if (!ok) settle();
    }
  } else if (warp == 5) {
    // the whole warp walks, one lane issues (see mma_f16_if)
    const uint32_t lead = elect_one() ? 1u : 0u;
    const uint32_t idesc = instr_desc(p.in_bf16, p.in_bf16, 0, 128, BN);
    const uint64_t ad0 = smem_desc(smem_u32(smem), 16, 1024, 2u), bd0 = ad0 + 128 * BK * 2 / 16;
    int s = 0;
    uint32_t par = 0;
    for (int k = kb; k < ke; ++k) {
      const int in = FLUSH ? (k - kb) % kFlushSteps : k - kb, part = FLUSH ? (k - kb) / kFlushSteps : 0;
      const uint32_t acc = tmem + (part & 1) * BN;
      if (FLUSH && in == 0) {
        if (part > 0) commit_if(lead, &bar->acc_full[(part - 1) & 1]);
        if (!warp_wait(&bar->acc_empty[part & 1], ((part >> 1) & 1) ^ 1, ctl)) break;
      }
      if (!warp_wait(&bar->full[s], par, ctl)) break;
      tc_fence_after();
      const uint32_t at = s * (C::STAGE / 16);
#pragma unroll
      for (int kk = 0; kk < BK / 16; ++kk)
        mma_f16_if<1>(lead, acc, ad0 + at + kk * 2, bd0 + at + kk * 2, idesc, in > 0 || kk > 0);
      commit_if(lead, &bar->empty[s]);
      if (++s == C::ST) {
        s = 0;
        par ^= 1;
      }
    }
    commit_if(lead, &bar->acc_full[FLUSH ? ((ke - kb - 1) / kFlushSteps) & 1 : 0]);
  } else {
    if (!SWAP) {
      for (int i = threadIdx.x; i < BN; i += kEpiThreads) {
        const int n = tb * BN + i;
        sBias[i] = p.bias != nullptr && n < p.N ? load_as_f32(p.bias, n, p.bias_dtype) : 0.f;
      }
      epi_sync();
    }
  }
  // The epilogue waits for the accumulator; every thread then meets the
  // cluster's other CTAs (or the block) once.
  bool good = false;
  const int row = (warp & 3) * 32 + lane;
  const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  if (warp < 4) {
    if constexpr (FLUSH) good = gather_parts<BN>(bar, tl, (ke - kb + kFlushSteps - 1) / kFlushSteps, 0, tl, ctl);
    else good = warp_wait(&bar->acc_full[0], 0, ctl);
    __syncwarp();
    tc_fence_after();
  }
  constexpr int CH = BN < 32 ? BN : 32;                  // accumulator columns at a time
  float* red = reinterpret_cast<float*>(smem);           // [BN][128]: the pipeline is drained
  __syncwarp();
  if (split > 1) {
    if (warp < 4 && good) {
#pragma unroll
      for (int c = 0; c < BN; c += CH) {
        uint32_t r[32];
        if constexpr (CH == 16) tmem_ld16(tl + c, r);
        else tmem_ld32(tl + c, r);
#pragma unroll
        for (int i = 0; i < CH; ++i) red[(c + i) * 128 + row] = __uint_as_float(r[i]);
      }
    }
    __syncwarp();
    cluster_sync();
  }
  if (warp < 4 && good) {
    // the columns of this CTA: all, or its share of a split tile
    const int c_lo = split > 1 ? BN * rank / split : 0;
    const int c_hi = split > 1 ? BN * (rank + 1) / split : BN;
    const uint32_t red_addr = smem_u32(red);
    if (SWAP) {
      const int64_t n = static_cast<int64_t>(ta) * 128 + row;
      const float bias = p.bias != nullptr && n < p.N ? load_as_f32(p.bias, n, p.bias_dtype) : 0.f;
      // columns [c, c + W) of the tile for output channel n
      auto put = [&](int c, auto& v, int count) {
        constexpr int W = sizeof(v) / sizeof(float);
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] += bias;
        activate(v, p);
        const int64_t m = static_cast<int64_t>(tb) * BN + c;
        if (n >= p.N) return;
        if (p.residual != nullptr) {
#pragma unroll
          for (int i = 0; i < W; ++i)
            if (i < count && m + i < p.M) v[i] += load_as_f32(p.residual, (m + i) * p.ldr + n, p.out_dtype);
        }
#pragma unroll
        for (int i = 0; i < W; ++i)
          if (i < count && m + i < p.M) store_from_f32(p.y, (m + i) * p.ldy + n, p.out_dtype, v[i]);
      };
      if (split > 1) {
        constexpr int W = BN / 2;                        // the widest share of a split tile
        const int count = c_hi - c_lo;
        float v[W];
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = 0.f;
        for (int q = 0; q < split; ++q) {
          const uint32_t at = map_rank(red_addr + (c_lo * 128 + row) * 4, q);
#pragma unroll
          for (int i = 0; i < W; ++i)
            if (i < count) v[i] += ld_cluster(at + i * 512);
        }
        put(c_lo, v, count);
      } else {
#pragma unroll 1
        for (int c = 0; c < BN; c += CH) {
          uint32_t r[32];
          __syncwarp();
          if constexpr (CH == 16) tmem_ld16(tl + c, r);
          else tmem_ld32(tl + c, r);
          float v[CH];
#pragma unroll
          for (int i = 0; i < CH; ++i) v[i] = __uint_as_float(r[i]);
          put(c, v, CH);
        }
      }
    } else if constexpr (BN >= 32) {
      const int64_t m0 = static_cast<int64_t>(ta) * 128 + (warp & 3) * 32;
      float* stage = reinterpret_cast<float*>(smem + C::RED) + (warp & 3) * kStageFloats;
      if (split > 1) {
        // a share of BN / split columns, 8 at a time
        for (int c = c_lo; c < c_hi; c += 8) {
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = 0.f;
          for (int q = 0; q < split; ++q) {
            const uint32_t at = map_rank(red_addr + (c * 128 + row) * 4, q);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += ld_cluster(at + i * 512);
          }
          if (tb * BN + c < p.N) finish_rows(p, v, sBias + c, m0, tb * BN + c, stage);
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < BN; c += 32) {
          uint32_t r[32];
          __syncwarp();
          tmem_ld32(tl + c, r);
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
          if (tb * BN + c < p.N) finish_rows(p, v, sBias + c, m0, tb * BN + c, stage);
        }
      }
    }
  }
  // no CTA leaves while another still reads its accumulators
  __syncwarp();
  if (split > 1) cluster_sync();
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::TCOLS);
  }
}

// ---------------------------------------------------------------- pairs of CTAs

template <int BN>
struct PairCfg {
  static constexpr int STAGE = (128 + BN / 2) * BK * 2;  // per CTA: its rows of x, its rows of W
  static constexpr int ST = BN == 256 ? 6 : 8;
  static constexpr int BIAS = 4 * BN * 4;                // each epilogue warp keeps its own copy
  static constexpr int OUT = 4 * 32 * 33 * 4;            // and a staging block
  static constexpr int SMEM = ST * STAGE + BIAS + OUT + 512 + 1024;
};
constexpr int kGroupM = 8;                               // tiles of x a column of W tiles is used for in a row

// BN 256, or 128 with FLUSH (its sums are registers).
template <int BN, bool FLUSH>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
linear_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                   const LinearParams p) {
  using C = PairCfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float* sBias = reinterpret_cast<float*>(smem + C::ST * C::STAGE);   // [4][BN]
  TileBars* bar = reinterpret_cast<TileBars*>(smem + C::ST * C::STAGE + C::BIAS + C::OUT);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int tiles_n = (p.N + BN - 1) / BN;
  const long long n_tiles = static_cast<long long>(p.tiles_a) * tiles_n;
  const int n_pairs = gridDim.x / 2, pair = blockIdx.x / 2;
  const int ksteps = (p.K + BK - 1) / BK;
  // tile order: kGroupM row tiles share each column tile while both are in L2
  auto place = [&](long long t, int& tm, int& tn) {
    const long long per = static_cast<long long>(kGroupM) * tiles_n;
    const int g = static_cast<int>(t / per), first = g * kGroupM;
    const int size = min(kGroupM, p.tiles_a - first), in = static_cast<int>(t % per);
    tm = first + in % size;
    tn = in / size;
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::ST; ++s) {
      mbar_init(&bar->full[s], 1);
      mbar_init(&bar->empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->acc_full[i], 1);
      mbar_init(&bar->acc_empty[i], 8);                  // four epilogue warps of both CTAs
    }
    bar->abort = 0;
    fence_mbarrier_init();
  }
  cluster_sync();
  if (warp == 5) {
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_u32(&bar->tmem_base)), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;
  const WaitCtl ctl{&bar->abort, p.status, p.timeout_ns};

  if (warp == 4) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (long long t = pair; t < n_tiles && ok; t += n_pairs) {
        int tm, tn;
        place(t, tm, tn);
        for (int k = 0; k < ksteps; ++k, ++it) {
          const int s = it % C::ST;
          ok = mbar_wait(&bar->empty[s], ((it / C::ST) & 1) ^ 1, ctl);
          if (!ok) break;
          if (leader) mbar_arrive_expect_tx(&bar->full[s], 2 * C::STAGE);
          uint8_t* dst = smem + s * C::STAGE;
          tma_load_2d_pair(&tmX, &bar->full[s], dst, k * BK, tm * 256 + static_cast<int>(rank) * 128);
          tma_load_2d_pair(&tmW, &bar->full[s], dst + 128 * BK * 2, k * BK, tn * BN + static_cast<int>(rank) * (BN / 2));
        }
      }
      // the last stages' commits have arrived before the CTA may exit
      for (int i = it > C::ST ? it - C::ST : 0; i < it && ok; ++i)
        ok = mbar_wait(&bar->empty[i % C::ST], (i / C::ST) & 1, ctl);
      if (!ok) settle();
    }
  } else if (warp == 5) {
    if (leader) {
      const uint32_t lead = elect_one() ? 1u : 0u;
      const uint32_t idesc = instr_desc(p.in_bf16, p.in_bf16, 0, 256, BN);
      const uint64_t ad0 = smem_desc(smem_u32(smem), 16, 1024, 2u), bd0 = ad0 + 128 * BK * 2 / 16;
      int s = 0, n = 0;
      uint32_t par = 0;
      bool ok = true;
      for (long long t = pair; t < n_tiles && ok; t += n_pairs, ++n) {
        for (int k = 0; k < ksteps; ++k) {
          const int in = FLUSH ? k % kFlushSteps : k;
          if (in == 0) {
            if (k > 0) commit_pair_if(lead, &bar->acc_full[(n++) & 1]);
            ok = warp_wait(&bar->acc_empty[n & 1], ((n >> 1) & 1) ^ 1, ctl);
            if (!ok) break;
          }
          ok = warp_wait(&bar->full[s], par, ctl);
          if (!ok) break;
          tc_fence_after();
          const uint32_t at = s * (C::STAGE / 16);
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            mma_f16_if<2>(lead, tmem + (n & 1) * BN, ad0 + at + kk * 2, bd0 + at + kk * 2, idesc, in > 0 || kk > 0);
          commit_pair_if(lead, &bar->empty[s]);
          if (++s == C::ST) {
            s = 0;
            par ^= 1;
          }
        }
        if (!ok) break;
        commit_pair_if(lead, &bar->acc_full[n & 1]);
      }
      if (!ok) settle();
    }
  } else {
    const uint32_t tl = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    float* stage = reinterpret_cast<float*>(smem + C::ST * C::STAGE + C::BIAS) + warp * kStageFloats;
    const int parts = FLUSH ? (ksteps + kFlushSteps - 1) / kFlushSteps : 1;
    int n = 0;                                           // accumulators so far
    for (long long t = pair; t < n_tiles; t += n_pairs, n += parts) {
      int tm, tn;
      place(t, tm, tn);
      const int buf = (n + parts - 1) & 1;
      // no barrier among the epilogue warps: one that gave up must not leave
      // the others waiting for it
      float* bias = sBias + warp * BN;
      __syncwarp();
      for (int i = lane; i < BN; i += 32) {
        const int c = tn * BN + i;
        bias[i] = p.bias != nullptr && c < p.N ? load_as_f32(p.bias, c, p.bias_dtype) : 0.f;
      }
      if constexpr (FLUSH) {
        if (!gather_parts<BN, true>(bar, tl, parts, n, tl + buf * BN, ctl)) break;
      } else {
        if (!warp_wait(&bar->acc_full[buf], (n >> 1) & 1, ctl)) break;
      }
      __syncwarp();
      tc_fence_after();
      const int64_t m0 = static_cast<int64_t>(tm) * 256 + rank * 128 + warp * 32;
#pragma unroll 1
      for (int c = 0; c < BN; c += 32) {
        uint32_t r[32];
        __syncwarp();
        tmem_ld32(tl + buf * BN + c, r);
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
        if (tn * BN + c < p.N) finish_rows(p, v, bias + c, m0, tn * BN + c, stage);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0)
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];"
                     ::"r"(map_rank(smem_u32(&bar->acc_empty[buf]), 0)) : "memory");
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 5) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

template <int BN, bool SWAP, bool DEEP, bool FLUSH = false>
cudaError_t launch_tile(const LinearParams& p, const CUtensorMap& ta, const CUtensorMap& tb, cudaStream_t st) {
  using C = TileCfg<BN, SWAP, DEEP, FLUSH>;
  auto kern = linear_tile_kernel<BN, SWAP, DEEP, FLUSH>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  const long long blocks = static_cast<long long>(p.tiles_a) * p.tiles_b * p.splits;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = static_cast<unsigned>(p.splits);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.splits > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, ta, tb, p);
}

template <int BN, bool FLUSH>
cudaError_t launch_pair(LinearParams p, const CUtensorMap& tx, const CUtensorMap& tw, cudaStream_t st) {
  using C = PairCfg<BN>;
  static_assert(C::SMEM <= 232448, "shared memory budget");
  auto kern = linear_pair_kernel<BN, FLUSH>;
  p.tiles_a = (p.M + 255) / 256;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  const long long n_tiles = static_cast<long long>(p.tiles_a) * ((p.N + BN - 1) / BN);
  const long long pairs = device_sm_count() / 2;
  const int grid = static_cast<int>(2 * (n_tiles < pairs ? n_tiles : pairs));
  kern<<<grid, kThreads, C::SMEM, st>>>(tx, tw, p);
  return cudaGetLastError();
}

}  // namespace

// Whether the accumulator is emptied on the way.  K products of one sign lose
// 5.4e-9 K of their sum (measured: 2304 x 2304, K = 2^16, 3.5e-4): a fifth of half
// a step of fp16 at K = 2^14, of bf16 at 2^17.  Ungathered, fp16 results were off
// by 1.7 times half a step at K = 2^16 and 13 times at 2^20.
static bool gathers(int K, int out_dtype) {
  return K > (out_dtype == JATTN_FP32 ? kFlushSteps * BK : (out_dtype == JATTN_FP16 ? 1 << 14 : 1 << 17));
}

// The kernel, tile and split of one problem: pure host arithmetic.
LinearPlan plan_linear(int M, int N, int K, int out_dtype) {
  LinearPlan pl{};
  const long long ksteps = (static_cast<long long>(K) + BK - 1) / BK;
  pl.flush = gathers(K, out_dtype);
  const int pn = pl.flush ? 128 : 256;
  const long long pair_tiles = static_cast<long long>((M + 255) / 256) * ((N + pn - 1) / pn);
  // 256 x 256 tiles once they nearly fill the 74 pairs (1536 x 3000 x 1360, 72
  // tiles: 17.6 us against 19.1; 1024 x 4096 x 1024, 64 tiles: 12.6 against
  // 11.8); emptying their accumulators on the way they need several rounds
  // (2048 x 2048 x 2048 to fp32, 128 tiles: 24 us against 21; 4096 x 2048 x 2048,
  // 256 tiles: 43 against 39)
  if (pair_tiles >= (pl.flush ? 296 : 68)) {
    pl.pair = true;
    pl.bn = pn;
    return pl;
  }
  pl.splits = 1;
  if (M <= 32) {
    // W streams once: CTAs for most SMs, but K steps enough to fill each one's
    // pipeline (4 x 4096 x 4096: 10.6 us with 4 splits, 12.2 with 2; 4 x 8192 x
    // 1024: 6.1 whole, 6.7 in halves).  Clusters of 8 only where they are few:
    // with an SM's shared memory each they do not all fit at once (4 x 2048 x
    // 8192: 17.8 us, with 4 splits 12.2; 4 x 1024 x 4096, 8 tiles: 6.7 and 8.0).
    pl.swap = true;
    pl.bn = M <= 16 ? 16 : 32;
    const long long tiles = (N + 127) / 128;
    while (pl.splits < 8 && tiles * pl.splits * 2 <= (pl.splits < 4 ? 148 : 64) &&
           ksteps / (pl.splits * 2) >= (tiles * pl.splits < 40 ? 6 : 12))
      pl.splits *= 2;
    return pl;
  }
  // 64 columns while the tiles do not outnumber the SMs, split in K where half
  // of them would idle (768 x 768 x 3000, 72 tiles: 13.7 us in halves, 17.3
  // whole, 20.9 in quarters; 1024 x 1024 x 1024, 128 tiles: 6.6 whole, 9.8 in
  // halves), otherwise 128 (512 x 4096 x 4096: 19.4 us with 128, 23.9 with 64)
  // -- unless two 64-column tiles fit on an SM and the epilogue, half as long
  // for them, weighs as much as the products: short sums (1000 x 1500 x 400
  // with gelu: 14.1 us, with 128 columns 19.9) and gathered ones (1531 x 777 x
  // 1003 to fp32 with silu: 21.7 and 31.7)
  const long long tiles = static_cast<long long>((M + 127) / 128) * ((N + 63) / 64);
  pl.bn = tiles <= 148 || (tiles <= 296 && (pl.flush || ksteps < 16)) ? 64 : 128;
  while (pl.splits < 4 && tiles * pl.splits * 2 <= 148 && ksteps / (pl.splits * 2) >= 4) pl.splits *= 2;
  return pl;
}

cudaError_t launch_repack(const void* const src[2], void* const dst[2], const int64_t ld[2], const int64_t rows[2],
                          int K, cudaStream_t st) {
  RepackParams p{};
  p.K = K;
  p.Kp = static_cast<int>((static_cast<int64_t>(K) + 7) / 8 * 8);
  int64_t most = 0;
  for (int i = 0; i < 2; ++i) {
    p.src[i] = static_cast<const uint16_t*>(src[i]);
    p.dst[i] = static_cast<uint16_t*>(dst[i]);
    p.ld[i] = ld[i];
    p.rows[i] = rows[i];
    if (src[i] != nullptr && rows[i] > most) most = rows[i];
  }
  const int64_t blocks = (most * (p.Kp / 8) + 255) / 256, cap = 16ll * device_sm_count();
  repack_kernel<<<dim3(static_cast<unsigned>(blocks < cap ? blocks : cap), 2), 256, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_linear(LinearParams p, const LinearPlan& pl, const CUtensorMap& tx, const CUtensorMap& tw,
                          cudaStream_t st) {
  p.vec_y = vector_bytes(p.y, p.ldy, p.out_dtype);
  p.vec_r = p.residual != nullptr ? vector_bytes(p.residual, p.ldr, p.out_dtype) : 0;
  if (pl.pair) return pl.flush ? launch_pair<128, true>(p, tx, tw, st) : launch_pair<256, false>(p, tx, tw, st);
  p.splits = pl.splits;
  const int rows_a = pl.swap ? p.N : p.M, rows_b = pl.swap ? p.M : p.N;
  p.tiles_a = (rows_a + 127) / 128;
  p.tiles_b = (rows_b + pl.bn - 1) / pl.bn;
  const CUtensorMap& ta = pl.swap ? tw : tx;
  const CUtensorMap& tb = pl.swap ? tx : tw;
  if (pl.flush) {
    if (pl.swap) return pl.bn == 16 ? launch_tile<16, true, false, true>(p, ta, tb, st) : launch_tile<32, true, false, true>(p, ta, tb, st);
    return pl.bn == 64 ? launch_tile<64, false, false, true>(p, ta, tb, st) : launch_tile<128, false, false, true>(p, ta, tb, st);
  }
  if (static_cast<long long>(p.tiles_a) * p.tiles_b * p.splits <= device_sm_count()) {
    if (pl.swap) return pl.bn == 16 ? launch_tile<16, true, true>(p, ta, tb, st) : launch_tile<32, true, true>(p, ta, tb, st);
    return pl.bn == 64 ? launch_tile<64, false, true>(p, ta, tb, st) : launch_tile<128, false, true>(p, ta, tb, st);
  }
  if (pl.swap) return pl.bn == 16 ? launch_tile<16, true, false>(p, ta, tb, st) : launch_tile<32, true, false>(p, ta, tb, st);
  return pl.bn == 64 ? launch_tile<64, false, false>(p, ta, tb, st) : launch_tile<128, false, false>(p, ta, tb, st);
}

}  // namespace jattn
