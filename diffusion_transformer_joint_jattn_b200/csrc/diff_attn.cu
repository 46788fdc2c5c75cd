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
// of its products: the exponentials bound it.
//   warps 0..3  softmax of map 0, warps 4..7 of map 1: one thread per query
//               row, online softmax with lazy rescale, P into the S columns;
//               then O_1 / l_1 - lambda O_2 / l_2 for half of the channels
//               each: both maps' accumulators lie in the same TMEM lanes, so
//               only the row sums and the norm's partial sums of squares go
//               through shared memory.
//   warp 8      MMA issuer, warp 9 TMA producer, warp 10 zeroes the V rows of
//               masked keys in shared memory (their P is 0, and 0 * NaN would
//               not be); warp 11 idle.
// Query rows of the heads that share a K/V head are packed into one row
// range where the strides allow it, so a cache is read once for the group.
// Few rows over a long cache: the keys are split over CTAs that write their
// normalised partial outputs and log-sum-exps, merged by a second kernel.
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
constexpr int kMmaWarp = 8, kProducerWarp = 9, kMaskWarp = 10;
constexpr int kThreads = 384;
// 2 x 128 x 216 + 128 x 72 = 64512 = 384 x 168, what the block launches with
constexpr uint32_t kRegsSoftmax = 216, kRegsOther = 72;
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleThreshold = 15.0f;   // log2 units; P <= 2^15 in 16 bits

__host__ __device__ constexpr uint32_t col_s(int t) { return static_cast<uint32_t>(t) * 128u; }
__host__ __device__ constexpr uint32_t col_o(int t) { return 256u + static_cast<uint32_t>(t) * 128u; }

template <int D>
struct Cfg {
  static constexpr int RB = D * 2;                    // row bytes
  static constexpr int NBOX = RB / 128;               // 128-byte swizzled boxes per tile
  static constexpr int BOXB = BM * 128;
  static constexpr int TB = BM * RB;
  static constexpr int KS = D == 128 ? 3 : 4;
  static constexpr int VS = D == 128 ? 3 : 4;
  static constexpr int SMEM = (1 + KS + VS) * TB + 256 + 1024;
};

struct __align__(8) Bars {
  uint64_t q_full;
  uint64_t k_full[4], k_empty[4];
  uint64_t v_full[4], v_empty[4], v_ready[4];
  uint64_t s_full[2], p_full[2], o_final[2];
  uint64_t exchange[2];
  uint64_t mma_final;
  uint32_t tmem_base;
  uint32_t abort;
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtl& ctl) {
  uint64_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    const bool ok = mbar_try_wait(bar, parity);
    if (__all_sync(0xffffffffu, ok)) return true;
    if ((i & 63u) == 63u) {
      int stop = 0;
      if (lane_id() == 0) {
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        if (*ctl.abort) stop = 1;
        else if (now - t0 > ctl.limit_ns) {
          atomicOr(ctl.status, JATTN_DEV_TIMEOUT);
          *ctl.abort = 1u;
          stop = 1;
        }
      }
      if (__shfl_sync(0xffffffffu, stop, 0)) return false;
    }
  }
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
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float row_max(const float (&v)[BN]) {
  float a[43];
#pragma unroll
  for (int i = 0; i < 42; ++i) a[i] = max3(v[3 * i], v[3 * i + 1], v[3 * i + 2]);
  a[42] = fmaxf(v[126], v[127]);
  float c[15];
#pragma unroll
  for (int i = 0; i < 14; ++i) c[i] = max3(a[3 * i], a[3 * i + 1], a[3 * i + 2]);
  c[14] = a[42];
  float e[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) e[i] = max3(c[3 * i], c[3 * i + 1], c[3 * i + 2]);
  return max3(e[0], e[1], fmaxf(e[2], fmaxf(e[3], e[4])));
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

// KIND: the operands' types and how P keeps its precision.  P in bf16 alone
// costs the output 1.9e-3 (relative, N(0, 1) inputs), more than the bf16
// output's own rounding, because the difference of the maps cancels.
enum : int {
  kF16 = 0,        // fp16 operands, P in fp16
  kBf16WideV = 1,  // bf16 Q and K; V converted to fp16 (scaled by a power of two per head), P in fp16
  kBf16Split = 2,  // bf16 operands, P as the sum of two bf16: twice the P.V products, no second copy of V
};

template <int D, int KIND>
__global__ void __launch_bounds__(kThreads, 1)
diff_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const DiffParams p) {
  using C = Cfg<D>;
  constexpr int DM = D / 2;
  constexpr bool QK_BF16 = KIND != kF16, PV_BF16 = KIND == kBf16Split;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + C::TB;
  uint8_t* sV = sK + C::KS * C::TB;
  Bars* bar = reinterpret_cast<Bars*>(sV + C::VS * C::TB);
  static_assert(sizeof(Bars) <= 256, "room for the barriers");
  // the epilogue's exchange lies over the Q tile, whose last use o_final proves
  float* sL = reinterpret_cast<float*>(sQ);                   // [2][BM] 1 / l
  float* sSq = sL + 2 * BM;                                   // [2][BM] sums of squares

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // this CTA's item: batch entry, group of heads, split of the keys, row tile
  int it = blockIdx.x;
  const int rt = it % p.n_rt;
  it /= p.n_rt;
  const int sp = it % p.splits;
  it /= p.splits;
  const int gi = it % p.n_groups, b = it / p.n_groups;
  const int kvh = static_cast<int>(static_cast<long long>(gi) * p.H_kv / p.n_groups);
  const int len = key_count(p, b);
  const int n_total = (len + BN - 1) / BN;
  const int t0 = static_cast<int>(static_cast<long long>(n_total) * sp / p.splits);
  const int n_kv = static_cast<int>(static_cast<long long>(n_total) * (sp + 1) / p.splits) - t0;
  const uint8_t* mask = p.key_mask != nullptr ? p.key_mask + static_cast<size_t>(b) * p.S_kv : nullptr;
  // V rows of masked keys have to be zeroed: a mask, or a length inside the
  // cache (rows past the cache arrive as zeros from TMA; the converted V has
  // its masked rows zeroed)
  const bool fix = KIND != kBf16WideV && (mask != nullptr || len < p.S_kv);

  if (threadIdx.x == 0) {
    mbar_init(&bar->q_full, 1);
    for (int s = 0; s < C::KS; ++s) {
      mbar_init(&bar->k_full[s], 1);
      mbar_init(&bar->k_empty[s], 1);
    }
    for (int s = 0; s < C::VS; ++s) {
      mbar_init(&bar->v_full[s], 1);
      mbar_init(&bar->v_empty[s], 1);
      mbar_init(&bar->v_ready[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bar->s_full[t], 1);
      mbar_init(&bar->p_full[t], BM);
      mbar_init(&bar->o_final[t], 1);
      mbar_init(&bar->exchange[t], 2 * BM);
    }
    mbar_init(&bar->mma_final, 1);
    bar->abort = 0;
    fence_mbarrier_init();
  }
  if (warp == kMmaWarp) {
    __syncwarp();
    tmem_alloc(&bar->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;
  const WaitCtl ctl{&bar->abort, p.status, p.timeout_ns};

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == kProducerWarp) {
      if (lane == 0 && n_kv > 0) {
        mbar_arrive_expect_tx(&bar->q_full, C::TB);
        for (int x = 0; x < C::NBOX; ++x) tma_load_4d(&tmQ, &bar->q_full, sQ + x * C::BOXB, x * 64, rt * BM, gi, b);
        int nk = 0, nv = 0;
        for (int j = 0; j < n_kv; ++j) {
          const int ks = nk % C::KS;
          if (!mbar_wait(&bar->k_empty[ks], ((nk / C::KS) & 1) ^ 1, ctl)) break;
          mbar_arrive_expect_tx(&bar->k_full[ks], C::TB);
          for (int x = 0; x < C::NBOX; ++x)
            tma_load_4d(&tmK, &bar->k_full[ks], sK + ks * C::TB + x * C::BOXB, x * 64, (t0 + j) * BN, kvh, b);
          ++nk;
          const int vs = nv % C::VS;
          if (!mbar_wait(&bar->v_empty[vs], ((nv / C::VS) & 1) ^ 1, ctl)) break;
          mbar_arrive_expect_tx(&bar->v_full[vs], C::TB);
          for (int x = 0; x < C::NBOX; ++x)
            tma_load_4d(&tmV, &bar->v_full[vs], sV + vs * C::TB + x * C::BOXB, x * 64, (t0 + j) * BN, kvh, b);
          ++nv;
        }
        // every load issued must have landed before the CTA may exit
        drain_wait(&bar->q_full, 0, ctl);
        for (int i = nk > C::KS ? nk - C::KS : 0; i < nk; ++i) drain_wait(&bar->k_full[i % C::KS], (i / C::KS) & 1, ctl);
        for (int i = nv > C::VS ? nv - C::VS : 0; i < nv; ++i) drain_wait(&bar->v_full[i % C::VS], (i / C::VS) & 1, ctl);
      }
    } else if (warp == kMmaWarp) {
      if (lane == 0 && n_kv > 0) {
        const uint32_t idesc_qk = instr_desc(QK_BF16, QK_BF16, 0, BM, BN);
        const uint32_t idesc_pv = instr_desc(PV_BF16, PV_BF16, 1, BM, D);
        const uint32_t sQa = smem_u32(sQ), sKa = smem_u32(sK), sVa = smem_u32(sV);
        bool any_mma = false;
        auto issue_qk = [&](int t, int ks) {
#pragma unroll
          for (int kk = 0; kk < DM / 16; ++kk) {
            const uint32_t at = t * DM * 2 + kk * 32;          // byte of the row
            const uint32_t off = at / 128 * C::BOXB + at % 128;
            mma_f16_ss(tmem + col_s(t), smem_desc(sQa + off, 16, 1024, 2u),
                       smem_desc(sKa + ks * C::TB + off, 16, 1024, 2u), idesc_qk, kk > 0);
          }
          any_mma = true;
        };
        auto issue_pv = [&](int t, int vs, bool acc) {
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            mma_f16_ts(tmem + col_o(t), tmem + col_s(t) + kk * 8,
                       smem_desc(sVa + vs * C::TB + kk * 16 * 128, C::BOXB, 1024, 2u), idesc_pv, acc || kk > 0);
          if constexpr (KIND == kBf16Split) {
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)               // the low parts, in the columns behind
              mma_f16_ts(tmem + col_o(t), tmem + col_s(t) + 64 + kk * 8,
                         smem_desc(sVa + vs * C::TB + kk * 16 * 128, C::BOXB, 1024, 2u), idesc_pv, 1);
          }
        };
        bool ok = mbar_wait(&bar->q_full, 0, ctl) && mbar_wait(&bar->k_full[0], 0, ctl);
        if (ok) {
          tc_fence_after();
          for (int t = 0; t < 2; ++t) {
            issue_qk(t, 0);
            mma_commit(&bar->s_full[t]);
          }
          mma_commit(&bar->k_empty[0]);
        }
        for (int j = 0; j < n_kv && ok; ++j) {
          const int vs = j % C::VS, ks = (j + 1) % C::KS;
          const bool more = j + 1 < n_kv;
          ok = mbar_wait(fix ? &bar->v_ready[vs] : &bar->v_full[vs], (j / C::VS) & 1, ctl);
          for (int t = 0; t < 2 && ok; ++t) {
            ok = mbar_wait(&bar->p_full[t], j & 1, ctl);
            if (!ok) break;
            tc_fence_after();
            issue_pv(t, vs, j > 0);
            if (t == 1) mma_commit(&bar->v_empty[vs]);
            if (more) {
              if (t == 0) {
                ok = mbar_wait(&bar->k_full[ks], ((j + 1) / C::KS) & 1, ctl);
                if (!ok) break;
                tc_fence_after();
              }
              issue_qk(t, ks);
              mma_commit(&bar->s_full[t]);
              if (t == 1) mma_commit(&bar->k_empty[ks]);
            } else {
              mma_commit(&bar->o_final[t]);
            }
          }
        }
        if (any_mma) {
          mma_commit(&bar->mma_final);
          drain_wait(&bar->mma_final, 0, ctl);
        }
      }
    } else if (warp == kMaskWarp && fix) {
      for (int j = 0; j < n_kv; ++j) {
        const int vs = j % C::VS, key0 = (t0 + j) * BN;
        bool drop[4];                                   // keys key0 + 32 w + lane
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int key = key0 + 32 * w + lane;
          drop[w] = key < p.S_kv && (key >= len || (mask != nullptr && __ldg(mask + key) == 0));
        }
        if (!warp_wait(&bar->v_full[vs], (j / C::VS) & 1, ctl)) break;
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
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int t = warp >> 2;                            // map of this warpgroup
    const int row = (warp & 3) * 32 + lane;             // TMEM lane == row in the tile
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_base + col_s(t), to = tmem + lane_base + col_o(t);
    const int r = rt * BM + row;                        // row of the group
    const bool live = r < p.R;
    const bool warp_live = rt * BM + (warp & 3) * 32 < p.R;
    const int head = gi * p.hpg + (live ? r / p.S_q : 0), s_q = live ? r % p.S_q : 0;
    const float c_j = p.scale_log2;
    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;
    uint8_t mb[4] = {1, 1, 1, 1};
    auto load_mask = [&](int kt) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int key = kt * BN + 32 * w + lane;
        mb[w] = key < p.S_kv ? __ldg(mask + key) : 0;
      }
    };
    if (mask != nullptr && n_kv > 0) load_mask(t0);
    for (int j = 0; j < n_kv; ++j) {
      const int kt = t0 + j;
      uint32_t keep[4] = {~0u, ~0u, ~0u, ~0u};
      if (mask != nullptr) {
#pragma unroll
        for (int w = 0; w < 4; ++w) keep[w] = __ballot_sync(0xffffffffu, mb[w] != 0);
        if (j + 1 < n_kv) load_mask(kt + 1);
      }
      ok = warp_wait(&bar->s_full[t], j & 1, ctl);
      if (!ok) break;
      __syncwarp();
      if (!warp_live) {                                 // rows past the last: nothing to compute
        mbar_arrive(&bar->p_full[t]);
        continue;
      }
      tc_fence_after();
      float v[BN];
      {
        uint32_t raw[BN];
        tmem_ld128(ts, raw);
#pragma unroll
        for (int e = 0; e < BN; ++e) v[e] = __uint_as_float(raw[e]);
      }
      const int valid = len - kt * BN;
      if (valid < BN) {
#pragma unroll
        for (int e = 0; e < BN; ++e)
          if (e >= valid) v[e] = -INFINITY;
      }
      if ((keep[0] & keep[1] & keep[2] & keep[3]) != ~0u) {
#pragma unroll
        for (int e = 0; e < BN; ++e)
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
      if (j > 0 && __any_sync(0xffffffffu, resc)) {
        // O_t is stable here: PV_t(j-1) completed before S_t(j) was signalled
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(to + c * 32, o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
          tmem_st32(to + c * 32, o);
        }
      }
      // no key so far: every probability is exp2(-inf) = 0
      const float neg_m = m_run == -INFINITY ? 0.f : -m_run;
      const float2 c2 = make_float2(c_j, c_j), nm2 = make_float2(neg_m, neg_m);
      float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t pk[32], lo[KIND == kBf16Split ? 32 : 1];
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const int e = half * 64 + 2 * c;
          const float2 x0 = __ffma2_rn(make_float2(v[e + 0], v[e + 1]), c2, nm2);
          const float2 x1 = __ffma2_rn(make_float2(v[e + 2], v[e + 3]), c2, nm2);
          const float2 e0 = make_float2(ex2_approx(x0.x), ex2_approx(x0.y));
          const float2 e1 = make_float2(ex2_approx(x1.x), ex2_approx(x1.y));
          acc0 = __fadd2_rn(acc0, e0);
          acc1 = __fadd2_rn(acc1, e1);
          // P in V's type (the MMA wants one type); l sums the unrounded values
          pk[c] = pack_x2<PV_BF16>(e0.x, e0.y);
          pk[c + 1] = pack_x2<PV_BF16>(e1.x, e1.y);
          if constexpr (KIND == kBf16Split) {
            lo[c] = pack_x2<true>(e0.x - __uint_as_float(pk[c] << 16), e0.y - __uint_as_float(pk[c] & 0xFFFF0000u));
            lo[c + 1] = pack_x2<true>(e1.x - __uint_as_float(pk[c + 1] << 16),
                                      e1.y - __uint_as_float(pk[c + 1] & 0xFFFF0000u));
          }
        }
        tmem_st32(ts + half * 32, pk);
        if constexpr (KIND == kBf16Split) tmem_st32(ts + 64 + half * 32, lo);
      }
      l_run += (acc0.x + acc0.y) + (acc1.x + acc1.y);
      tc_fence_before();
      mbar_arrive(&bar->p_full[t]);
    }
    if (ok && n_kv > 0) ok = warp_wait(&bar->o_final[t], 0, ctl);
    __syncwarp();
    tc_fence_after();
    float inv = l_run == 0.f ? 0.f : 1.f / l_run;
    if constexpr (KIND == kBf16WideV)                   // undo V's power of two
      inv *= pow2(v_exponent(__ldg(p.v_amax + static_cast<size_t>(b) * p.H_kv + kvh)));
    const float lse2 = l_run == 0.f ? -INFINITY : m_run + __log2f(l_run);
    const size_t rows = static_cast<size_t>(p.B) * p.H * p.S_q;
    const size_t rg = (static_cast<size_t>(b) * p.H + head) * p.S_q + s_q;
    if (p.splits > 1) {
      // this split's normalised output and log-sum-exp of its map
      if (ok && warp_live) {
        const size_t at = (static_cast<size_t>(sp) * 2 + t) * rows + rg;
        float* dst = p.part_o + at * D;
        if (n_kv > 0) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            __syncwarp();
            tmem_ld32(to + c, o);
            if (live) {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4*>(dst + c + e) =
                    make_float4(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv,
                                __uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
            }
          }
        }
        // a split without keys leaves its output unwritten: weight 0 by its -inf
        if (live) p.part_l[at] = lse2;
      }
    } else {
      const float lam = ok && live ? lambda_of(p, head, DM) : 0.f;
      sL[t * BM + row] = inv;
      tc_fence_before();
      mbar_arrive(&bar->exchange[0]);
      ok = warp_wait(&bar->exchange[0], 0, ctl) && ok;
      tc_fence_after();
      // channels [t * D / 2, +D / 2) of the row
      const float w1 = sL[row], w2 = -lam * sL[BM + row];
      float o[DM];
      float sq = 0.f;
      __syncwarp();
      if (n_kv > 0 && ok) {
        const uint32_t o1 = tmem + lane_base + col_o(0) + t * DM, o2 = tmem + lane_base + col_o(1) + t * DM;
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
      if (p.norm_w != nullptr) {
        sSq[t * BM + row] = sq;
        mbar_arrive(&bar->exchange[1]);
        ok = warp_wait(&bar->exchange[1], 0, ctl) && ok;
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
      if (ok && live) {
        __nv_bfloat16* dst = p.o + ((static_cast<size_t>(b) * p.S_q + s_q) * p.H + head) * D + t * DM;
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
        if (p.lse != nullptr) p.lse[static_cast<size_t>(t) * rows + rg] = lse2 * 0.69314718055994531f;
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

// Merge of the splits, one warp per query row: each map's outputs weighted by
// 2^(lse_s - lse), then the difference and the norm.
template <int D>
__global__ void __launch_bounds__(128) diff_merge_kernel(const DiffParams p) {
  constexpr int E = D / 32;                             // channels per lane
  const int lane = threadIdx.x & 31;
  const size_t rows = static_cast<size_t>(p.B) * p.H * p.S_q;
  const size_t rg = static_cast<size_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (rg >= rows) return;
  const int s_q = static_cast<int>(rg % p.S_q);
  const size_t bh = rg / p.S_q;
  const int head = static_cast<int>(bh % p.H), b = static_cast<int>(bh / p.H);
  float a1 = 0.f, a2 = 0.f;
  const size_t plane = static_cast<size_t>(p.H) * (D / 2);
  for (int i = lane; i < D / 2; i += 32) {
    const float* l = p.lam + static_cast<size_t>(head) * (D / 2) + i;
    a1 = fmaf(l[0], l[plane], a1);
    a2 = fmaf(l[2 * plane], l[3 * plane], a2);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a1 += __shfl_xor_sync(0xffffffffu, a1, o);
    a2 += __shfl_xor_sync(0xffffffffu, a2, o);
  }
  const float lam = expf(a1) - expf(a2) + p.lambda_init;
  float out[E];
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = 0.f;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    float mx = -INFINITY;
    for (int s = 0; s < p.splits; ++s) {
      const float l = p.part_l[(static_cast<size_t>(s) * 2 + t) * rows + rg];
      mx = l > mx || l != l ? l : mx;                   // a NaN stays
    }
    float acc[E], tot = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    if (mx != -INFINITY) {
      for (int s = 0; s < p.splits; ++s) {
        const size_t at = (static_cast<size_t>(s) * 2 + t) * rows + rg;
        const float l = p.part_l[at];
        if (l == -INFINITY) continue;                   // no keys: its output was not written
        const float w = ex2_approx(l - mx);
        tot += w;
        const float* src = p.part_o + at * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(w, src[e], acc[e]);
      }
    }
    const float inv = mx == -INFINITY ? 0.f : 1.f / tot;
    const float f = t == 0 ? inv : -lam * inv;
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] = fmaf(f, acc[e], out[e]);
    if (p.lse != nullptr && lane == 0)
      p.lse[static_cast<size_t>(t) * rows + rg] =
          mx == -INFINITY ? -INFINITY : (mx + __log2f(tot)) * 0.69314718055994531f;
  }
  if (p.norm_w != nullptr) {
    float sq = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) sq = fmaf(out[e], out[e], sq);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    const float f = rsqrtf(sq * (1.f / D) + p.eps) * (1.f - p.lambda_init);
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] *= f * __ldg(p.norm_w + lane * E + e);
  }
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + ((static_cast<size_t>(b) * p.S_q + s_q) * p.H + head) * D) + lane * (E / 2);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) dst[e] = pack_x2<true>(out[2 * e], out[2 * e + 1]);
}

template <int D, int KIND>
cudaError_t launch_t(const DiffParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                     cudaStream_t st) {
  using C = Cfg<D>;
  static_assert(C::SMEM <= 232448, "shared memory budget");
  auto kern = diff_attn_kernel<D, KIND>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  if (KIND == kBf16WideV && p.S_kv > 0) {
    const dim3 grid(static_cast<unsigned>((p.S_kv + kConvRows - 1) / kConvRows), static_cast<unsigned>(p.B * p.H_kv));
    if ((e = cudaMemsetAsync(p.v_amax, 0, static_cast<size_t>(p.B) * p.H_kv * 4, st)) != cudaSuccess) return e;
    widen_v_kernel<D, false><<<grid, 256, 0, st>>>(p);
    widen_v_kernel<D, true><<<grid, 256, 0, st>>>(p);
  }
  const long long items = static_cast<long long>(p.B) * p.n_groups * p.splits * p.n_rt;
  kern<<<static_cast<unsigned>(items), kThreads, C::SMEM, st>>>(tq, tk, tv, p);
  if ((e = cudaGetLastError()) != cudaSuccess || p.splits == 1) return e;
  const size_t rows = static_cast<size_t>(p.B) * p.H * p.S_q;
  diff_merge_kernel<D><<<static_cast<unsigned>((rows + 3) / 4), 128, 0, st>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const DiffParams& p, bool in_bf16, const CUtensorMap& tq, const CUtensorMap& tk,
                     const CUtensorMap& tv, cudaStream_t st) {
  if (!in_bf16) return launch_t<D, kF16>(p, tq, tk, tv, st);
  return p.v16 != nullptr ? launch_t<D, kBf16WideV>(p, tq, tk, tv, st) : launch_t<D, kBf16Split>(p, tq, tk, tv, st);
}

}  // namespace

// Splits of the keys: none while the items alone give every SM a CTA.
int diff_splits(long long items, int S_kv) {
  const int tiles = (S_kv + BN - 1) / BN;
  if (items >= 148 || tiles < 8) return 1;
  long long s = 444 / items;
  if (s > tiles / 4) s = tiles / 4;
  if (s > 64) s = 64;
  return s < 1 ? 1 : static_cast<int>(s);
}

// Whether bf16 operands get an fp16 copy of V: worth its three passes over V
// once several row tiles walk each V tile.
bool diff_widens_v(int n_rt) { return n_rt >= 4; }

cudaError_t launch_diff_attn(const DiffParams& p, int d, bool in_bf16, const CUtensorMap& tq, const CUtensorMap& tk,
                             const CUtensorMap& tv, cudaStream_t st) {
  return d == 128 ? launch_d<128>(p, in_bf16, tq, tk, tv, st) : launch_d<64>(p, in_bf16, tq, tk, tv, st);
}

}  // namespace jattn
