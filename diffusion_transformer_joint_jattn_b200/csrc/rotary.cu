// Rotary embedding of queries and keys that are not in the joint [B, S, 3, H,
// d] streams of the prologue: any strides, interleaved or half pairs, the
// first `rot` channels of each of `parts` equal parts of a head, one position
// per token or one per (t, row, col) axis, the frequencies given as a table.
//
//   (x_i, x_j) -> scale * (x_i cos a - x_j sin a, x_i sin a + x_j cos a),
//   a = pos * freq of the pair (negated for the inverse, which is also the
//   gradient: the transpose of a rotation); j = i + 1 or i + rot / 2.
//
// Bound by HBM: every element is read and written once and costs a few
// flops.  A block forms the fp64 angles of its tokens once; a thread owns U
// channel pairs of one token and walks heads of q and k with their cosines and
// sines in registers.  Its two 16-byte loads of a head are adjacent
// (interleaved, one access) or rot / 2 apart (half), kHeadsInFlight heads at a
// time.  Enough blocks per SM hide the loads better than several heads per
// thread do: 2 x 16896 tokens x 48 heads of 128 bf16 channels took 144 us with
// one head at 6 blocks per SM, 151 with two at 4, 177 with three at 4 (830 MB:
// 5.8 TB/s, 88% of a copy).  Those are interleaved pairs; half pairs of the same
// tensors take 171 us (bf16) and 165 (fp16): their accesses are 16 bytes, and the
// forms of 8 pairs spill 40 to 52 bytes at the 40 registers of 6 blocks.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "jattn.h"
#include "jattn_internal.h"
#include "rope_math.cuh"

namespace jattn {

namespace {

constexpr int kRotThreads = 256;
constexpr int kHeadsInFlight = 1;
constexpr int kRounds = 8;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// N elements of one access, at most 32 bytes (8 x 32 bits in one instruction:
// a thread's 16-byte halves of a 32-byte sector in two instructions would
// reach L2 as two partial writes).
template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
  T e[N];
};
template <typename T, int N>
__device__ __forceinline__ Vec<T, N> load_vec(const T* p) {
  if constexpr (sizeof(T) * N == 32) {
    union {
      Vec<T, N> v;
      uint32_t w[8];
    } r;
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]),
                   "=r"(r.w[7])
                 : "l"(p));
    return r.v;
  } else {
    return *reinterpret_cast<const Vec<T, N>*>(p);
  }
}
template <typename T, int N>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, N>& v) {
  if constexpr (sizeof(T) * N == 32) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(v.e);
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    *reinterpret_cast<Vec<T, N>*>(p) = v;
  }
}

// A block: p.tile tokens x p.units units x p.groups head groups = its 256
// threads (the last ones may be idle), units fastest, then tokens.  blockIdx.y
// = share of the heads.  Each (token, pair) angle is formed once per block, in
// shared memory; a thread then keeps its unit's in registers for all its
// heads.
// How a unit of U pairs lies in memory.
enum : int {
  kPairs = 0,       // interleaved: one access of 2 U channels
  kHalves = 1,      // half: two accesses of U channels, rot / 2 apart
  kSingles = 2,     // interleaved, U = 1, rows of odd strides: two single channels
};

template <typename T, int U, int MODE>
__global__ void __launch_bounds__(kRotThreads, 6) rotary_kernel(const RotaryParams p) {
  extern __shared__ float2 table[];                    // [tile][rot / 2]
  const int n_pairs = p.rot / 2;
  const long long tok0 = static_cast<long long>(blockIdx.x) * p.tile;
  for (int i = threadIdx.x; i < p.tile * n_pairs; i += kRotThreads) {
    const long long tok = tok0 + i / n_pairs;
    const int pair = i % n_pairs;
    if (tok < p.tokens) {
      const long long b = tok / p.S, s = tok % p.S;
      const int axis = pair < p.axis_end[0] ? 0 : (pair < p.axis_end[1] ? 1 : 2);
      float c, sn;
      angle_cos_sin(p.pos[b * p.pos_stride_b + s * p.n_axes + axis], p.freqs[pair], c, sn);
      table[i] = make_float2(c * p.scale, sn * (p.inverse ? -p.scale : p.scale));
    }
  }
  __syncthreads();
  const int u = threadIdx.x % p.units;
  const int at = threadIdx.x / p.units;
  const int tl = at % p.tile, group = at / p.tile;
  const long long tok = tok0 + tl;
  if (group >= p.groups || tok >= p.tokens) return;
  const int b = static_cast<int>(tok / p.S), s = static_cast<int>(tok % p.S);
  // channel offsets of the unit's accesses and its first pair
  constexpr bool HALF = MODE == kHalves;
  const int n_rot_units = HALF ? n_pairs / U : p.units;
  int c0 = u * 2 * U, c1 = c0 + U, pair0 = u * U;
  if (HALF && u < n_rot_units) {
    c0 = u * U;
    c1 = c0 + n_pairs;
  } else if (HALF) {
    c0 = p.rot + (u - n_rot_units) * 2 * U;
    c1 = c0 + U;
    pair0 = n_pairs;                                   // past the last pair: copied
  }
  float cs[U], sn[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const float2 e = pair0 + i < n_pairs ? table[tl * n_pairs + pair0 + i] : make_float2(1.f, 0.f);
    cs[i] = e.x;
    sn[i] = e.y;
  }
  const int n = p.d / p.parts;
  const int total = (p.H[0] + p.H[1]) * p.parts;
  const int step = p.groups * p.shares;                // head parts first, first + step, ...
  for (int h0 = blockIdx.y * p.groups + group; h0 < total; h0 += step * kHeadsInFlight) {
    constexpr int N = MODE == kPairs ? 2 * U : U, NV = MODE == kPairs ? 1 : 2;
    Vec<T, N> x[kHeadsInFlight][NV];
    T* dst[kHeadsInFlight];
#pragma unroll
    for (int k = 0; k < kHeadsInFlight; ++k) {
      const int hp = min(h0 + k * step, total - 1);
      const int head = hp / p.parts, part = hp % p.parts;
      const int t = head < p.H[0] ? 0 : 1;
      const int h = t == 0 ? head : head - p.H[0];
      const T* src = static_cast<const T*>(p.x[t]) + b * p.xs[t][0] + s * p.xs[t][1] + h * p.xs[t][2] + part * n;
      dst[k] = static_cast<T*>(p.y[t]) + b * p.ys[t][0] + s * p.ys[t][1] + h * p.ys[t][2] + part * n;
      if (h0 + k * step < total) {
        x[k][0] = load_vec<T, N>(src + c0);
        if constexpr (NV == 2) x[k][1] = load_vec<T, N>(src + c1);
      }
    }
#pragma unroll
    for (int k = 0; k < kHeadsInFlight; ++k) {
      if (h0 + k * step >= total) break;
      // pairs past rot are copied, not turned by 0: 0 * inf is NaN
      if (HALF ? u < n_rot_units : true) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
          T& first = NV == 2 ? x[k][0].e[i % N] : x[k][0].e[(2 * i) % N];
          T& second = NV == 2 ? x[k][NV - 1].e[i % N] : x[k][0].e[(2 * i + 1) % N];
          if (HALF || pair0 + i < n_pairs) {
            float y0, y1;
            rotate_pair(to_f32(first), to_f32(second), cs[i], sn[i], y0, y1);
            first = from_f32<T>(y0);
            second = from_f32<T>(y1);
          }
        }
      }
      store_vec<T, N>(dst[k] + c0, x[k][0]);
      if constexpr (NV == 2) store_vec<T, N>(dst[k] + c1, x[k][1]);
    }
  }
}

// Whether units of u pairs fit the layout: every access inside one region
// (rotated or copied), aligned, and of at most 16 bytes (half) or 32.
bool fits(const RotaryParams& p, int u, int esize, int mode) {
  const int n = p.d / p.parts, w = mode == kPairs ? 2 * u : u;   // elements of one access
  if (w * esize > (mode == kPairs ? 32 : 16) || n % (2 * u) != 0) return false;
  if (mode == kHalves && (p.rot / 2 % u != 0 || (n - p.rot) % (2 * u) != 0)) return false;
  const uintptr_t bytes = static_cast<uintptr_t>(w) * esize;
  for (int t = 0; t < 2; ++t) {
    if (p.H[t] == 0) continue;
    if (reinterpret_cast<uintptr_t>(p.x[t]) % bytes || reinterpret_cast<uintptr_t>(p.y[t]) % bytes) return false;
    for (int i = 0; i < 3; ++i)
      if (p.xs[t][i] % w || p.ys[t][i] % w) return false;
  }
  return true;
}

template <typename T, int U, int MODE>
cudaError_t launch_u(RotaryParams p, cudaStream_t st) {
  const int total = (p.H[0] + p.H[1]) * p.parts;
  p.units = p.d / p.parts / (2 * U);
  if (p.units > kRotThreads) return cudaErrorInvalidConfiguration;
  // Tokens and head groups per block: tile * groups slots of `units` threads.
  // Of the tiles whose rounds over the heads leave at most 5% more threads idle
  // than the best, the one nearest kRounds rounds (fewer: the angles are not
  // paid off; more: few tokens' rows per block); small problems take fewer
  // tokens, so that every SM has blocks.
  const int slots = kRotThreads / p.units;
  int rounds[kRotThreads + 1], used[kRotThreads + 1], best = 0;
  for (int tile = 1; tile <= slots; ++tile) {
    const int g = slots / tile < total ? slots / tile : total;
    rounds[tile] = (total + g - 1) / g;
    used[tile] = static_cast<int>(1000ll * total * tile / (static_cast<long long>(rounds[tile]) * slots));   // per mille
    if (used[tile] > best) best = used[tile];
  }
  p.tile = 1;
  int gap = INT32_MAX;
  for (int tile = 1; tile <= slots; ++tile) {
    const int d = rounds[tile] > kRounds ? rounds[tile] - kRounds : kRounds - rounds[tile];
    if (used[tile] >= best - 50 && d < gap && tile * p.rot * 4 <= 32768) {
      gap = d;
      p.tile = tile;
    }
  }
  while (p.tile > 1 && p.tokens / p.tile < 2 * 148) p.tile /= 2;
  p.groups = slots / p.tile < total ? slots / p.tile : total;
  const long long blocks = (p.tokens + p.tile - 1) / p.tile;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  // few tokens: the heads over more blocks
  const int most = (total + p.groups - 1) / p.groups;
  long long shares = (2 * 148 + blocks - 1) / blocks;
  if (shares > most) shares = most;
  p.shares = static_cast<int>(shares);
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(p.shares));
  const size_t smem = static_cast<size_t>(p.tile) * (p.rot / 2) * sizeof(float2);
  if (smem > 49152) return cudaErrorInvalidConfiguration;
  rotary_kernel<T, U, MODE><<<grid, kRotThreads, smem, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int MODE>
cudaError_t launch_mode(const RotaryParams& p, cudaStream_t st) {
  constexpr int es = sizeof(T);
  if constexpr (es == 2)
    if (fits(p, 8, es, MODE)) return launch_u<T, 8, MODE>(p, st);
  if (fits(p, 4, es, MODE)) return launch_u<T, 4, MODE>(p, st);
  if (fits(p, 2, es, MODE)) return launch_u<T, 2, MODE>(p, st);
  if (fits(p, 1, es, MODE)) return launch_u<T, 1, MODE>(p, st);
  return launch_u<T, 1, MODE == kPairs ? kSingles : MODE>(p, st);
}

template <typename T>
cudaError_t launch_dtype(const RotaryParams& p, bool half, cudaStream_t st) {
  return half ? launch_mode<T, kHalves>(p, st) : launch_mode<T, kPairs>(p, st);
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, int dtype, bool half, cudaStream_t st) {
  if (dtype == JATTN_FP32) return launch_dtype<float>(p, half, st);
  if (dtype == JATTN_FP16) return launch_dtype<__half>(p, half, st);
  return launch_dtype<__nv_bfloat16>(p, half, st);
}

}  // namespace jattn
