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
// (interleaved) or rot / 2 apart (half), kHeadsInFlight heads at a time.
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
constexpr int kHeadsInFlight = 2;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

template <typename T, int U>
struct alignas(sizeof(T) * U) Vec {
  T e[U];
};

// A block: p.tile tokens x p.units units x p.groups head groups = its 256
// threads (the last ones may be idle), units fastest, then tokens.  blockIdx.y
// = share of the heads.  Each (token, pair) angle is formed once per block, in
// shared memory; a thread then keeps its unit's in registers for all its
// heads.
template <typename T, int U, bool HALF>
__global__ void __launch_bounds__(kRotThreads, 3) rotary_kernel(const RotaryParams p) {
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
  // channel offsets of the unit's two vectors and its first pair
  const int n_rot_units = HALF ? n_pairs / U : p.units;
  int c0, c1, pair0;
  if (HALF && u < n_rot_units) {
    c0 = u * U;
    c1 = c0 + n_pairs;
    pair0 = c0;
  } else if (HALF) {
    c0 = p.rot + (u - n_rot_units) * 2 * U;
    c1 = c0 + U;
    pair0 = n_pairs;                                   // past the last pair: copied
  } else {
    c0 = u * 2 * U;
    c1 = c0 + U;
    pair0 = u * U;
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
  using V = Vec<T, U>;
  for (int h0 = blockIdx.y * p.groups + group; h0 < total; h0 += step * kHeadsInFlight) {
    V a[kHeadsInFlight], c[kHeadsInFlight];
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
        a[k] = *reinterpret_cast<const V*>(src + c0);
        c[k] = *reinterpret_cast<const V*>(src + c1);
      }
    }
#pragma unroll
    for (int k = 0; k < kHeadsInFlight; ++k) {
      if (h0 + k * step >= total) break;
      // pairs past rot have cos 1 and sin 0, but are copied: 0 * inf is NaN
      if (HALF) {
        if (u < n_rot_units) {
#pragma unroll
          for (int i = 0; i < U; ++i) {
            float y0, y1;
            rotate_pair(to_f32(a[k].e[i]), to_f32(c[k].e[i]), cs[i], sn[i], y0, y1);
            a[k].e[i] = from_f32<T>(y0);
            c[k].e[i] = from_f32<T>(y1);
          }
        }
      } else {
        T v[2 * U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          v[i] = a[k].e[i];
          v[U + i] = c[k].e[i];
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          if (pair0 + i < n_pairs) {
            float y0, y1;
            rotate_pair(to_f32(v[2 * i]), to_f32(v[2 * i + 1]), cs[i], sn[i], y0, y1);
            v[2 * i] = from_f32<T>(y0);
            v[2 * i + 1] = from_f32<T>(y1);
          }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          a[k].e[i] = v[i];
          c[k].e[i] = v[U + i];
        }
      }
      *reinterpret_cast<V*>(dst[k] + c0) = a[k];
      *reinterpret_cast<V*>(dst[k] + c1) = c[k];
    }
  }
}

// Whether U elements per vector fit the layout: both vectors of every unit
// inside one region (rotated or copied) and aligned.
bool fits(const RotaryParams& p, int u, int esize, bool half) {
  const int n = p.d / p.parts;
  if (u * esize > 16) return false;
  if (half ? (p.rot / 2 % u != 0 || (n - p.rot) % (2 * u) != 0) : n % (2 * u) != 0) return false;
  if (n % u != 0) return false;
  const int64_t bytes = static_cast<int64_t>(u) * esize;
  for (int t = 0; t < 2; ++t) {
    if (p.H[t] == 0) continue;
    if (reinterpret_cast<uintptr_t>(p.x[t]) % bytes || reinterpret_cast<uintptr_t>(p.y[t]) % bytes) return false;
    for (int i = 0; i < 3; ++i)
      if (p.xs[t][i] % u || p.ys[t][i] % u) return false;
  }
  return true;
}

template <typename T, int U>
cudaError_t launch_u(RotaryParams p, bool half, cudaStream_t st) {
  const int total = (p.H[0] + p.H[1]) * p.parts;
  p.units = p.d / p.parts / (2 * U);
  if (p.units > kRotThreads) return cudaErrorInvalidConfiguration;
  // Tokens per block: 8 heads of each in flight side by side where there are
  // that many tokens for every SM; then as many head groups as threads are left.
  const int slots = kRotThreads / p.units;
  p.tile = slots / 8 > 0 ? slots / 8 : 1;
  while (p.tile > 1 && p.tokens / p.tile < 2 * 148) p.tile /= 2;
  while (p.tile > 1 && p.tile * p.rot * 4 > 32768) p.tile /= 2;
  p.groups = slots / p.tile;
  if (p.groups > total) p.groups = total;
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
  if (half) rotary_kernel<T, U, true><<<grid, kRotThreads, smem, st>>>(p);
  else rotary_kernel<T, U, false><<<grid, kRotThreads, smem, st>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_dtype(const RotaryParams& p, bool half, cudaStream_t st) {
  if constexpr (sizeof(T) == 2)
    if (fits(p, 8, 2, half)) return launch_u<T, 8>(p, half, st);
  if (fits(p, 4, sizeof(T), half)) return launch_u<T, 4>(p, half, st);
  if (fits(p, 2, sizeof(T), half)) return launch_u<T, 2>(p, half, st);
  return launch_u<T, 1>(p, half, st);
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, int dtype, bool half, cudaStream_t st) {
  if (dtype == JATTN_FP32) return launch_dtype<float>(p, half, st);
  if (dtype == JATTN_FP16) return launch_dtype<__half>(p, half, st);
  return launch_dtype<__nv_bfloat16>(p, half, st);
}

}  // namespace jattn
