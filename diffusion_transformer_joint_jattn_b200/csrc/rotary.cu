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
// flops.  A thread owns U channel pairs of one token and walks a share of
// the heads of q and k with their cosines and sines in registers, so the
// fp64 angles and the sincos are paid once per share and no table passes
// through memory.  Its two 16-byte loads of a head are adjacent (interleaved)
// or rot / 2 apart (half); four heads are in flight per thread.
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
constexpr int kHeadsInFlight = 4;

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

// One thread: token = (b, s), unit u of a part, heads [share * per, +per) of
// the H_q * parts + H_k * parts head parts.
template <typename T, int U, bool HALF>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotaryParams p) {
  const long long gid = static_cast<long long>(blockIdx.x) * kRotThreads + threadIdx.x;
  const int u = static_cast<int>(gid % p.units);
  const long long rest = gid / p.units;
  const long long tok = rest % p.tokens;
  const long long share = rest / p.tokens;
  if (share >= p.shares) return;
  const int b = static_cast<int>(tok / p.S), s = static_cast<int>(tok % p.S);
  // channel offsets of the unit's two vectors and its first pair
  const int n_rot_units = HALF ? p.rot / 2 / U : p.units;
  int c0, c1, pair0;
  if (HALF && u < n_rot_units) {
    c0 = u * U;
    c1 = c0 + p.rot / 2;
    pair0 = c0;
  } else if (HALF) {
    c0 = p.rot + (u - n_rot_units) * 2 * U;
    c1 = c0 + U;
    pair0 = p.rot / 2;                              // past the last pair: copied
  } else {
    c0 = u * 2 * U;
    c1 = c0 + U;
    pair0 = u * U;
  }
  float cs[U], sn[U];
  const int32_t* pos = p.pos + static_cast<long long>(b) * p.pos_stride_b + static_cast<long long>(s) * p.n_axes;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
    const int pair = pair0 + i;
    if (pair < p.rot / 2) {
      const int axis = pair < p.axis_end[0] ? 0 : (pair < p.axis_end[1] ? 1 : 2);
      angle_cos_sin(pos[axis], p.freqs[pair], cs[i], sn[i]);
      cs[i] *= p.scale;
      sn[i] *= p.inverse ? -p.scale : p.scale;
    }
  }
  const int n = p.d / p.parts;
  const int total = (p.H[0] + p.H[1]) * p.parts;
  const int lo = static_cast<int>(share) * p.per, hi = min(lo + p.per, total);
  using V = Vec<T, U>;
  for (int h0 = lo; h0 < hi; h0 += kHeadsInFlight) {
    V a[kHeadsInFlight], c[kHeadsInFlight];
    T* dst[kHeadsInFlight];
#pragma unroll
    for (int k = 0; k < kHeadsInFlight; ++k) {
      const int hp = min(h0 + k, hi - 1);
      const int head = hp / p.parts, part = hp % p.parts;
      const int t = head < p.H[0] ? 0 : 1;
      const int h = t == 0 ? head : head - p.H[0];
      const T* src = static_cast<const T*>(p.x[t]) + b * p.xs[t][0] + s * p.xs[t][1] + h * p.xs[t][2] + part * n;
      dst[k] = static_cast<T*>(p.y[t]) + b * p.ys[t][0] + s * p.ys[t][1] + h * p.ys[t][2] + part * n;
      if (h0 + k < hi) {
        a[k] = *reinterpret_cast<const V*>(src + c0);
        c[k] = *reinterpret_cast<const V*>(src + c1);
      }
    }
#pragma unroll
    for (int k = 0; k < kHeadsInFlight; ++k) {
      if (h0 + k >= hi) break;
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
          if (pair0 + i < p.rot / 2) {
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
  // Heads per thread: as many as leave two full waves of threads (148 SMs x
  // 2048) busy, at least one batch of kHeadsInFlight (fewer heads per thread
  // only repeat the angles once the GPU is full).
  const long long owners = p.tokens * p.units;
  long long shares = (2ll * 148 * 2048 + owners - 1) / owners;
  const long long most = (total + kHeadsInFlight - 1) / kHeadsInFlight;
  if (shares > most) shares = most;
  p.per = static_cast<int>((total + shares - 1) / shares);
  p.shares = (total + p.per - 1) / p.per;
  const long long blocks = (owners * p.shares + kRotThreads - 1) / kRotThreads;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  if (half) rotary_kernel<T, U, true><<<static_cast<unsigned>(blocks), kRotThreads, 0, st>>>(p);
  else rotary_kernel<T, U, false><<<static_cast<unsigned>(blocks), kRotThreads, 0, st>>>(p);
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
