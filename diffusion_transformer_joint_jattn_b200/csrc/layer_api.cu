// C-ABI entry points of the layer around the attention (rotary embedding,
// linear layer, differential attention): argument validation before any
// launch, tensor maps, launches on the caller's stream.
#include <cmath>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "jattn.h"
#include "jattn_internal.h"

namespace {

constexpr uint64_t kTimeoutNs = 2000000000ull;   // 2 s per pipeline wait

bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
int elem_bytes(jattn_dtype t) { return t == JATTN_FP32 ? 4 : 2; }
bool is_16bit(jattn_dtype t) { return t == JATTN_BF16 || t == JATTN_FP16; }
bool is_float(jattn_dtype t) { return is_16bit(t) || t == JATTN_FP32; }

jattn_status from_cuda(cudaError_t e) { return e == cudaSuccess ? JATTN_OK : JATTN_ERR_CUDA; }

// 2-D map of a [rows][cols] 16-bit matrix, boxes of 64 columns x box_rows.
bool matrix_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
  const uint64_t dims[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)};
  const uint64_t strides[1] = {static_cast<uint64_t>(rows > 1 ? ld : (cols + 7) / 8 * 8) * 2};
  const uint32_t box[2] = {64u, static_cast<uint32_t>(box_rows)};
  return jattn::encode_map16(m, base, 2, dims, strides, box);
}

// (d, rows, heads, batch) map of 16-bit elements, boxes of 64 channels x
// box_rows rows; a dimension of one element gets a harmless stride.
bool heads_map(CUtensorMap* m, const void* base, int d, int64_t rows, int64_t heads, int64_t batch, int64_t row_stride,
               int64_t head_stride, int64_t batch_stride, int box_rows = 128) {
  const uint64_t dims[4] = {static_cast<uint64_t>(d), static_cast<uint64_t>(rows), static_cast<uint64_t>(heads),
                            static_cast<uint64_t>(batch)};
  const uint64_t strides[3] = {static_cast<uint64_t>(rows > 1 ? row_stride : d) * 2,
                               static_cast<uint64_t>(heads > 1 ? head_stride : d) * 2,
                               static_cast<uint64_t>(batch > 1 ? batch_stride : d) * 2};
  const uint32_t box[4] = {64u, static_cast<uint32_t>(box_rows), 1u, 1u};
  return jattn::encode_map16(m, base, 4, dims, strides, box);
}

// Row ranges of a call: the rows of the heads that share a K/V head form one
// range when they are equally spaced in memory.
struct DiffRanges {
  int n_groups, hpg, R, n_rt;
  int64_t items;
  jattn::DiffWalk walk;
  bool widen;                   // with bf16 operands
  int64_t row_stride, group_stride;
};

jattn_status diff_ranges(const jattn_diff_shape* s, DiffRanges* r) {
  if (s == nullptr) return JATTN_ERR_INVALID_ARG;
  if (s->B < 0 || s->H < 1 || s->H_kv < 1 || s->S_q < 0 || s->S_kv < 0) return JATTN_ERR_INVALID_ARG;
  if (s->S_q > (1 << 24) || s->S_kv > (1 << 24) || s->H % s->H_kv != 0) return JATTN_ERR_INVALID_ARG;
  if (static_cast<int64_t>(s->B) * s->H > 65535) return JATTN_ERR_INVALID_ARG;
  if (s->d != 64 && s->d != 128) return JATTN_ERR_UNSUPPORTED;
  const int64_t size[3][3] = {{s->B, s->H, s->S_q}, {s->B, s->H_kv, s->S_kv}, {s->B, s->H_kv, s->S_kv}};
  const int64_t* stride[3] = {s->q_stride, s->k_stride, s->v_stride};
  for (int t = 0; t < 3; ++t)
    for (int i = 0; i < 3 && size[t][0] * size[t][2] > 0; ++i)     // no elements: no strides
      if (size[t][i] > 1 && (stride[t][i] < s->d || stride[t][i] % 8 != 0 || stride[t][i] >= (int64_t{1} << 38)))
        return JATTN_ERR_INVALID_ARG;
  const int G = s->H / s->H_kv;
  const bool packed = G == 1 || s->S_q == 1 || s->q_stride[1] == s->S_q * s->q_stride[2];
  r->n_groups = packed ? s->H_kv : s->H;
  r->hpg = packed ? G : 1;
  const int64_t rows = static_cast<int64_t>(r->hpg) * s->S_q;
  r->n_rt = static_cast<int>((rows + 127) / 128);
  if (rows > (1 << 30) || static_cast<int64_t>(s->B) * r->n_groups * r->n_rt > (1 << 30)) return JATTN_ERR_INVALID_ARG;
  r->R = static_cast<int>(rows);
  r->row_stride = s->S_q == 1 ? s->q_stride[1] : s->q_stride[2];
  r->group_stride = r->hpg * s->q_stride[1];
  r->items = static_cast<int64_t>(s->B) * r->n_groups * r->n_rt;
  const int sms = jattn::device_sm_count();
  r->walk = jattn::diff_walk(r->items, r->n_rt, s->S_kv, sms);
  r->widen = jattn::diff_widens_v(r->items, r->n_rt, s->S_kv, sms);
  return JATTN_OK;
}

// Workspace segments, each 256-byte aligned: the splits' partial results, the
// sums that long walks empty their accumulators into, the fp16 copy of V and its
// per-head magnitudes.
struct DiffLayout {
  size_t part_o, part_l, sums, sums_m, v16, v_amax, total;
};

DiffLayout diff_layout(const jattn_diff_shape* s, const DiffRanges& r, bool in_bf16) {
  DiffLayout L{};
  size_t off = 0;
  auto seg = [&](size_t bytes) { const size_t at = off; off += (bytes + 255) / 256 * 256; return at; };
  if (r.walk.merge) {
    L.part_o = seg(static_cast<size_t>(r.walk.ctas) * 4 * 128 * s->d * 4);
    L.part_l = seg(static_cast<size_t>(r.walk.ctas) * 4 * 128 * 4);
  }
  if (s->S_kv > jattn::kGatherKeys) {
    L.sums = seg(static_cast<size_t>(r.walk.ctas) * 256 * s->d * 4);
    L.sums_m = seg(static_cast<size_t>(r.walk.ctas) * 256 * 4);
  }
  if (in_bf16 && r.widen) {
    L.v16 = seg(static_cast<size_t>(s->B) * s->H_kv * s->S_kv * s->d * 2);
    L.v_amax = seg(static_cast<size_t>(s->B) * s->H_kv * 4);
  }
  L.total = off;
  return L;
}

bool linear_sizes(const jattn_linear_shape* s) {
  const int32_t most = 1 << 30;
  return s != nullptr && s->M >= 0 && s->M <= most && s->N >= 0 && s->N <= most && s->K >= 1 && s->K <= most;
}
int64_t padded(int64_t k) { return (k + 7) / 8 * 8; }

// Which operands of the linear layer TMA cannot address (one row needs no
// stride), and where their copies go in the workspace.
struct LinearCopies {
  bool x, w;
  size_t w_at, total;
};

LinearCopies linear_copies(const jattn_linear_shape* s, const void* x, const void* w) {
  LinearCopies c{};
  if (s->M == 0 || s->N == 0) return c;
  auto bytes = [&](int64_t rows) { return (static_cast<size_t>(rows) * padded(s->K) * 2 + 255) / 256 * 256; };
  c.x = !aligned(x, 16) || (s->M > 1 && s->ldx % 8 != 0);
  c.w = !aligned(w, 16) || (s->N > 1 && s->ldw % 8 != 0);
  c.w_at = c.x ? bytes(s->M) : 0;
  c.total = c.w_at + (c.w ? bytes(s->N) : 0);
  return c;
}

}  // namespace

namespace jattn {

int device_sm_count() {
  static int cached[64] = {};
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  if (cached[dev] > 0) return cached[dev];
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
  cached[dev] = n;
  return n;
}

}  // namespace jattn

extern "C" {

jattn_status jattn_rotary(const jattn_rotary_tensor* tensors, int32_t n_tensors, jattn_dtype dtype, int32_t B,
                          int32_t S, int32_t d, int32_t parts, int32_t rot, const int32_t* pos,
                          int64_t pos_stride_b, const int32_t* split, const double* freqs,
                          jattn_rotary_layout layout, float scale, int32_t inverse, void* stream) {
  if (tensors == nullptr || n_tensors < 1 || n_tensors > 2 || B < 0 || S < 0 || d < 2 || d > 8192 || parts < 1)
    return JATTN_ERR_INVALID_ARG;
  if (!is_float(dtype)) return JATTN_ERR_UNSUPPORTED;
  if (layout != JATTN_ROTARY_INTERLEAVED && layout != JATTN_ROTARY_HALF) return JATTN_ERR_INVALID_ARG;
  if (d % parts != 0 || d / parts % 2 != 0 || rot < 2 || rot % 2 != 0 || rot > d / parts || d / parts > 512)
    return JATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return JATTN_ERR_INVALID_ARG;
  jattn::RotaryParams p{};
  p.axis_end[0] = p.axis_end[1] = p.axis_end[2] = rot / 2;
  p.n_axes = 1;
  if (split != nullptr) {
    if (split[0] < 0 || split[1] < 0 || split[2] < 0 || ((split[0] | split[1] | split[2]) & 1) != 0 ||
        static_cast<int64_t>(split[0]) + split[1] + split[2] != rot)
      return JATTN_ERR_INVALID_ARG;
    p.n_axes = 3;
    p.axis_end[0] = split[0] / 2;
    p.axis_end[1] = (split[0] + split[1]) / 2;
  }
  int64_t heads = 0;
  for (int t = 0; t < n_tensors; ++t) {
    const jattn_rotary_tensor& x = tensors[t];
    if (x.H < 0) return JATTN_ERR_INVALID_ARG;
    heads += x.H;
    p.H[t] = x.H;
    p.x[t] = x.x;
    p.y[t] = x.y;
    for (int i = 0; i < 3; ++i) {
      p.xs[t][i] = x.x_stride[i];
      p.ys[t][i] = x.y_stride[i];
    }
  }
  if (heads * parts > (1 << 24)) return JATTN_ERR_INVALID_ARG;
  if (B == 0 || S == 0 || heads == 0) return JATTN_OK;
  if (pos == nullptr || freqs == nullptr) return JATTN_ERR_INVALID_ARG;
  if (!aligned(pos, 4) || !aligned(freqs, 8)) return JATTN_ERR_ALIGNMENT;
  for (int t = 0; t < n_tensors; ++t) {
    if (p.H[t] == 0) continue;
    if (p.x[t] == nullptr || p.y[t] == nullptr) return JATTN_ERR_INVALID_ARG;
    if (!aligned(p.x[t], elem_bytes(dtype)) || !aligned(p.y[t], elem_bytes(dtype))) return JATTN_ERR_ALIGNMENT;
  }
  // a head of one tensor is written while another block reads the other tensor's
  if (n_tensors == 2 && p.H[0] > 0 && p.H[1] > 0 && (p.y[0] == p.y[1] || p.y[0] == p.x[1] || p.y[1] == p.x[0]))
    return JATTN_ERR_INVALID_ARG;
  p.B = B;
  p.S = S;
  p.d = d;
  p.parts = parts;
  p.rot = rot;
  p.pos = pos;
  p.pos_stride_b = pos_stride_b;
  p.freqs = freqs;
  p.scale = scale;
  p.inverse = inverse != 0;
  p.tokens = static_cast<long long>(B) * S;
  return from_cuda(jattn::launch_rotary(p, dtype, layout == JATTN_ROTARY_HALF, static_cast<cudaStream_t>(stream)));
}

size_t jattn_linear_workspace(const jattn_linear_shape* s, const void* x, const void* w) {
  if (!linear_sizes(s)) return 0;
  return linear_copies(s, x, w).total;
}

jattn_status jattn_linear(const jattn_linear_shape* s, const void* x, const void* w, const void* bias,
                          const void* residual, void* y, void* workspace, size_t workspace_bytes, void* stream) {
  if (!linear_sizes(s)) return JATTN_ERR_INVALID_ARG;
  if (!is_16bit(s->in_dtype) || !is_float(s->out_dtype)) return JATTN_ERR_UNSUPPORTED;
  if (bias != nullptr && !is_float(s->bias_dtype)) return JATTN_ERR_UNSUPPORTED;
  if (s->act < JATTN_ACT_NONE || s->act > JATTN_ACT_RELU) return JATTN_ERR_UNSUPPORTED;
  if (s->M == 0 || s->N == 0) return JATTN_OK;
  if (x == nullptr || w == nullptr || y == nullptr || y == x || y == w) return JATTN_ERR_INVALID_ARG;
  const int64_t most = int64_t{1} << 38;
  if (s->ldx < s->K || s->ldw < s->K || s->ldy < s->N || s->ldx >= most || s->ldw >= most || s->ldy >= most)
    return JATTN_ERR_INVALID_ARG;
  if (residual != nullptr && (s->ldr < s->N || s->ldr >= most || (residual == y && s->ldr != s->ldy)))
    return JATTN_ERR_INVALID_ARG;
  const int ob = elem_bytes(s->out_dtype);
  if (!aligned(x, 2) || !aligned(w, 2) || !aligned(y, ob)) return JATTN_ERR_ALIGNMENT;
  if (residual != nullptr && !aligned(residual, ob)) return JATTN_ERR_ALIGNMENT;
  if (bias != nullptr && !aligned(bias, elem_bytes(s->bias_dtype))) return JATTN_ERR_ALIGNMENT;
  // operands that TMA cannot address are copied into the workspace
  const LinearCopies c = linear_copies(s, x, w);
  if (c.total > 0 && (workspace == nullptr || workspace_bytes < c.total)) return JATTN_ERR_INVALID_ARG;
  if (c.total > 0 && !aligned(workspace, 256)) return JATTN_ERR_ALIGNMENT;
  jattn::LinearParams p{};
  p.M = s->M;
  p.N = s->N;
  p.K = s->K;
  p.ldy = s->ldy;
  p.ldr = s->ldr;
  p.bias = bias;
  p.residual = residual;
  p.y = y;
  p.in_bf16 = s->in_dtype == JATTN_BF16;
  p.out_dtype = s->out_dtype;
  p.bias_dtype = s->bias_dtype;
  p.act = s->act;
  p.timeout_ns = kTimeoutNs;
  p.status = jattn::device_status_ptr();
  if (p.status == nullptr) return JATTN_ERR_CUDA;
  if (c.total > 0) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const void* src[2] = {c.x ? x : nullptr, c.w ? w : nullptr};
    void* dst[2] = {ws, ws + c.w_at};
    const int64_t ld[2] = {s->ldx, s->ldw}, rows[2] = {s->M, s->N};
    if (jattn::launch_repack(src, dst, ld, rows, s->K, static_cast<cudaStream_t>(stream)) != cudaSuccess)
      return JATTN_ERR_CUDA;
    if (c.x) x = dst[0];
    if (c.w) w = dst[1];
  }
  const jattn::LinearPlan plan = jattn::plan_linear(s->M, s->N, s->K, s->out_dtype);
  CUtensorMap tx, tw;
  const int bx = plan.pair ? 128 : (plan.swap ? plan.bn : 128), bw = plan.pair ? plan.bn / 2 : (plan.swap ? 128 : plan.bn);
  if (!matrix_map(&tx, x, s->M, s->K, c.x ? padded(s->K) : s->ldx, bx) ||
      !matrix_map(&tw, w, s->N, s->K, c.w ? padded(s->K) : s->ldw, bw))
    return JATTN_ERR_CUDA;
  return from_cuda(jattn::launch_linear(p, plan, tx, tw, static_cast<cudaStream_t>(stream)));
}

size_t jattn_fwd_diff_workspace(const jattn_diff_shape* shape, jattn_dtype in_dtype) {
  DiffRanges r;
  if (!is_16bit(in_dtype) || diff_ranges(shape, &r) != JATTN_OK) return 0;
  return diff_layout(shape, r, in_dtype == JATTN_BF16).total;
}

jattn_status jattn_fwd_diff(const jattn_diff_shape* s, jattn_dtype in_dtype, const void* q, const void* k, const void* v,
                            const float* lam, float lambda_init, const float* norm_w, float eps,
                            const int32_t* kv_len, const uint8_t* key_mask, void* workspace, size_t workspace_bytes,
                            void* o, float* lse, float softmax_scale, void* stream) {
  if (!is_16bit(in_dtype)) return JATTN_ERR_UNSUPPORTED;
  DiffRanges r;
  const jattn_status st = diff_ranges(s, &r);
  if (st != JATTN_OK) return st;
  if (!std::isfinite(softmax_scale) || !std::isfinite(lambda_init)) return JATTN_ERR_INVALID_ARG;
  if (norm_w != nullptr && (!(eps > 0.f) || !std::isfinite(eps))) return JATTN_ERR_INVALID_ARG;
  if (s->B == 0 || s->S_q == 0) return JATTN_OK;
  if (q == nullptr || lam == nullptr || o == nullptr) return JATTN_ERR_INVALID_ARG;
  if (s->S_kv > 0 && (k == nullptr || v == nullptr)) return JATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lam, 16) ||
      !aligned(norm_w, 16) || !aligned(kv_len, 4) || !aligned(lse, 4))
    return JATTN_ERR_ALIGNMENT;
  const bool in_bf16 = in_dtype == JATTN_BF16;
  const DiffLayout L = diff_layout(s, r, in_bf16);
  const size_t need = L.total;
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return JATTN_ERR_INVALID_ARG;
  if (need > 0 && !aligned(workspace, 256)) return JATTN_ERR_ALIGNMENT;
  // a tile's rows are written while others read q, k and v
  if (o == q || (s->S_kv > 0 && (o == k || o == v))) return JATTN_ERR_INVALID_ARG;
  jattn::DiffParams p{};
  p.B = s->B;
  p.H = s->H;
  p.H_kv = s->H_kv;
  p.S_q = s->S_q;
  p.S_kv = s->S_kv;
  p.n_groups = r.n_groups;
  p.hpg = r.hpg;
  p.R = r.R;
  p.n_rt = r.n_rt;
  p.items = r.items;
  p.items_whole = r.walk.items_whole;
  p.ctas = r.walk.ctas;
  p.merge = r.walk.merge;
  const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt(0.5f * static_cast<float>(s->d));
  p.scale_log2 = scale * 1.4426950408889634f;
  p.lam = lam;
  p.lambda_init = lambda_init;
  p.norm_w = norm_w;
  p.eps = eps;
  p.kv_len = kv_len;
  p.key_mask = key_mask;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (r.walk.merge) {
    p.part_o = reinterpret_cast<float*>(ws + L.part_o);
    p.part_l = reinterpret_cast<float*>(ws + L.part_l);
  }
  if (s->S_kv > jattn::kGatherKeys) {
    p.sums = reinterpret_cast<float*>(ws + L.sums);
    p.sums_m = reinterpret_cast<float*>(ws + L.sums_m);
  }
  const bool widen = in_bf16 && r.widen;
  if (widen) {
    p.v = static_cast<const __nv_bfloat16*>(v);
    for (int i = 0; i < 3; ++i) p.v_stride[i] = s->v_stride[i];
    p.v16 = reinterpret_cast<__half*>(ws + L.v16);
    p.v_amax = reinterpret_cast<uint32_t*>(ws + L.v_amax);
  }
  p.timeout_ns = kTimeoutNs;
  p.status = jattn::device_status_ptr();
  if (p.status == nullptr) return JATTN_ERR_CUDA;
  CUtensorMap tq, tk, tv;
  // without keys nothing is loaded: any valid address does
  const void* kb = s->S_kv > 0 ? k : q;
  const void* vb = s->S_kv > 0 ? v : q;
  const int64_t skv = s->S_kv > 0 ? s->S_kv : 1;
  const int64_t D = s->d, contiguous[3] = {s->H_kv * skv * D, skv * D, D};
  const int64_t* vs = widen ? contiguous : s->v_stride;
  if (widen) vb = p.v16;
  if (!heads_map(&tq, q, s->d, r.R, r.n_groups, s->B, r.row_stride, r.group_stride, s->q_stride[0],
                 r.R <= jattn::kQuadRows ? jattn::kQuadRows : 128) ||
      !heads_map(&tk, kb, s->d, skv, s->H_kv, s->B, s->k_stride[2], s->k_stride[1], s->k_stride[0]) ||
      !heads_map(&tv, vb, s->d, skv, s->H_kv, s->B, vs[2], vs[1], vs[0]))
    return JATTN_ERR_CUDA;
  return from_cuda(jattn::launch_diff_attn(p, s->d, in_bf16, tq, tk, tv,
                                           static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
