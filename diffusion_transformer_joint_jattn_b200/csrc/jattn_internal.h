// Parameter blocks and launchers shared by the C-ABI layer (jattn_api.cu)
// and the kernel translation units.  Not part of the public interface.
#pragma once

#include <cmath>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

namespace jattn {

// Rotary frequencies of the d/2 channel pairs, built on the host once per
// call: pair p lies on axis axis[p] (0 = t, 1 = row, 2 = col: spans of
// split[0], split[1], split[2] channels in that order) and turns by
// pos_axis * omega[p], omega[p] = theta^(-2i/n) for its index i inside its
// axis span of n channels.  Passed by value in the kernel parameters.
struct RopeTable {
  double omega[64];
  uint8_t axis[64];
};

inline RopeTable make_rope_table(double theta, const int split[3], int d) {
  RopeTable t{};
  for (int p = 0; p < d / 2 && p < 64; ++p) {
    int axis, i, n;
    if (p < split[0] / 2) { axis = 0; i = p; n = split[0]; }
    else if (p < (split[0] + split[1]) / 2) { axis = 1; i = p - split[0] / 2; n = split[1]; }
    else { axis = 2; i = p - (split[0] + split[1]) / 2; n = split[2]; }
    t.axis[p] = static_cast<uint8_t>(axis);
    t.omega[p] = std::pow(theta, -2.0 * static_cast<double>(i) / static_cast<double>(n));
  }
  return t;
}

struct RopeParams {
  const __nv_bfloat16* src[3];  // txt, img, ref streams [B, S_part, 3, H, d]
  int S_part[3];
  int B, H, S, d, nblk;
  const int32_t* pos;           // [S, 3]
  double theta;
  int split[3];
  RopeTable rope;               // frequencies of theta / split (make_rope_table)
  void* dst[3];                 // q, k, v [B, H, S, d]
  float* scales;                // e4m3 output: [3][B][H][nblk]
  const float* norm_w;          // query/key RMSNorm weights [3][2][d], or null
  float eps;                    // RMSNorm epsilon
  void* q16;                    // e4m3 output with token repair: also fp16 Q [B, H, S, d], else null
  float* score;                 // with token repair: [2][B, H, S], |k|^2 then |v|^2 per token, else null
  int hp;                       // fp16 output of the high-precision path: power-of-two range scales in
                                //   `scales` ([3][B][H][nblk]), pair statistics and norm factors below
  float* pair_stat;             // hp: [2][B*H][nblk][d/2] max squared channel-pair norm over each block
  float* norm_r;                // hp with norm_w: [2][B*H][S] RMSNorm factor of every Q / K row
  uint32_t* status;
};

// Exact (16-bit) keys and values of the repaired tokens.
struct GatherParams {
  const __nv_bfloat16* src[3];  // txt, img, ref streams [B, S_part, 3, H, d]
  int S_part[3];
  int B, H, S, d, n;            // n repaired tokens per (b, h)
  const int32_t* pos;           // [S, 3]
  double theta;
  int split[3];
  RopeTable rope;
  const float* norm_w;          // as RopeParams
  float eps;
  const int32_t* idx;           // [B*H][n] token indices
  void* k_out;                  // fp16 [B*H][n][d], rotated (and normalised) keys
  void* v_out;                  // fp16 [B*H][n][d]
  uint8_t* k8;                  // e4m3 [B*H][S][d] keys / values of the FP8 pass: the repaired
  uint8_t* v8;                  //   tokens' rows are set to code 0 (logit exactly 0, value 0)
  uint32_t* status;
};

cudaError_t launch_repair_gather(const GatherParams& p, cudaStream_t st);
// Per (b, h): the n largest scores |k|^2 + |v|^2 (ties to the lower index)
// -> idx [B*H][n] in index order, and the key mask [B*H][n_kv][4] words with
// their bits set.  score holds the [2][B*H][S] K and V planes; the K plane is
// overwritten with the sums.
cudaError_t launch_repair_select(float* score, int BH, int S, int n, int n_kv, int32_t* idx,
                                 uint32_t* kmask, cudaStream_t st);

// High-precision 16-bit path: channel pairs per (b, h) whose rotated Q / K
// values get an fp16 low part, and the columns of one correction row
// (hi and lo of 2 * kCorrPairs channels).
constexpr int kCorrPairs = 4;
constexpr int kCorrCols = 4 * kCorrPairs;

struct CorrParams {
  const __nv_bfloat16* src[3];  // txt, img, ref streams [B, S_part, 3, H, d]
  int S_part[3];
  int B, H, BH, S, d, nblk;
  const int32_t* pos;           // [S, 3]
  double theta;
  int split[3];
  RopeTable rope;
  const float* norm_w;          // query/key RMSNorm weights [3][2][d], or null
  const float* norm_r;          // with norm_w: [2][B*H][S] row factors written by the prologue
  const float* scales;          // [3][B][H][nblk] power-of-two range scales written by the prologue
  const float* pair_stat;       // [2][B*H][nblk][d/2] written by the prologue
  int32_t* sel;                 // [B*H][kCorrPairs] selected pairs, ascending
  void* qc;                     // fp16 [B*H][S][kCorrCols]: [hi | lo] of the selected Q channels
  void* kc;                     // fp16 [B*H][S][kCorrCols]: [lo | hi] of the selected K channels
};

cudaError_t launch_qk_correction(const CorrParams& p, cudaStream_t st);

// Block-sparse attention: selection of the key tiles each 256-row query
// block attends to.
struct SparseParams {
  const void* q;                // [B*H][S][d] 16-bit (rotated)
  const void* k;
  int BH, S, d, nblk, n_qb;     // nblk = ceil(S / 128) key tiles, n_qb = ceil(S / 256) query blocks
  float scale;                  // softmax scale
  float tau;                    // keep a key block iff its estimated share >= tau / nblk
  float* pool;                  // [2][B*H][nblk][d] column sums of every 128-token tile of Q, K
  float* logits;                // [B*H][n_qb][nblk] block logits (scratch of the selection)
  int32_t* kv_list;             // [B*H][n_qb][nblk] kept key tiles, ascending (first kv_count entries)
  int32_t* kv_count;            // [B*H][n_qb]
};

cudaError_t launch_block_select(const SparseParams& p, bool in_bf16, cudaStream_t st);

struct QuantParams {
  const void* x;                // [BH, S, d] 16-bit
  void* x8;                     // [BH, S, d] e4m3
  float* scales;                // [BH][nblk]
  int BH, S, d, nblk;
};

struct FwdParams {
  int B, H, S, n_tiles;         // queries: S rows, n_tiles = ceil(S / 128)
  int S_kv, n_kv;               // keys: S_kv rows (= S except for a residual pass), n_kv = ceil(S_kv / 128)
  float scale_log2;             // softmax_scale * log2(e)
  __nv_bfloat16* o;             // [B, S, H, d]
  float* lse;                   // [B, H, S] or null
  const float* scales;          // fp8 and the high-precision fp16 path: [3][B][H][n_tiles]
  const uint32_t* kmask;        // null, or [B*H][n_kv][4] words: bit set = key left out of this pass
  const float* lse_prev;        // null, or [B, H, S]: o already holds a partial result with this
                                // LSE over other keys; the pass merges its own into o (and lse)
  const int32_t* kv_list;       // null, or [B*H][n_qp][n_kv]: the key tiles each pair of query
  const int32_t* kv_count;      //   tiles walks, ascending, and how many ([B*H][n_qp]); n_qp =
                                //   ceil(n_tiles / 2); every count >= 1
  uint32_t* status;
  uint64_t timeout_ns;
  long long* trace;             // development timing probe; always null in the library
};

// Rotary embedding of strided q and k (t = 0, 1).  Strides in elements, over
// (batch entry, token, head).
struct RotaryParams {
  const void* x[2];
  void* y[2];
  int H[2];                     // heads; 0 = tensor absent
  int64_t xs[2][3], ys[2][3];
  int B, S, d, parts, rot;      // each of the `parts` equal parts of a head turns its first rot channels
  const int32_t* pos;           // [B or 1][S][n_axes]
  int64_t pos_stride_b;
  int n_axes;
  int axis_end[3];              // pairs below axis_end[0] turn by axis 0, below axis_end[1] by axis 1, ...
  const double* freqs;          // [rot / 2]
  float scale;                  // factor of the rotated channels
  int inverse;
  long long tokens;             // B * S
  int units, tile, groups, shares;   // set by the launcher
};
cudaError_t launch_rotary(const RotaryParams& p, int dtype, bool half, cudaStream_t st);

// Linear layer y = act(x w^T + bias) + residual.
struct LinearPlan {
  bool pair;                    // 256 x bn tiles by CTA pairs
  bool flush;                   // accumulators emptied into registers on the way
  bool swap;                    // few rows: W's rows are the MMA's rows
  int bn, splits;               // columns of a tile; parts of K of the one-CTA tiles
};
struct LinearParams {
  int M, N, K;
  int64_t ldy, ldr;
  const void* bias;             // [N] or null
  const void* residual;         // [M][N] of out_dtype, or null
  void* y;
  int in_bf16, out_dtype, bias_dtype, act;
  uint32_t* status;
  uint64_t timeout_ns;
  // set by the launcher
  int tiles_a, tiles_b, splits;
  int vec_y, vec_r;             // bytes of the widest aligned access of y's and residual's rows, 0 = elements
};
LinearPlan plan_linear(int M, int N, int K, int out_dtype);
// tx, tw: 2-D maps with 64-element boxes of plan.pair ? 128 : (swap ? bn : 128) rows of x and
// plan.pair ? bn / 2 : (swap ? 128 : bn) rows of w.
cudaError_t launch_linear(LinearParams p, const LinearPlan& plan, const CUtensorMap& tx, const CUtensorMap& tw,
                          cudaStream_t st);
// Copies of up to two [rows][K] 16-bit operands (src null: none) into rows of K rounded up to 8 elements,
// zeros behind K.
cudaError_t launch_repack(const void* const src[2], void* const dst[2], const int64_t ld[2], const int64_t rows[2],
                          int K, cudaStream_t st);

// Differential attention.  n_groups row ranges per batch entry: H_kv ranges
// of the packed rows (head, query) of the heads that share a K/V head, or H
// ranges of one head's queries.
struct DiffParams {
  int B, H, H_kv, S_q, S_kv;
  int n_groups, hpg, R, n_rt;   // heads and rows of a range, its 128-row tiles
  long long items;              // B * n_groups * n_rt
  long long items_whole;        // the items below this number are walked whole, the others shared by all CTAs
  int ctas;                     // of the walk
  int merge;                    // items are shared: parts to merge
  float scale_log2;
  const float* lam;             // [4][H][d / 2]
  float lambda_init;
  const float* norm_w;          // [d] or null
  float eps;
  const int32_t* kv_len;        // [B] or null
  const uint8_t* key_mask;      // [B][S_kv], nonzero = takes part, or null
  __nv_bfloat16* o;             // [B][S_q][H][d]
  float* lse;                   // [2][B][H][S_q] or null
  float* part_o;                // [2 * ctas][2][128][d]: the parts of shared items
  float* part_l;                // [2 * ctas][2][128], log2 units
  float* sums;                  // S_kv > kGatherKeys: [ctas][256][d], every softmax thread's sums of its row
  float* sums_m;                // with sums: [ctas][256], the maxima they are relative to, log2 units
  const __nv_bfloat16* v;       // with v16: the bf16 values it is made from, and their strides in elements
  int64_t v_stride[3];          //   over (batch entry, head, token)
  __half* v16;                  // null, or [B][H_kv][S_kv][d]: fp16 copy of v, divided by a power of two per head
  uint32_t* v_amax;             // with v16: [B][H_kv] bits of the largest finite magnitudes
  uint32_t* status;
  uint64_t timeout_ns;
};
struct DiffWalk {
  long long items_whole;
  int ctas, merge;
};
DiffWalk diff_walk(long long items, int n_rt, int S_kv, int sms);
bool diff_widens_v(long long items, int n_rt, int S_kv, int sms);
// Ranges of at most this many rows are walked by a kernel of their own.
constexpr int kQuadRows = 32;
// A row's accumulator is emptied after this many keys.
constexpr int kGatherKeys = 32768;
// The maps describe (d, rows, heads or ranges, batch) with boxes of 64 x 128 (q's: 64 x 32 where R <= kQuadRows).
cudaError_t launch_diff_attn(const DiffParams& p, int d, bool in_bf16, const CUtensorMap& tq, const CUtensorMap& tk,
                             const CUtensorMap& tv, cudaStream_t st);

// out_kind: 0 = fp16, 1 = bf16, 2 = e4m3
cudaError_t launch_rope_qkv(const RopeParams& p, int out_kind, cudaStream_t st);
cudaError_t launch_quant_fp8(const QuantParams& p, bool in_bf16, cudaStream_t st);

// 16-bit forward (in_bf16 selects the operand type) and e4m3 forward.  The
// tensor maps describe q, k, v as 3-D [BH][S][d] with 128-row boxes.
cudaError_t launch_fwd_f16(const FwdParams& p, int d, bool in_bf16, const CUtensorMap& tq,
                           const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st);
cudaError_t launch_fwd_fp8(const FwdParams& p, int d, const CUtensorMap& tq, const CUtensorMap& tk,
                           const CUtensorMap& tv, cudaStream_t st);
// High-precision 16-bit forward: fp16 operands with power-of-two block scales
// in p.scales and the correction tiles described by tqc / tkc ([BH][S][16]
// fp16, 32-byte swizzle, 128-row boxes).
cudaError_t launch_fwd_f16_hp(const FwdParams& p, int d, const CUtensorMap& tq, const CUtensorMap& tk,
                              const CUtensorMap& tv, const CUtensorMap& tqc, const CUtensorMap& tkc,
                              cudaStream_t st);

// Rows of the K / V tiles the forward kernels walk (the TMA box height).
int fwd_kv_rows();

// The current device's status word (null on error) and multiprocessor count.
uint32_t* device_status_ptr();
int device_sm_count();
// cuTensorMapEncodeTiled of `rank` dimensions of 16-bit elements (128-byte
// swizzle, zeros out of bounds); false on error.  strides in bytes, rank - 1.
bool encode_map16(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                  const uint32_t* box);

cudaError_t launch_selftest_wait(uint32_t* status, uint64_t limit_ns, cudaStream_t st);

// Unique id of the calling thread's current CUDA context (0 when there is
// none or it cannot be read).  Device addresses of file-scope __device__
// variables are cached per context: a cudaDeviceReset makes a new context,
// whose id differs, and the address is looked up again.
unsigned long long current_context_id();

}  // namespace jattn
