// internal.h -- launchers and host-side structures shared by the libhmoe translation units.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "common.cuh"

namespace hmoe {

// Count of kernel launches issued by the library (read by hmoe_launch_count).
void count_launches(int n);

// ---------------------------------------------------------------- routing
int route_chunks(int T);
cudaError_t launch_route(const float* logits, int T, int E, int k, int* ids, float* gates, int* perm,
                         int* offsets, int* chunk_cnt, int* chunk_base, cudaStream_t st);

// perm[t] = t, offsets = {0, T}, gates[t] = 1 (the dense Linear's route geometry).
cudaError_t launch_identity_route(int T, int* perm, int* offsets, float* gates, int num_sms, cudaStream_t st);

// ---------------------------------------------------------------- packing
// Geometry of one expert block inside a tier buffer: W13 tiles then W2 tiles.
struct ExpertGeom {
  int H, I;
  int rt13, kb13, rt2, kb2;  // row tiles / k-blocks of each matrix
  size_t tile;               // tile bytes of the format
  size_t w13_bytes, w2_bytes, expert_bytes;
};
ExpertGeom expert_geom(int H, int I, int fmt);

// nvfp4_nibbles: store NVFP4 codes in the nibble layout of MXFP4 (fp16 operand layers) instead of
// the shift-and-mask layout (bf16 operand layers).
cudaError_t launch_pack_matrix(int fmt, int which, const void* codes, const void* scales, int N, int K, int I,
                               uint8_t* dst, bool nvfp4_nibbles, cudaStream_t st);
// Test export of the dequantised operands (pack.cu): the tensor-core tile, or with
// decode_operand the weight-streaming kernel's operand plus its per-group scales.
cudaError_t launch_debug_dequant(int fmt, int which, const uint8_t* src, int N, int K, int I, void* dst,
                                 float* scales_out, bool decode_operand, int act_type, bool nf3_tile,
                                 cudaStream_t st);

// ---------------------------------------------------------------- streaming GEMM (any T; the decode path)
// Largest number of k-blocks per row tile in a pipeline stage of the
// streaming kernel (a stage holds two row tiles).
constexpr int STREAM_MAX_KBS = 4;
// The streaming kernel's work items are pairs of row tiles (one activation
// load serves both) when the batch can make at least this many W13 pair
// items per CTA, counting min(T * topk, E) token groups; else single row
// tiles, so that small batches keep more SMs busy. The choice depends only
// on the batch size and the layer, so every tier order of a forward makes
// the same choice and sums in the same order.
constexpr int STREAM_PAIR_MIN_ITEMS_PER_CTA = 2;
// One matrix of the expert FFN as the streaming kernel sees it.
struct StreamPhase {
  int rows, K;               // rows = 2I (W13) or H (W2); K = H or I
  int RT, KB;                // row tiles, k-blocks
  int kbs;                   // k-blocks per row tile and pipeline stage, items of two row tiles
  int kbs1;                  // k-blocks per pipeline stage, items of one row tile (up to 2 STREAM_MAX_KBS)
  const uint16_t* act;       // W13: x [T][H] by token; W2: h [S][I] by permuted position (operand type)
  int act_stride;
  size_t kept_off, nf3_off;  // byte offset of this matrix inside an expert's block
};

struct StreamParams {
  const uint8_t* kept_buf;
  const uint8_t* nf3_buf;
  int kept_fmt;
  int act_type;          // ACT_BF16 or ACT_F16: operand, h and output type
  float act_scale13;     // the W13 input's activation global scale (W4A4), else 1
  float act_scale2;      // the W2 input's activation global scale (W4A4), else 1
  int nf3_tile;          // 1: NF3 decoded to the tile values rne(cb * s) (W4A4 layers); 0: raw codes, scale on sums
  int H, I, E, topk, T;
  StreamPhase ph[2];     // [0] W13 (output h), [1] W2 (output y)
  int ph_begin, ph_end;  // phases this launch runs: [0,2) both (W2 items wait on done13), [0,1) or [1,2)
  int group_tokens;      // tokens per token group (<= 8)
  int pair_items;        // 1: work items are pairs of row tiles; 0: single row tiles
  int tier_mask;         // bit 0: kept experts, bit 1: NF3 experts
  size_t kept_expert_bytes, nf3_expert_bytes;
  const int* offsets;
  const int* perm;
  int* queue;                // [2] work-queue head and finished-CTA count, self-cleaning
  int* done13;               // [token groups] finished W13 warp-items per group, self-cleaning ([0,2) only)
  uint16_t* h_out;           // W13 output: [S][I] in the operand type (bf16 or fp16 bits), row = permuted position p
  float* y_out;              // W2 output:  [S][H] fp32, row = flat slot s
  int* status;
  unsigned long long wait_limit_ns;  // bound on every wait
  int debug_no_copies;               // test hook: the producer issues nothing
  ExpertTable tab;
};

int stream_grid(int num_sms);
cudaError_t launch_stream_gemm(const StreamParams& p, int grid, cudaStream_t st);

// ---------------------------------------------------------------- tensor-core grouped GEMM (large T)
struct GroupedParams {
  const uint8_t* kept_buf;
  const uint8_t* nf3_buf;
  int kept_fmt;
  int act_type;        // ACT_BF16 or ACT_F16
  float act_scale;     // this GEMM's input activation global scale (W4A4), else 1
  int which;           // 13: B = gathered x, output h;  2: B = h, output y
  int H, I, E, topk, T;
  int K, RT, KB;
  int tier_mask;
  size_t kept_expert_bytes, nf3_expert_bytes;
  size_t kept_w2_off, nf3_w2_off;
  const int* offsets;
  const int* perm;
  uint16_t* h_out;     // [S][I] in the operand type
  float* y_out;
  int* status;
  unsigned long long wait_limit_ns;
  int pair;            // 1: the CTA-pair kernel; 0: the one-CTA kernel (the default)
  ExpertTable tab;
};
cudaError_t launch_grouped_gemm(const GroupedParams& p, const uint16_t* b_src, int b_rows, int num_sms,
                                cudaStream_t st);
// xg[p] = x[perm[p] / k] for the S permuted slots (2-byte elements of either operand type).
cudaError_t launch_gather_rows(const uint16_t* x, const int* perm, int S, int k, int T, int H, uint16_t* xg,
                               int* status, int num_sms, cudaStream_t st);

// NVFP4 activation quantisation of n_values (a multiple of 16, rows of a
// multiple of 16 laid end to end) with global scale g (actquant.cu). With
// out set: the operand values e2m1 * e4m3 in the activation type (out may be
// x); else the codes (8 bytes per 16 values) and E4M3 scale bytes.
cudaError_t launch_act_quant(const uint16_t* x, long long n_values, float g, int act_type, uint16_t* out,
                             uint8_t* codes, uint8_t* scales, int num_sms, cudaStream_t st);

// out[t][c] = act(sum_j gates[t*k+j] * y[t*k+j][c]), act = bf16 or fp16 by act_type
cudaError_t launch_finalize(const float* y, const float* gates, int T, int k, int H, uint16_t* out, int act_type,
                            cudaStream_t st);

// ---------------------------------------------------------------- rows sorted by expert and back (dispatch.cu)
// One pass of spread (tokens to rows) or collect (rows to tokens).
struct RowsParams {
  int T, H, E, topk, R;    // R: rows of the sorted buffer
  int row_dtype;           // hmoe_row_dtype of v, other, rows and out
  const void* v;           // [T][H]: spread's source; collect's dot operand, or NULL (no dot products)
  const void* other;       // [R][H]: spread's dot operand, or NULL (no dot products)
  const void* rows_in;     // [R][H]: collect's source
  void* rows_out;          // [R][H]: spread's result
  void* out;               // [T][H]: collect's result
  const float* gates;      // [T][topk], or NULL (weights of one)
  const int* ids;          // [T][topk], read with dlogits
  const int* row_slot;     // [R], read by spread where has_pads
  const int* slot_row;     // [T][topk]
  float* dgates;           // [T][topk], or NULL
  float* dlogits;          // [T][E], or NULL
  int* status;
  int has_pads;            // 1: the maps may hold rows without a slot, which spread fills with zeros
};
// The row maps and the rows of one dispatch (p: spread's parameters).
cudaError_t launch_dispatch(const RowsParams& p, const int* perm, const int* offsets, int align, int capacity,
                            int* row_slot, int* slot_row, int* row_offsets, int num_sms, cudaStream_t st);
cudaError_t launch_spread(const RowsParams& p, int num_sms, cudaStream_t st);
cudaError_t launch_collect(const RowsParams& p, int num_sms, cudaStream_t st);

// ---------------------------------------------------------------- low-rank adapters (lora.cu)
// The packed buffer: ranks int32 [slots], scales fp32 [slots] (each padded to
// 256 bytes), then one block per slot. With r16 the slot's rank rounded up to
// 16, a block holds ceil(K / 64) tiles of A, each r16 rows of 64 values in the
// tensor cores' K-major 128-byte-swizzled layout, then ceil(N / 64) tiles of
// B, each 64 rows (in the order of lora_b_byte) of r16 values in the K-major
// layout without swizzle (16-byte core-matrix rows: [r16 / 8][64][8 values]).
// Either tile is r16 * 128 bytes.
// Rows and columns past the rank, K and N hold zeros.
constexpr int LORA_MAX_RANK = 128;
constexpr int LORA_MAX_SLOTS = 512;
constexpr int LORA_MAX_ROWS = 1 << 26;  // of a batch: what a row's word in the plan holds
struct LoraGeom {
  int K, N, slots, max_r16;
  int KB, NB;                  // 64-wide tiles of K and of N
  size_t scale_off, block_off; // byte offsets of the scales and of slot 0's block
  size_t b_off, block_bytes;   // B tiles in a block sized for max_r16, and that block's bytes
};
__host__ __device__ inline LoraGeom lora_geom(int K, int N, int slots, int max_rank) {
  LoraGeom g;
  g.K = K;
  g.N = N;
  g.slots = slots;
  g.max_r16 = (max_rank + 15) / 16 * 16;
  g.KB = (K + 63) / 64;
  g.NB = (N + 63) / 64;
  g.scale_off = ((size_t)slots * 4 + 255) / 256 * 256;
  g.block_off = 2 * g.scale_off;
  g.b_off = (size_t)g.KB * g.max_r16 * 128;
  g.block_bytes = g.b_off + (size_t)g.NB * g.max_r16 * 128;
  return g;
}
// Marks every slot empty (rank 0).
cudaError_t launch_lora_clear(const LoraGeom& g, uint8_t* packed, cudaStream_t st);
cudaError_t launch_lora_load(const LoraGeom& g, uint8_t* packed, int slot, const uint16_t* A, const uint16_t* B,
                             int rank, float scale, cudaStream_t st);
struct LoraParams {
  LoraGeom g;
  const uint8_t* packed;
  int T, act_type;
  const uint16_t* x;
  const uint16_t* base;   // NULL: zeros
  uint16_t* out;
  size_t ldx, ldbase, ldout;  // row strides in elements
  const int* ids;
  int* status;
  unsigned long long wait_limit_ns;
  int tile_rows;          // rows of a tile of the plan
  // Scratch of the larger batches (lora.cu), see LoraScratch.
  int* meta;
  int4* tiles;
  int* perm;
  float* u;
  float* part;
  uint32_t* bound;        // NULL where u's rows have no power of two (lora.cu)
};
// Up to this many rows a batch is one launch that finds its groups itself and
// keeps nothing outside it: no scratch but the (then unused) meta words.
constexpr int LORA_ONE_LAUNCH_ROWS = 128;
// Scratch of a larger batch of T rows: the rows grouped by adapter (perm), cut
// into tiles of up to LORA_TILE_ROWS rows (tiles: adapter or -1, first
// position, rows, rank), A x of every position (u), and the sums of the pieces
// of tiles, two for each CTA (part), a bound on |A x| of every position, in
// bits (bound). meta: tiles with an adapter, all tiles.
constexpr int LORA_TILE_ROWS = 128;
constexpr int LORA_MIN_TILE_ROWS = 16;  // of the plan for the small kernel
constexpr int LORA_MAX_CTAS = 160;
struct LoraScratch {
  size_t meta, tiles, perm, u, bound, part, total;
};
inline LoraScratch lora_scratch(const LoraGeom& g, int T) {
  auto pad = [](size_t b) { return (b + 255) / 256 * 256; };
  const size_t most = (size_t)T / LORA_MIN_TILE_ROWS + (size_t)(T < g.slots + 1 ? T : g.slots + 1);
  LoraScratch s;
  s.meta = 0;
  s.tiles = s.meta + 256;
  s.perm = s.tiles + pad(most * 16);
  s.u = s.perm + pad((size_t)T * 4);
  s.bound = s.u + pad((size_t)T * g.max_r16 * 4);
  s.part = s.bound + pad((size_t)T * 4);
  s.total = T <= LORA_ONE_LAUNCH_ROWS ? s.tiles : s.part + (size_t)LORA_MAX_CTAS * 2 * LORA_TILE_ROWS * g.max_r16 * 4;
  return s;
}
cudaError_t launch_lora_forward(const LoraParams& p, int num_sms, cudaStream_t st);

// Raises a kernel's dynamic shared-memory limit once per device: the
// attribute belongs to the current device, so a process that launches on
// several GPUs sets it on each. done is the kernel's bit mask of devices
// already set (ids 0..63; a higher id sets it on every call).
template <typename Kernel>
inline cudaError_t ensure_smem_attr(Kernel* kernel, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0ull;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

}  // namespace hmoe
